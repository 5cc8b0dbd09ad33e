"""Queries and KV rows rotated by positions of several axes, against the definition in 64 bits and against the same tokens
turned by a table of their own angles on one axis."""
import pytest
import torch

import mla_paged_latent_gb300 as mla
from chunk_helpers import H, generator, normal

pytestmark = pytest.mark.gpu
EPS = 1e-6
ORDERS = {"one": (1, [0] * 32), "sections": (3, [0] * 8 + [1] * 12 + [2] * 12), "in turn": (3, [i % 3 for i in range(32)]),
          "two of four": (4, [3] * 5 + [1] * 27), "four": (4, [3, 0, 2, 1] * 8)}


class Step:
    def __init__(self, seed, tokens, heads, width, layout, order, page=16, max_pos=500, norm=False):
        g = generator(seed)
        self.layout, self.page, self.width, self.norm = layout, page, width, norm
        self.row = mla.ROW_ELEMS[layout]
        self.nope = width - 64
        self.axes, self.axis_of_pair = ORDERS[order]
        self.pages = -(-tokens // page) + 1
        self.q = normal(g, tokens, heads, width)
        self.raw = normal(g, tokens, self.row)
        self.slots = torch.randperm(self.pages * page, generator=g, device="cuda")[:tokens].int()
        self.positions = torch.randint(max_pos, (self.axes, tokens), generator=g, device="cuda", dtype=torch.int32)
        self.freqs = torch.randn(max_pos, 64, generator=g, device="cuda")
        self.gain = (1 + 0.2 * torch.randn(512, generator=g, device="cuda")).to(torch.bfloat16)
        self.q_gain = (1 + 0.2 * torch.randn(512, generator=g, device="cuda")).to(torch.bfloat16)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def new_cache(self):
        return torch.zeros(self.pages, mla.mla_page_bytes(self.layout, self.page), dtype=torch.uint8, device="cuda")

    def turns(self):
        """(cos, sin) of every token and pair, fp32 [tokens, 64]."""
        at = self.positions[torch.tensor(self.axis_of_pair, device="cuda")].long().clamp(0, self.freqs.shape[0] - 1)
        return self.freqs.view(-1, 32, 2)[at, torch.arange(32, device="cuda")[:, None]].transpose(0, 1).reshape(-1, 64).contiguous()

    def call(self, q_nope=None, q_pe=None, out=None, cache=None, raw=None, **kw):
        out = torch.full_like(self.q, 7.0) if out is None else out
        cache = self.new_cache() if cache is None else cache
        mla.mla_qkv_norm_rope_axes(self.q[..., :self.nope] if q_nope is None else q_nope,
                                   self.q[..., self.nope:] if q_pe is None else q_pe, self.raw if raw is None else raw,
                                   self.slots, self.positions, self.axis_of_pair, self.gain, EPS, self.freqs, out, cache,
                                   self.layout, self.page, q_norm_weight=self.q_gain if self.norm else None,
                                   q_eps=EPS if self.norm else None, status=self.status, **kw)
        return out, cache

    def reference(self):
        """(queries, their bound): sums of 512 squares, the root and the products are off by 2^-20 of the value in fp32, a
        rotation by 2^-22 of its two terms' magnitudes on top of its inputs', and the result is rounded once."""
        x = self.q.double()
        off = torch.zeros_like(x)
        if self.norm:
            rms = torch.sqrt((x[..., :512] ** 2).mean(-1, keepdim=True) + EPS)
            x[..., :512] = x[..., :512] / rms * self.q_gain.double()
            off[..., :512] = 2.0 ** -20 * x[..., :512].abs()
        t = self.turns().double().view(-1, 1, 32, 2)
        u, v = x[..., self.nope::2].clone(), x[..., self.nope + 1::2].clone()
        c, s = t[..., 0], t[..., 1]
        near = 2.0 ** -19 if self.norm else 2.0 ** -22
        off[..., self.nope::2] = near * ((u * c).abs() + (v * s).abs())
        off[..., self.nope + 1::2] = near * ((u * s).abs() + (v * c).abs())
        x[..., self.nope::2], x[..., self.nope + 1::2] = u * c - v * s, u * s + v * c
        return x, off * (1 + H) + H * x.abs() + 1e-38


WIDTHS = [(192, 0), (192, 2), (192, 4), (576, 0), (576, 2), (576, 4), (512, 1), (512, 3)]


@pytest.mark.parametrize("width, layout", WIDTHS)
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("norm", [False, True])
def test_queries_and_rows(width, layout, order, norm):
    if width == 192 and norm:
        norm = False
    s = Step(1, 37, 6, width, layout, order, norm=norm)
    out, cache = s.call()
    want, bound = s.reference()
    assert ((out.double() - want).abs() <= bound).all()
    # the rows: bit for bit those of the fused write by a table that holds each token's angles
    same = s.new_cache()
    at = torch.arange(37, dtype=torch.int32, device="cuda")
    mla.mla_kv_write_norm_rope(s.raw, s.slots, at, s.gain, EPS, s.turns(), same, layout, s.page)
    assert torch.equal(cache, same)
    assert s.status.item() == 0


@pytest.mark.parametrize("width, layout", [(576, 0), (576, 4), (512, 1), (512, 3)])
@pytest.mark.parametrize("norm", [False, True])
def test_one_axis_is_the_ordinary_step(width, layout, norm):
    s = Step(2, 50, 5, width, layout, "one", norm=norm)
    out, cache = s.call()
    q, kv = torch.empty_like(out), s.new_cache()
    mla.mla_qkv_norm_rope(s.q[..., :s.nope], s.q[..., s.nope:], s.raw, s.slots, s.positions[0].contiguous(), s.gain, EPS, s.freqs,
                          q, kv, layout, s.page, q_norm_weight=s.q_gain if norm else None, q_eps=EPS if norm else None)
    assert torch.equal(cache, kv)
    assert torch.equal(out, q)


@pytest.mark.parametrize("tokens, heads", [(1, 1), (1, 128), (3, 7), (65, 9), (700, 128), (2000, 3)])
@pytest.mark.parametrize("width, layout", [(192, 0), (576, 2), (512, 3)])
def test_sizes(tokens, heads, width, layout):
    s = Step(3, tokens, heads, width, layout, "four")
    want, bound = s.reference()
    assert ((s.call()[0].double() - want).abs() <= bound).all()


@pytest.mark.parametrize("width, layout", [(192, 4), (576, 0), (512, 1)])
@pytest.mark.parametrize("norm", [False, True])
def test_in_place_and_strided(width, layout, norm):
    s = Step(4, 33, 10, width, layout, "in turn", norm=norm and width != 192)
    want, cache = s.call()
    nope = s.q[..., :s.nope].transpose(0, 1).contiguous().transpose(0, 1)
    pe = torch.zeros(33, 10, 200, dtype=torch.bfloat16, device="cuda")
    pe[..., 136:] = s.q[..., s.nope:]
    raw = torch.zeros(33, s.row + 24, dtype=torch.bfloat16, device="cuda")
    raw[:, :s.row] = s.raw
    out, other = s.call(nope, pe[..., 136:], raw=raw[:, :s.row])
    assert torch.equal(out, want) and torch.equal(other, cache)
    q = s.q.clone()
    out, other = s.call(q[..., :s.nope], q[..., s.nope:], out=q)
    assert torch.equal(q, want) and torch.equal(other, cache)
    # in place for one part only
    q = s.q.clone()
    q[..., s.nope:] = 0
    s.call(q[..., :s.nope], s.q[..., s.nope:], out=q)
    assert torch.equal(q, want)


@pytest.mark.parametrize("width, layout", [(192, 0), (576, 4), (512, 1)])
def test_padding_and_bad_positions(width, layout):
    s = Step(5, 24, 6, width, layout, "two of four")
    clean, clean_cache = s.call()
    s.positions[0, 2] = -1            # no pair has axis 0: not read
    s.positions[3, 4] = 500           # past the table
    s.positions[1, 5] = -3            # before it, on one axis only, with a slot
    s.slots[6] = -1                   # no row, queries all the same
    s.positions[:, 7], s.slots[7] = -1, -1          # padding
    s.positions[1, 8], s.slots[8] = -1, -1          # half of it: reported
    out, cache = s.call()
    assert s.status.item() == 8
    gone = [4, 5, 7, 8]
    kept = [i for i in range(24) if i not in gone]
    assert torch.equal(out[kept], clean[kept]) and (out[gone] == 7).all()
    rows, want = (torch.empty(24, s.row, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = Step(5, 24, 6, width, layout, "two of four").slots
    mla.mla_kv_read(cache, layout, s.page, slots, rows)
    mla.mla_kv_read(clean_cache, layout, s.page, slots, want)
    kept = [i for i in kept if i != 6]
    assert torch.equal(rows[kept], want[kept]) and (rows[gone + [6]] == 0).all()
    s = Step(5, 24, 6, width, layout, "two of four")
    s.positions[:, 7], s.slots[7] = -1, -1
    s.call()
    assert s.status.item() == 0
    s.slots[3] = s.pages * s.page + 2
    out, _ = s.call()
    assert s.status.item() == 4 and torch.equal(out[3], clean[3])
