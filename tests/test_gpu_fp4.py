"""The 4-bit latent cache on the GPU: its write, its read back, the step that prepares queries and
appends KV rows, and the decode over it (dense, causal, sink, top-k, windows, split, captured),
against the oracle and plain float64 forms, with bounds derived from the roundings."""
import numpy as np
import pytest
import torch

import mla_paged_latent_gb300 as mla
import oracle
import workloads
from fp4_helpers import assert_decode, attend, bf16_f64, decode, dense_slots, listed_slots, rows_of
from gpu_helpers import DeviceWorkload, bf16_tensor, bf16_to_f64

pytestmark = pytest.mark.gpu
FP4 = [mla.MLA_KV_FP4_448_UE8M0, mla.MLA_KV_FP4_512_UE8M0]
LAYOUTS = [0, 1, 2, 3, 4]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_paged_latent_gb300 import build
    build.build()
    mla.load()


def _bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(
        np.uint16).copy()


def _bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _table(max_pos):
    theta = np.outer(np.arange(max_pos), 10000.0 ** (-np.arange(32) / 32.0))
    f = np.zeros((max_pos, 64), np.float32)
    f[:, 0::2], f[:, 1::2] = np.cos(theta), np.sin(theta)
    return f


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------------- write and read back
@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("ps,n", [(1, 3), (8, 1), (16, 70), (64, 200)])
def test_kv_write_bit_exact(layout, ps, n):
    rng = np.random.default_rng(100 + layout + n)
    pages = n // ps + 3
    width = workloads._DQK[layout]
    kv0 = rng.integers(0, 256, (pages, workloads.page_bytes(layout, ps)), dtype=np.uint8)
    bits = _bits(rng.standard_normal((n, width)) * 2.0 ** rng.integers(-30, 30, (n, 1)))
    if n > 20:
        x = np.zeros((10, width))
        x[1] = -0.0
        x[2] = 1e-12
        x[3, :64] = np.linspace(-7, 7, 64)
        x[4, :32] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4     # every tie of a group with e = 0
        x[5, :32] = [-0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0] * 4
        x[6] = 3e38
        x[7] = 1e-40                                                     # bf16 subnormals
        bits[:10] = _bits(x)
        bits[8, 3], bits[8, 40] = 0x7FC0, 0xFFC1                         # NaN of either sign, two groups
        bits[9, 70], bits[9, 71] = 0x7F80, 0xFF80                        # infinities
    slots = rng.permutation(pages * ps)[:n].astype(np.int32)
    ok = slots.copy()
    if n > 20:
        slots[11], slots[12] = -1, pages * ps + 3                        # skipped; reported and not written
        ok[11] = ok[12] = -1
    ref = oracle.kv_write(bits, ok, kv0, layout, ps)
    kv, st = _cuda(kv0), _status()
    mla.mla_kv_write(bf16_tensor(bits), _cuda(slots), kv, layout, ps, status=st)
    diff = np.argwhere(kv.cpu().numpy() != ref)
    assert diff.size == 0, f"{len(diff)} bytes differ, first at {diff[:5].tolist()}"
    assert int(st.item()) == (4 if n > 20 else 0)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("ps", [8, 64])
def test_kv_read_exact(layout, ps):
    """Rows at slots in any order, some twice, against the oracle's decoded row rounded to bf16;
    negative slots and slots past the cache leave their rows as they were."""
    rng = np.random.default_rng(110 + layout + ps)
    pages, n = 7, 90
    width = workloads._DQK[layout]
    bits = _bits(rng.standard_normal((pages * ps, width)) * 2.0 ** rng.integers(-9, 9, (pages * ps, 1)))
    kv = oracle.kv_write(bits, np.arange(pages * ps, dtype=np.int32),
                         np.zeros((pages, workloads.page_bytes(layout, ps)), np.uint8), layout, ps)
    slots = rng.integers(0, pages * ps, n).astype(np.int32)
    slots[5], slots[6], slots[89] = slots[4], -1, pages * ps
    before = rng.integers(0, 1 << 15, (n, width), dtype=np.uint16)
    rows, st = bf16_tensor(before), _status()
    mla.mla_kv_read(_cuda(kv), layout, ps, _cuda(slots), rows, status=st)
    got = _bits_of(rows)
    assert int(st.item()) == 4
    for r, s in enumerate(slots):
        want = before[r] if s < 0 or s >= pages * ps else oracle.bf16_encode(
            oracle.decode_row(kv, layout, ps, s // ps, s % ps))
        assert np.array_equal(got[r], want), r
    mla.mla_kv_read(_cuda(kv), layout, ps, _cuda(slots[:0]), rows[:0])  # nothing to do


@pytest.mark.parametrize("layout", FP4)
def test_kv_gather_exact(layout):
    w = workloads.generate(workloads.dsv3(batch=2, seqlens=(77, 150), len_dist="fixed", page_size=16, layout=layout,
                                          new_rows=False))
    for b, L in enumerate((77, 150)):
        out = torch.empty(L, workloads._DQK[layout], device="cuda")
        mla.mla_kv_gather(_cuda(w.kv_cache), layout, 16, _cuda(w.block_table[b]), L, out)
        assert np.array_equal(out.cpu().numpy().astype(np.float64),
                              oracle.kv_gather(w.kv_cache, layout, 16, w.block_table[b], L))


@pytest.mark.parametrize("layout", FP4)
def test_nan_scale_reads_as_nan(layout):
    kv = np.zeros((1, workloads.page_bytes(layout, 8)), np.uint8)
    kv[:, 8 * workloads._ROW_BYTES[layout]] = 255   # row 0, group 0
    rows = torch.empty(1, workloads._DQK[layout], dtype=torch.bfloat16, device="cuda")
    mla.mla_kv_read(_cuda(kv), layout, 8, _cuda(np.zeros(1, np.int32)), rows)
    assert rows[0, :32].isnan().all() and not rows[0, 32:].isnan().any()


def _as_held(bits, nope):
    """What a 4-bit row keeps of the bf16 row that was written, in float64, by group."""
    kv = oracle.kv_write(bits[None], np.zeros(1, np.int32),
                         np.zeros((1, workloads.page_bytes(3 if nope == 448 else 4, 1)), np.uint8),
                         3 if nope == 448 else 4, 1)
    return oracle.decode_row(kv, 3 if nope == 448 else 4, 1, 0, 0)


@pytest.mark.parametrize("layout", FP4)
def test_kv_write_norm_rope(layout):
    """The fused write: the kernel normalises in fp32 and the oracle in fp64, so a value within about
    2^-20 of a bf16 rounding border may land on the other side: one bf16 step (2^-7), which may carry a
    code over its own border: the two e2m1 neighbours of a group's grid. Nearly all bytes agree."""
    rng = np.random.default_rng(120 + layout)
    ps, pages, n, max_pos, eps = 16, 12, 150, 4096, 1e-6
    width, nope, rb = workloads._DQK[layout], workloads._NOPE[layout], workloads._ROW_BYTES[layout]
    kv0 = rng.integers(0, 256, (pages, workloads.page_bytes(layout, ps)), dtype=np.uint8)
    raw = _bits(rng.standard_normal((n, width)) * 2.0 ** rng.integers(-20, 20, (n, 1)))
    raw[0] = 0
    w, freqs = _bits(1 + 0.2 * rng.standard_normal(512)), _table(max_pos)
    pos = rng.integers(0, max_pos, n).astype(np.int32)
    pos[2], pos[3] = -1, max_pos
    slots = rng.permutation(pages * ps)[:n].astype(np.int32)
    slots[4] = -1
    ref = oracle.kv_write_norm_rope(raw, slots, pos, w, eps, freqs, kv0, layout, ps)
    kv, st = _cuda(kv0), _status()
    mla.mla_kv_write_norm_rope(bf16_tensor(raw), _cuda(slots), _cuda(pos), bf16_tensor(w), eps, _cuda(freqs), kv, layout,
                               ps, status=st)
    got = kv.cpu().numpy()
    assert int(st.item()) == 8
    assert np.mean(got != ref) <= 2e-3
    written = np.zeros_like(kv0, bool)
    for r, s in enumerate(slots):
        if s < 0 or not 0 <= pos[r] < max_pos:
            continue
        p, o = divmod(int(s), ps)
        written[p, o * rb:(o + 1) * rb] = True
        written[p, ps * rb + 16 * o:ps * rb + 16 * o + 16] = True
        g, e = rows_of(got, layout, ps, [s])[0], rows_of(ref, layout, ps, [s])[0]
        top = np.abs(e[:nope]).reshape(-1, 32).max(1).repeat(32)
        # neighbours on a grid whose largest step is a third of its largest value, or (a group maximum on the
        # border of two scales) on grids a factor of two apart
        assert np.all(np.abs(g[:nope] - e[:nope]) <= top * (2 / 3) + 1e-38)
        assert np.all(np.abs(g[nope:] - e[nope:]) <= np.abs(e[nope:]) * 2.0 ** -7 + 1e-38)
    assert np.array_equal(got[~written], kv0[~written])


# ----------------------------------------------------------------------------- queries and KV rows
def _qkv_inputs(rng, layout, T, N, max_pos, form):
    """Device queries by `form` and their plain [T, N, width] bits."""
    width = workloads._DQK[layout]
    nope = width - 64
    bits = _bits(rng.standard_normal((T, N, width)) * 2.0 ** rng.integers(-6, 6, (T, N, 1)))
    q = bf16_tensor(bits)
    if form == "heads first":       # the absorbed part from a product batched over heads, RoPE from another tensor
        qn = q[..., :nope].transpose(0, 1).contiguous().transpose(0, 1)
        big = torch.zeros(T, N, 192, dtype=torch.bfloat16, device="cuda")
        big[..., 128:] = q[..., nope:]
        return qn, big[..., 128:], bits
    return q[..., :nope], q[..., nope:], bits


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,N,norm,form", [(1, 1, True, "rows"), (3, 16, False, "heads first"),
                                           (13, 5, True, "heads first"), (40, 64, True, "rows"),
                                           (9, 128, False, "rows")])
def test_qkv_norm_rope(layout, T, N, norm, form):
    """Queries within half a bf16 step of the float64 result, with 2^-18 for the fp32 arithmetic (512 sums,
    one square root, four products: relative to the value, or to its RoPE pair); KV bytes equal to the
    fused write's."""
    rng = np.random.default_rng(130 + layout + T)
    ps, max_pos, eps = 16, 700, 1e-5
    width = workloads._DQK[layout]
    pages = T // ps + 2
    qn, qp, bits = _qkv_inputs(rng, layout, T, N, max_pos, form)
    wide = bf16_tensor(_bits(rng.standard_normal((T, width + 64))))
    kv_raw = wide[:, 64:]                           # a slice of a wider projection
    kw, qw = bf16_tensor(_bits(1 + 0.2 * rng.standard_normal(512))), bf16_tensor(_bits(1 + 0.2 * rng.standard_normal(512)))
    freqs = _table(max_pos)
    pos = rng.integers(0, max_pos, T).astype(np.int32)
    slots = rng.permutation(pages * ps)[:T].astype(np.int32)
    want_status = 0
    if T > 8:
        pos[1], slots[1] = -1, -1                   # padding: nothing written, nothing said
        pos[2] = max_pos                            # reported
        slots[3] = -1                               # a token without a KV row: its queries are prepared
        slots[4] = pages * ps                       # past the cache: its queries are prepared
        want_status = 8 | 4
    kv0 = rng.integers(0, 256, (pages, workloads.page_bytes(layout, ps)), dtype=np.uint8)
    before = rng.integers(0, 1 << 15, (T, N, width), dtype=np.uint16)
    q_out, kv, st = bf16_tensor(before), _cuda(kv0), _status()
    mla.mla_qkv_norm_rope(qn, qp, kv_raw, _cuda(slots), _cuda(pos), kw, eps, _cuda(freqs), q_out, kv, layout, ps,
                          q_norm_weight=qw if norm else None, q_eps=eps if norm else None, status=st)
    assert int(st.item()) == want_status
    kv2, st2 = _cuda(kv0), _status()
    mla.mla_kv_write_norm_rope(kv_raw.contiguous(), _cuda(slots), _cuda(pos), kw, eps, _cuda(freqs), kv2, layout, ps,
                               status=st2)
    assert torch.equal(kv, kv2)
    got = _bits_of(q_out)
    skip = (pos < 0) | (pos >= max_pos)
    assert np.array_equal(got[skip], before[skip])
    x = bf16_f64(bits[~skip])
    p = pos[~skip]
    if norm:
        x[..., :512] *= bf16_f64(_bits_of(qw)) / np.sqrt((x[..., :512] ** 2).mean(-1, keepdims=True) + float(np.float32(eps)))
    z = x[..., -64::2] + 1j * x[..., -63::2]
    z = z * (freqs[p, 0::2].astype(np.float64) + 1j * freqs[p, 1::2])[:, None]
    size = np.abs(x)
    size[..., -64::2] = size[..., -63::2] = np.abs(z)
    x[..., -64::2], x[..., -63::2] = z.real, z.imag
    err = np.abs(bf16_f64(got[~skip]) - x)
    assert np.all(err <= np.abs(x) * 2.0 ** -8 + size * 2.0 ** -18 + 1e-38)
    if not norm:                                    # what is only copied keeps its bits
        assert np.array_equal(got[~skip][..., :width - 64], bits[~skip][..., :width - 64])


def test_qkv_norm_without_gain_is_gain_one():
    rng = np.random.default_rng(140)
    T, N, ps = 6, 8, 16
    for layout in (3, 4):
        width = workloads._DQK[layout]
        qn, qp, _ = _qkv_inputs(rng, layout, T, N, 10, "rows")
        args = (qn, qp, bf16_tensor(_bits(rng.standard_normal((T, width)))), _cuda(np.arange(T, dtype=np.int32)),
                _cuda(np.arange(T, dtype=np.int32)), torch.ones(512, dtype=torch.bfloat16, device="cuda"), 1e-6,
                _cuda(_table(10)))
        a, b = (torch.empty(T, N, width, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kv = torch.zeros(1, mla.mla_page_bytes(layout, ps), dtype=torch.uint8, device="cuda")
        mla.mla_qkv_norm_rope(*args, a, kv, layout, ps, q_eps=1e-6)
        mla.mla_qkv_norm_rope(*args, b, kv, layout, ps, q_eps=1e-6,
                              q_norm_weight=torch.ones(512, dtype=torch.bfloat16, device="cuda"))
        assert torch.equal(a, b)


@pytest.mark.parametrize("layout", [1, 3, 4])
def test_qkv_in_place(layout):
    """q_out may be the queries' own memory, row for row."""
    rng = np.random.default_rng(150 + layout)
    T, N, ps = 11, 24, 16
    width = workloads._DQK[layout]
    q = bf16_tensor(_bits(rng.standard_normal((T, N, width))))
    kv_raw = bf16_tensor(_bits(rng.standard_normal((T, width))))
    i = _cuda(np.arange(T, dtype=np.int32))
    ones = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    outs = []
    for own in (False, True):
        qq = q.clone()
        out = qq if own else torch.empty_like(qq)
        kv = torch.zeros(2, mla.mla_page_bytes(layout, ps), dtype=torch.uint8, device="cuda")
        mla.mla_qkv_norm_rope(qq[..., :width - 64], qq[..., width - 64:], kv_raw, i, i, ones, 1e-6, _cuda(_table(32)), out,
                              kv, layout, ps, q_norm_weight=ones, q_eps=1e-6)
        outs.append(out)
    assert torch.equal(*outs)


def test_qkv_many_rows():
    """More query rows than one wave of blocks, an odd count, each row where it belongs."""
    rng = np.random.default_rng(160)
    T, N, layout, ps = 1003, 40, 4, 64
    bits = rng.integers(0, 1 << 14, (T, N, 576)).astype(np.uint16)     # finite, positive, all different rows
    q = bf16_tensor(bits)
    kv = torch.zeros(16, mla.mla_page_bytes(layout, ps), dtype=torch.uint8, device="cuda")
    i = _cuda(np.arange(T, dtype=np.int32))
    out = torch.empty_like(q)
    freqs = torch.zeros(T, 64, device="cuda")
    freqs[:, 0::2] = 1                                                 # the identity
    mla.mla_qkv_norm_rope(q[..., :512], q[..., 512:], q[:, 0].contiguous(), i, i,
                          torch.ones(512, dtype=torch.bfloat16, device="cuda"), 1e-6, freqs, out, kv, layout, ps)
    assert torch.equal(out, q)


# ----------------------------------------------------------------------------- decode
def _run(w, num_sms=None, min_splits=None):
    d = DeviceWorkload(w)
    out, lse = d.run(num_sms=num_sms, min_splits=min_splits, write=False)
    return d, out, lse


LENS = {"edges": (0, 1, 63, 64, 65, 127, 128, 129), "ragged": (200, 1, 515, 64, 1000), "one": (1,), "long": (3001, 130)}


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("lens,heads,ps,splits", [
    ("edges", 16, 16, 1), ("edges", 128, 64, 1), ("edges", 64, 8, 3), ("ragged", 1, 64, 1), ("ragged", 20, 32, 2),
    ("ragged", 130, 128, 1), ("one", 128, 64, 1), ("one", 8, 256, 4), ("long", 64, 64, 1), ("long", 128, 16, 6)])
def test_decode_dense(layout, lens, heads, ps, splits):
    w = workloads.generate(workloads.dsv4(batch=len(LENS[lens]), seqlens=LENS[lens], len_dist="fixed", heads=heads,
                                          layout=layout, page_size=ps, sink=heads != 20, new_rows=False,
                                          tail_fill="nan", seed=heads + splits))
    _, out, lse = _run(w, min_splits=splits)
    assert_decode(out, lse, decode(w, w.kv_cache, dense_slots(w)), f"{lens} {heads}")


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("sq,heads,sms", [(2, 64, None), (4, 128, None), (3, 16, None), (5, 20, 3), (1, 64, 2), (7, 9, None)])
def test_decode_causal(layout, sq, heads, sms):
    """Draft tokens see the rows up to their own; requests shorter than the drafts leave some with none."""
    w = workloads.generate(workloads.verify(batch=4, sq=sq, heads=heads, seqlens=(sq - 1, sq, 64 + sq, 333),
                                            len_dist="fixed", layout=layout, new_rows=False, tail_fill="nan"))
    _, out, lse = _run(w, num_sms=sms)
    assert_decode(out, lse, decode(w, w.kv_cache, dense_slots(w)), f"sq {sq}")


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("topk,heads,sq,splits", [(1, 16, 1, 1), (63, 64, 1, 1), (200, 128, 1, 3), (257, 64, 2, 2),
                                                  (130, 24, 1, 1)])
def test_decode_topk(layout, topk, heads, sq, splits):
    w = workloads.generate(workloads.sparse(batch=3, sq=sq, heads=heads, seqlens=(1000, 90, 300), layout=layout, topk=topk,
                                            page_size=32, min_splits=splits, new_rows=False))
    idx = w.indices
    idx[0, :topk // 3] = -1                       # holes at the front
    if topk > 60:
        idx[0, 50:56] = idx[0, 49]                # the same row several times
        idx[0, 60] = 1000                         # past the request
    idx[-1] = -1                                  # a token with nothing listed
    _, out, lse = _run(w)
    assert_decode(out, lse, decode(w, w.kv_cache, listed_slots(w)), f"top {topk}")


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("window,ps,heads", [(1, 8, 64), (96, 64, 64), (128, 128, 20), (40, 32, 128),
                                             (300, 256, 128)])
def test_decode_windows(layout, window, ps, heads):
    w = workloads.generate(workloads.dsv4(batch=9, seqlens=(300,) * 9, len_dist="fixed", heads=heads, layout=layout,
                                          page_size=ps, new_rows=False))
    rng = np.random.default_rng(170 + window)
    pages, T = w.kv_cache.shape[0], 9
    idx, lens = np.full((T, window), -1, np.int32), rng.integers(0, window + 1, T).astype(np.int32)
    lens[0], lens[1] = 0, window
    for t in range(T):
        n = int(lens[t])
        first = int(rng.integers(0, pages - 1)) * ps + int(rng.integers(0, max(1, min(ps, 2 * ps - n))))
        idx[t, :n] = first + np.arange(n)
    runs = torch.zeros(T, 4, dtype=torch.int32, device="cuda")
    mla.mla_swa_plan(_cuda(idx), ps, 1, runs, topk_lengths=_cuda(lens))
    plan = mla.mla_decode_plan(np.full(T, window, np.int32), 1, heads, window)
    ws = mla.alloc_workspace(plan.workspace_bytes)
    out = torch.empty(T, heads, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(T, heads, device="cuda")
    mla.mla_decode_runs(bf16_tensor(w.q), _cuda(w.kv_cache), layout, ps, runs, window, 1, w.cfg.sm_scale,
                        _cuda(plan.sched), _cuda(plan.num_splits), plan.num_partitions, plan.total_splits, ws, out, lse,
                        sink=_cuda(w.sink))
    assert mla.mla_read_status(ws) == 0
    assert_decode(bf16_to_f64(out), lse.cpu().numpy().astype(np.float64),
                  decode(w, w.kv_cache, lambda t: idx[t, :lens[t]]), f"window {window}")


@pytest.mark.parametrize("layout", FP4)
def test_decode_moving_maximum(layout):
    """Scores that climb along the context by far more than the rescale threshold, and fall again: the running
    maximum has to move many times, in every head at its own rows."""
    w = workloads.generate(workloads.dsv3(batch=2, seqlens=(1500, 700), len_dist="fixed", heads=64, layout=layout,
                                          new_rows=False, seed=5))
    ps, rb, nope = 64, workloads._ROW_BYTES[layout], workloads._NOPE[layout]
    kv = w.kv_cache.copy()
    q = np.zeros(w.q.shape, np.float32)
    rng = np.random.default_rng(6)
    q[..., :nope] = rng.standard_normal(q[..., :nope].shape) * 0.02
    q[..., nope] = 1 + rng.random(q.shape[:2])                  # the first RoPE element carries the climb
    w.q[:] = _bits(q)
    for b, L in enumerate(w.seqlens):
        j = np.arange(L)
        climb = np.where(j < 2 * L // 3, j * 4.0, 8.0 * (L - j)) / w.cfg.sm_scale
        page = w.block_table[b, j // ps]
        col = (j % ps) * rb + rb - 128
        bits = _bits(climb)
        kv[page, col], kv[page, col + 1] = bits & 255, bits >> 8
    w.kv_cache[:] = kv
    _, out, lse = _run(w)
    q64 = bf16_f64(w.q)
    for b in range(2):
        k = rows_of(w.kv_cache, layout, ps, dense_slots(w)(b))
        ref, ref_lse, mean, _ = attend(q64[b], k, float(np.float32(w.cfg.sm_scale)))
        # scores reach 12000: fp32 keeps them to 2^-10 absolute (12000 * 2^-24 for the sum and as much for the
        # scale and the exponent's argument), which moves a weight by 3 * 2^-10 at most
        assert np.all(np.abs(out[b] - ref) <= (2.0 ** -8 + 2 * 3 * 2.0 ** -10) * mean + 2.0 ** -8 * np.abs(ref))
        assert np.all(np.abs(lse[b] - ref_lse) <= 4 * 2.0 ** -10)


@pytest.mark.parametrize("layout", FP4)
def test_decode_wide_scales(layout):
    """Scale bytes from 20 to 140 in one cache (values from 2^-107 to 6 * 2^13): no scale is flushed or clipped. The
    queries' NoPE part is zero, so the scores stay small; V is what ranges."""
    w = workloads.generate(workloads.dsv3(batch=2, seqlens=(300, 77), len_dist="fixed", heads=16, layout=layout,
                                          new_rows=False, seed=7))
    ps, rb, nope = 64, workloads._ROW_BYTES[layout], workloads._NOPE[layout]
    rng = np.random.default_rng(8)
    sc = w.kv_cache[:, ps * rb:ps * (rb + 16)].reshape(-1, ps, 16)
    sc[..., :nope // 32] = rng.integers(20, 141, sc[..., :nope // 32].shape)
    # one magnitude per column group, so that small ones are not lost beside large ones
    sc[..., :nope // 32] = np.clip(np.arange(nope // 32) * 8 + 20 + sc[..., :nope // 32] % 4, 20, 140)
    w.kv_cache[:, ps * rb:ps * (rb + 16)] = sc.reshape(-1, ps * 16)
    q = bf16_f64(w.q)
    q[..., :nope] = 0
    w.q[:] = _bits(q)
    _, out, lse = _run(w)
    assert_decode(out, lse, decode(w, w.kv_cache, dense_slots(w)), "wide scales")


@pytest.mark.parametrize("layout", FP4)
def test_decode_of_a_nan_group(layout):
    """A NaN group reaches the heads that see its row, and no other request."""
    w = workloads.generate(workloads.dsv4(batch=2, seqlens=(100, 100), len_dist="fixed", heads=64, layout=layout,
                                          new_rows=False))
    w.kv_cache[w.block_table[0, 0], 64 * workloads._ROW_BYTES[layout] + 5] = 255
    d = DeviceWorkload(w)
    d.make_plan()
    d.decode()
    torch.cuda.synchronize()
    assert d.out[0].isnan().all() and d.lse[0].isnan().all()
    assert torch.isfinite(d.out[1].float()).all() and torch.isfinite(d.lse[1]).all()


@pytest.mark.parametrize("layout", FP4)
def test_decode_reports_a_bad_page(layout):
    """A block-table entry outside the cache is reported, its rows left out; the other request is whole."""
    w = workloads.generate(workloads.dsv4(batch=2, seqlens=(200, 130), len_dist="fixed", heads=64, layout=layout,
                                          new_rows=False))
    good = w.block_table.copy()
    w.block_table[0, 1] = w.kv_cache.shape[0] + 7
    d = DeviceWorkload(w)
    d.make_plan()
    d.decode()
    with pytest.raises(mla.MlaError) as e:
        mla.mla_read_status(d.ws)
    assert e.value.code == -5
    w.block_table[:] = good

    def rows(t):
        s = dense_slots(w)(t)
        return s[(np.arange(s.size) < 64) | (np.arange(s.size) >= 128)] if t == 0 else s

    assert_decode(bf16_to_f64(d.out), d.lse.cpu().numpy().astype(np.float64), decode(w, w.kv_cache, rows), "bad page")


@pytest.mark.parametrize("layout", FP4)
def test_decode_static_workspace(layout):
    w = workloads.generate(workloads.dsv4(batch=3, seqlens=(900, 1, 400), len_dist="fixed", heads=64, layout=layout,
                                          new_rows=False))
    d, out, lse = _run(w, num_sms=8)
    o2, l2, st = torch.empty_like(d.out), torch.empty_like(d.lse), _status()
    mla.mla_decode_static_workspace(d.q, d.kv, layout, 64, d.bt, d.sl, 1, w.cfg.sm_scale, d.sched, d.ns,
                                    d.plan.num_partitions, d.plan.total_splits, o2, l2, sink=d.sink, status_out=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(o2, d.out) and torch.equal(l2, d.lse)


@pytest.mark.parametrize("layout", FP4)
def test_decode_is_repeatable_and_captured(layout):
    """Two eager calls and two replays of a captured call give the same bits; the captured call reads what
    the cache and the queries hold at its replay; rows behind the outputs stay as they were."""
    w = workloads.generate(workloads.dsv4(batch=5, seqlens=(1, 64, 700, 2000, 90), len_dist="fixed", heads=128,
                                          layout=layout, new_rows=False))
    d = DeviceWorkload(w)
    T, N = w.q.shape[:2]
    back_o = torch.full((T + 2, N, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    back_l = torch.full((T + 2, N), 7.0, device="cuda")
    d.out, d.lse = back_o[:T], back_l[:T]
    d.make_plan(min_splits=2)
    d.decode()
    first = back_o.clone(), back_l.clone()
    d.decode()
    assert torch.equal(back_o, first[0]) and torch.equal(back_l, first[1])
    assert bool((back_o[T:] == 7).all()) and bool((back_l[T:] == 7).all())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        d.decode()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.decode()
    back_o.fill_(7)
    back_l.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(back_o, first[0]) and torch.equal(back_l, first[1])
    w.q[:] = w.q[::-1].copy()
    d.q.copy_(bf16_tensor(w.q))
    g.replay()
    assert mla.mla_read_status(d.ws) == 0
    assert_decode(bf16_to_f64(d.out), d.lse.cpu().numpy().astype(np.float64), decode(w, w.kv_cache, dense_slots(w)),
                  "replayed on other queries")


def test_two_decodes_on_two_streams():
    """Calls with workspaces of their own may run at the same time."""
    ws = [workloads.generate(workloads.dsv4(batch=4, seqlens=(900, 300, 64, 1), len_dist="fixed", heads=64, layout=la,
                                            new_rows=False, seed=la)) for la in FP4]
    ds = [DeviceWorkload(w) for w in ws]
    for d in ds:
        d.make_plan(num_sms=40)
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(3):
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                d.decode()
    torch.cuda.synchronize()
    for d, w in zip(ds, ws):
        assert mla.mla_read_status(d.ws) == 0
        assert_decode(bf16_to_f64(d.out), d.lse.cpu().numpy().astype(np.float64), decode(w, w.kv_cache, dense_slots(w)),
                      f"layout {w.cfg.layout}")


@pytest.mark.parametrize("layout", FP4)
def test_pages_past_32_bits(layout):
    """Rows whose byte offsets are past 2^31 and 2^32: written, read back and decoded at the end of a 4.6 GB cache."""
    ps, heads, L = 64, 64, 190
    pb = mla.mla_page_bytes(layout, ps)
    pages = 4_600_000_000 // pb
    kv = torch.zeros(pages, pb, dtype=torch.uint8, device="cuda")
    width = workloads._DQK[layout]
    rng = np.random.default_rng(180 + layout)
    at = np.array([pages - 1, 2_200_000_000 // pb, pages - 5], np.int32)
    slots = (at[np.arange(L) // ps].astype(np.int64) * ps + np.arange(L) % ps).astype(np.int32)
    bits = _bits(rng.standard_normal((L, width)))
    mla.mla_kv_write(bf16_tensor(bits), _cuda(slots), kv, layout, ps)
    rows = torch.empty(L, width, dtype=torch.bfloat16, device="cuda")
    mla.mla_kv_read(kv, layout, ps, _cuda(slots), rows)
    small = oracle.kv_write(bits, np.arange(L, dtype=np.int32), np.zeros((3, pb), np.uint8), layout, ps)
    k = rows_of(small, layout, ps, np.arange(L))
    assert np.array_equal(bf16_to_f64(rows), k)
    q = _bits(rng.standard_normal((1, heads, width)))
    plan = mla.mla_decode_plan([L], 1, heads)
    ws = mla.alloc_workspace(plan.workspace_bytes)
    out = torch.empty(1, heads, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, heads, device="cuda")
    mla.mla_decode(bf16_tensor(q), kv, layout, ps, _cuda(at[None]), _cuda(np.array([L], np.int32)), 1, 0.05,
                   _cuda(plan.sched), _cuda(plan.num_splits), plan.num_partitions, plan.total_splits, ws, out, lse)
    assert mla.mla_read_status(ws) == 0
    ref = attend(bf16_f64(q[0]), k, float(np.float32(0.05)))
    assert_decode(bf16_to_f64(out), lse.cpu().numpy().astype(np.float64), (ref[0][None], ref[1][None], ref[2][None], ref[3]),
                  "far pages")


@pytest.mark.parametrize("layout", FP4)
def test_timed_out_wait_is_reported(layout):
    """The withheld signal (mla_decode's test flag) ends the call with MLA_STATUS_WAIT_TIMEOUT, and the next
    call is whole."""
    w = workloads.generate(workloads.dsv4(batch=3, seqlens=(64, 700, 1300), len_dist="fixed", heads=64, layout=layout,
                                          new_rows=False))
    d = DeviceWorkload(w)
    p = d.make_plan()
    mla.mla_decode(d.q, d.kv, layout, 64, d.bt, d.sl, 1, w.cfg.sm_scale, d.sched, d.ns, p.num_partitions, p.total_splits,
                   d.ws, d.out, d.lse, sink=d.sink, _test_withhold_signal=True)
    with pytest.raises(mla.MlaError):
        mla.mla_read_status(d.ws)
    out, lse = d.run(write=False)
    assert_decode(out, lse, decode(w, w.kv_cache, dense_slots(w)), "after a timed-out call")


# ----------------------------------------------------------------------------- 128 query rows a request: CTA pairs
@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("sq,heads,splits", [(1, 128, 1), (1, 256, 3), (3, 128, 1), (2, 192, 2)])
def test_pairs_and_single_sms_agree(layout, sq, heads, splits):
    """Query rows in groups of 128, on CTA pairs and, by the flag, on single SMs."""
    w = workloads.generate(workloads.verify(batch=3, sq=sq, heads=heads, seqlens=(1, 700, 66), len_dist="fixed",
                                            layout=layout, new_rows=False, tail_fill="nan"))
    d = DeviceWorkload(w)
    p = d.make_plan(min_splits=splits)
    ref = decode(w, w.kv_cache, dense_slots(w))
    for single in (False, True):
        d.out.fill_(7)
        mla.mla_decode(d.q, d.kv, layout, 64, d.bt, d.sl, sq, w.cfg.sm_scale, d.sched, d.ns, p.num_partitions,
                       p.total_splits, d.ws, d.out, d.lse, sink=d.sink, causal=True, single_sm=single)
        assert mla.mla_read_status(d.ws) == 0
        assert_decode(bf16_to_f64(d.out), d.lse.cpu().numpy().astype(np.float64), ref, f"single_sm {single}")


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("topk,heads,sq", [(300, 256, 1), (65, 128, 3)])
def test_pairs_listed_rows(layout, topk, heads, sq):
    """Several groups of 128 query rows over one token's list, and several tokens with lists of their own."""
    w = workloads.generate(workloads.sparse(batch=2, sq=sq, heads=heads, seqlens=(1000, 90), layout=layout, topk=topk,
                                            page_size=16, new_rows=False))
    w.indices[0, ::7] = -1
    w.indices[-1] = -1
    w.indices[-1, topk - 1] = 3                   # a single row, listed last
    _, out, lse = _run(w)
    assert_decode(out, lse, decode(w, w.kv_cache, listed_slots(w)), f"top {topk}")


@pytest.mark.parametrize("layout", FP4)
def test_pairs_wide_scales(layout):
    """Scale bytes from 20 to 140 in one cache, one magnitude per column group (as for single SMs above)."""
    w = workloads.generate(workloads.dsv3(batch=2, seqlens=(300, 77), len_dist="fixed", heads=128, layout=layout,
                                          new_rows=False, seed=9))
    ps, rb, nope = 64, workloads._ROW_BYTES[layout], workloads._NOPE[layout]
    sc = w.kv_cache[:, ps * rb:ps * (rb + 16)].reshape(-1, ps, 16)
    sc[..., :nope // 32] = np.clip(np.arange(nope // 32) * 8 + 20 + np.arange(ps)[:, None] % 4, 20, 140)
    w.kv_cache[:, ps * rb:ps * (rb + 16)] = sc.reshape(-1, ps * 16)
    q = bf16_f64(w.q)
    q[..., :nope] = 0
    w.q[:] = _bits(q)
    _, out, lse = _run(w)
    assert_decode(out, lse, decode(w, w.kv_cache, dense_slots(w)), "wide scales")


@pytest.mark.parametrize("layout", FP4)
def test_pairs_nan_group_and_bad_page(layout):
    """A NaN group reaches its own request only; a bad page's rows are left out and reported; and a timed-out wait
    ends the call, after which the next is whole."""
    w = workloads.generate(workloads.dsv4(batch=3, seqlens=(200, 100, 400), len_dist="fixed", heads=128, layout=layout,
                                          new_rows=False))
    held = w.kv_cache.copy()
    w.kv_cache[w.block_table[1, 0], 64 * workloads._ROW_BYTES[layout] + 5] = 255
    good = w.block_table.copy()
    w.block_table[0, 1] = w.kv_cache.shape[0] + 7
    d = DeviceWorkload(w)
    p = d.make_plan()
    d.decode()
    with pytest.raises(mla.MlaError) as e:
        mla.mla_read_status(d.ws)
    assert e.value.code == -5
    assert d.out[1].isnan().all() and d.lse[1].isnan().all()
    w.block_table[:] = good
    w.kv_cache[:] = held

    def rows(t):
        s = dense_slots(w)(t)
        return s[(np.arange(s.size) < 64) | (np.arange(s.size) >= 128)] if t == 0 else s

    out, lse = bf16_to_f64(d.out), d.lse.cpu().numpy().astype(np.float64)
    ref = decode(w, held, rows)
    keep = [0, 2]
    assert_decode(out[keep], lse[keep], tuple(x[keep] if isinstance(x, np.ndarray) and x.ndim else x for x in ref),
                  "the other requests")
    d = DeviceWorkload(w)
    p = d.make_plan()
    mla.mla_decode(d.q, d.kv, layout, 64, d.bt, d.sl, 1, w.cfg.sm_scale, d.sched, d.ns, p.num_partitions, p.total_splits,
                   d.ws, d.out, d.lse, sink=d.sink, _test_withhold_signal=True)
    with pytest.raises(mla.MlaError):
        mla.mla_read_status(d.ws)
    out, lse = d.run(write=False)
    assert_decode(out, lse, decode(w, w.kv_cache, dense_slots(w)), "after a timed-out call")


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("ps,heads,splits", [(8, 128, 2), (1024, 128, 1), (4096, 64, 3), (32, 384, 1), (64, 4096, 1)])
def test_decode_page_sizes_and_head_counts(layout, ps, heads, splits):
    """Pages smaller and much larger than a tile, many groups of query rows, and requests that share pages."""
    w = workloads.generate(workloads.dsv4(batch=3, seqlens=(3000, 777, 3000) if heads < 4096 else (130, 1, 70),
                                          len_dist="fixed", heads=heads, layout=layout, page_size=ps, new_rows=False,
                                          tail_fill="nan", seed=ps))
    w.block_table[2] = w.block_table[0]
    _, out, lse = _run(w, min_splits=splits)
    assert_decode(out, lse, decode(w, w.kv_cache, dense_slots(w)), f"pages of {ps}, {heads} heads")


@pytest.mark.parametrize("layout,heads", [(3, 64), (4, 128)])
def test_step_captured_on_a_side_stream(layout, heads):
    """A decode step captured once (queries and rows prepared, the decode, the rows read back) on a stream of its own,
    replayed with other queries, rows, positions and slots; the second replay finds the first one's rows."""
    rng = np.random.default_rng(210 + layout)
    ps, B, max_pos = 16, 4, 300
    width = workloads._DQK[layout]
    table = rng.permutation(64)[:B * 16].reshape(B, 16).astype(np.int32)
    ctx = np.array([0, 17, 120, 47])
    slot_of = lambda b, j: table[b, j // ps].astype(np.int64) * ps + j % ps  # noqa: E731
    held = np.zeros((64, workloads.page_bytes(layout, ps)), np.uint8)
    for b in range(B):
        j = np.arange(ctx[b])
        held = oracle.kv_write(_bits(rng.standard_normal((ctx[b], width))), slot_of(b, j).astype(np.int32), held, layout, ps)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        kv, freqs, gain = _cuda(held), _cuda(_table(max_pos)), torch.ones(512, dtype=torch.bfloat16, device="cuda")
        q = torch.zeros(B, heads, width, dtype=torch.bfloat16, device="cuda")
        prepared, raw = torch.empty_like(q), torch.zeros(B, width, dtype=torch.bfloat16, device="cuda")
        slots, pos, lens = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
        bt, st = _cuda(table), _status()
        plan = mla.mla_decode_plan(ctx + 3, 1, heads)  # each request has as many 64-row blocks in every step
        ws, sched, ns = mla.alloc_workspace(plan.workspace_bytes), _cuda(plan.sched), _cuda(plan.num_splits)
        out = torch.empty(B, heads, 512, dtype=torch.bfloat16, device="cuda")
        lse, back = torch.empty(B, heads, device="cuda"), torch.empty_like(raw)

        def step():
            mla.mla_qkv_norm_rope(q[..., :width - 64], q[..., width - 64:], raw, slots, pos, gain, 1e-6, freqs, prepared,
                                  kv, layout, ps, q_eps=1e-6, status=st)
            mla.mla_decode(prepared, kv, layout, ps, bt, lens, 1, 0.07, sched, ns, plan.num_partitions, plan.total_splits,
                           ws, out, lse)
            mla.mla_kv_read(kv, layout, ps, slots, back, status=st)

        def fill(ctx):
            q.copy_(bf16_tensor(_bits(rng.standard_normal((B, heads, width)))))
            raw.copy_(bf16_tensor(_bits(rng.standard_normal((B, width)))))
            slots.copy_(_cuda(np.array([slot_of(b, ctx[b]) for b in range(B)]).astype(np.int32)))
            pos.copy_(_cuda(ctx.astype(np.int32)))
            lens.copy_(_cuda((ctx + 1).astype(np.int32)))

        fill(ctx)
        step()                                        # the first step, eager
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        step()
    for _ in range(2):
        ctx = ctx + 1
        with torch.cuda.stream(stream):
            fill(ctx)
            g.replay()
        stream.synchronize()
        assert int(st.item()) == 0
        bytes_now, q64 = kv.cpu().numpy(), bf16_f64(_bits_of(prepared))
        got, glse = bf16_to_f64(out), lse.cpu().numpy().astype(np.float64)
        for b in range(B):
            k = rows_of(bytes_now, layout, ps, slot_of(b, np.arange(ctx[b] + 1)))
            assert_decode(got[b], glse[b], attend(q64[b], k, float(np.float32(0.07))), f"request {b}")
            assert np.array_equal(bf16_to_f64(back[b]), k[-1])
            assert k[-1].any()


# ----------------------------------------------------------------------------- a step as a whole
@pytest.mark.parametrize("layout,heads,sq", [(3, 64, 1), (4, 128, 1), (4, 64, 3)])
def test_serving_steps(layout, heads, sq):
    """Three decode steps as a program runs them: the step's queries prepared and its rows appended, then the
    decode over the cache that now holds them, then the cached rows read back for a bf16 consumer. Every
    step is checked against plain attention over the rows as the oracle writes them."""
    rng = np.random.default_rng(190 + layout + sq)
    ps, B, max_pos, eps = 16, 3, 600, 1e-6
    width = workloads._DQK[layout]
    ctx = np.array([5, 130, 47])
    pages = 64
    table = rng.permutation(pages)[:B * 20].reshape(B, 20).astype(np.int32)
    kv_ref = np.zeros((pages, workloads.page_bytes(layout, ps)), np.uint8)
    slot_of = lambda b, j: table[b, j // ps].astype(np.int64) * ps + j % ps  # noqa: E731
    for b in range(B):  # the prompts' rows
        j = np.arange(ctx[b])
        kv_ref = oracle.kv_write(_bits(rng.standard_normal((ctx[b], width))), slot_of(b, j).astype(np.int32), kv_ref,
                                 layout, ps)
    kv = _cuda(kv_ref)
    kw, freqs = _bits(1 + 0.1 * rng.standard_normal(512)), _table(max_pos)
    scale, sink = 0.06, rng.standard_normal(heads).astype(np.float32)
    for _ in range(3):
        T = B * sq
        pos = (ctx[:, None] + np.arange(sq)).reshape(-1).astype(np.int32)
        req = np.repeat(np.arange(B), sq)
        slots = np.array([slot_of(b, j) for b, j in zip(req, pos)]).astype(np.int32)
        raw, qraw = _bits(rng.standard_normal((T, width))), _bits(rng.standard_normal((T, heads, width)))
        q = bf16_tensor(qraw)
        ctx = ctx + sq
        mla.mla_qkv_norm_rope(q[..., :width - 64], q[..., width - 64:], bf16_tensor(raw), _cuda(slots), _cuda(pos),
                              bf16_tensor(kw), eps, _cuda(freqs), q, kv, layout, ps, q_eps=eps)
        plan = mla.mla_decode_plan(ctx, sq, heads)
        ws = mla.alloc_workspace(plan.workspace_bytes)
        out = torch.empty(T, heads, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(T, heads, device="cuda")
        mla.mla_decode(q, kv, layout, ps, _cuda(table), _cuda(ctx.astype(np.int32)), sq, scale, _cuda(plan.sched),
                       _cuda(plan.num_splits), plan.num_partitions, plan.total_splits, ws, out, lse, sink=_cuda(sink),
                       causal=sq > 1)
        assert mla.mla_read_status(ws) == 0
        # the rows as the GPU holds them (fp32 against fp64 norms may differ by a code): all but a few bytes agree
        kv_ref = oracle.kv_write_norm_rope(raw, slots, pos, kw, eps, freqs, kv_ref, layout, ps)
        held = kv.cpu().numpy()
        assert np.mean(held != kv_ref) <= 2e-3
        q64 = bf16_f64(_bits_of(q))
        got, glse = bf16_to_f64(out), lse.cpu().numpy().astype(np.float64)
        for t in range(T):
            k = rows_of(held, layout, ps, slot_of(req[t], np.arange(pos[t] + 1)))
            ref = attend(q64[t], k, float(np.float32(scale)), sink.astype(np.float64))
            assert_decode(got[t], glse[t], ref, f"token {t}")
        back = torch.empty(T, width, dtype=torch.bfloat16, device="cuda")
        mla.mla_kv_read(kv, layout, ps, _cuda(slots), back)
        assert np.array_equal(bf16_to_f64(back), rows_of(held, layout, ps, slots))


def test_sparse_prefill_over_a_quantised_cache():
    """Rows of a 4-bit cache read back as one bf16 run, which mla_sparse_prefill attends over."""
    rng = np.random.default_rng(200)
    layout, ps, n, T, N, topk = 4, 64, 300, 6, 32, 50
    kv = torch.zeros(6, mla.mla_page_bytes(layout, ps), dtype=torch.uint8, device="cuda")
    slots = rng.permutation(6 * ps)[:n].astype(np.int32)
    mla.mla_kv_write(bf16_tensor(_bits(rng.standard_normal((n, 576)))), _cuda(slots), kv, layout, ps)
    run = torch.empty(n, 576, dtype=torch.bfloat16, device="cuda")
    mla.mla_kv_read(kv, layout, ps, _cuda(slots), run)
    idx = np.stack([rng.permutation(n)[:topk] for _ in range(T)]).astype(np.int32)
    idx[1, 5:] = -1
    q = _bits(rng.standard_normal((T, N, 576)))
    plan = mla.mla_decode_plan(np.full(T, n), 1, N, topk)
    ws = mla.alloc_workspace(plan.workspace_bytes)
    out = torch.empty(T, N, 512, dtype=torch.bfloat16, device="cuda")
    lse, mx = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda")
    mla.mla_sparse_prefill(bf16_tensor(q), run, _cuda(idx), 0.05, _cuda(plan.sched), _cuda(plan.num_splits),
                           plan.num_partitions, plan.total_splits, ws, out, mx, lse)
    assert mla.mla_read_status(ws) == 0
    held = rows_of(kv.cpu().numpy(), layout, ps, slots)
    for t in range(T):
        ref = attend(bf16_f64(q[t]), held[idx[t][idx[t] >= 0]], float(np.float32(0.05)))
        assert_decode(bf16_to_f64(out)[t], lse[t].cpu().numpy().astype(np.float64), ref, f"token {t}")


@pytest.mark.parametrize("rows,splits", [(16, 5), (16, 16), (20, 33), (128, 77), (96, 2), (400, 21)])
def test_combine_of_many_splits(rows, splits):
    """Partials merged in 64 bits: few rows and many, counts of splits on both sides of a group of loads and of a
    warp, empty partials among them (their values not numbers), a row with nothing, a request left alone."""
    rng = np.random.default_rng(rows + splits)
    B = 2
    ns = np.array([0, splits, splits + 1], np.int32)      # the second request is not split: left as it was
    po = rng.standard_normal((splits + 1, rows, 512)).astype(np.float32)
    pl = (3 * rng.standard_normal((splits + 1, rows))).astype(np.float32)
    empty = rng.random((splits + 1, rows)) < 0.2
    empty[:, 3] = True
    pl[empty], po[empty] = -np.inf, np.nan
    sink = rng.standard_normal(rows).astype(np.float32)
    out = torch.full((B * rows, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B * rows,), 7.0, device="cuda")
    mla.mla_combine(_cuda(po), _cuda(pl), _cuda(ns), rows, rows, out, lse, sink=_cuda(sink))
    torch.cuda.synchronize()
    assert bool((out[rows:] == 7).all()) and bool((lse[rows:] == 7).all())
    got, glse = bf16_to_f64(out)[:rows], lse.cpu().numpy().astype(np.float64)[:rows]
    for r in range(rows):
        on = ~empty[:splits, r]
        if not on.any():
            assert np.isneginf(glse[r]) and np.all(got[r] == 0)
            continue
        l, o = pl[:splits, r][on].astype(np.float64), po[:splits, r][on].astype(np.float64)
        ref_lse = np.log(np.exp(l).sum())
        w = np.exp(l - ref_lse) / (1 + np.exp(float(sink[r]) - ref_lse))
        # fp32 weights: the exponentials and the logarithm (2 units each), their arguments (|lse| below 16: 2^-20)
        # and the sums of up to 77 terms (77 * 2^-24 of their magnitudes); then one rounding to bf16
        mean = w @ np.abs(o)
        assert abs(glse[r] - ref_lse) <= 2.0 ** -19
        assert np.all(np.abs(got[r] - w @ o) <= (2.0 ** -17) * mean + 2.0 ** -8 * np.abs(w @ o))
