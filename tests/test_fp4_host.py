"""4-bit rows without a GPU: the oracle's codec, layouts and write against plain numpy forms, and
the refusals of the entry points that take them (made before any device work)."""
import ctypes

import numpy as np
import pytest
import torch

import mla_paged_latent_gb300 as mla
import oracle
import workloads
from fp4_helpers import E2M1, attend, bf16_f64, decode, dense_slots, listed_slots, rows_of
from mla_paged_latent_gb300 import build as mla_build

FP4 = [mla.MLA_KV_FP4_448_UE8M0, mla.MLA_KV_FP4_512_UE8M0]


@pytest.fixture(scope="module")
def lib():
    mla_build.build()
    return mla.load()


def _bf16_bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(
        np.uint16).copy()


def test_e2m1_codec():
    assert np.array_equal(oracle.e2m1_decode(np.arange(16)), E2M1)
    assert np.array_equal(np.signbit(oracle.e2m1_decode([0, 8])), [False, True])
    # every value between two grid points goes to the nearer one, a tie to the even code
    for c in range(7):
        lo, hi = E2M1[c], E2M1[c + 1]
        mid = (lo + hi) / 2
        assert oracle.e2m1_encode(mid) == (c if c % 2 == 0 else c + 1)
        assert oracle.e2m1_encode(np.nextafter(mid, 0)) == c and oracle.e2m1_encode(np.nextafter(mid, 9)) == c + 1
        assert oracle.e2m1_encode(-np.nextafter(mid, 9)) == c + 9
    assert oracle.e2m1_encode([6.0, 7.5, 1e30, np.inf, -np.inf, -0.0]).tolist() == [7, 7, 7, 7, 15, 8]


def test_group_exponent():
    for e in (-40, -3, 0, 5, 120):
        assert oracle.group_exponent_fp4(6.0 * 2.0 ** e) == e
        assert oracle.group_exponent_fp4(np.nextafter(6.0 * 2.0 ** e, np.inf)) == e + 1
        assert oracle.group_exponent_fp4(4.0 * 2.0 ** e) == e
        assert oracle.group_exponent_fp4(np.nextafter(3.0 * 2.0 ** e, np.inf)) == e
    assert oracle.group_exponent_fp4(np.inf) == 127


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("ps", [1, 2, 8, 64])
def test_page_bytes(lib, layout, ps):
    row, nope = ((352, 448), (384, 512))[layout - 3]
    want = -(-ps * (row + 16) // row) * row
    info = oracle.layout_info(layout, ps)
    assert mla.mla_page_bytes(layout, ps) == want == info["page_bytes"] == workloads.page_bytes(layout, ps)
    assert info["row_bytes"] == row and info["nope"] == nope and info["n_scales"] == nope // 32
    assert mla.DQK[layout] == mla.ROW_ELEMS[layout] == info["dqk"] == nope + 64


@pytest.mark.parametrize("layout", FP4)
def test_oracle_write_and_read(layout):
    """The written bytes decode to the nearest value of each group's grid; the smallest exponent that
    keeps the group's largest element inside it is taken; bytes of other rows stay."""
    rng = np.random.default_rng(layout)
    ps, pages, n = 8, 5, 30
    nope, width = workloads._NOPE[layout], workloads._DQK[layout]
    kv0 = rng.integers(0, 256, (pages, workloads.page_bytes(layout, ps)), dtype=np.uint8)
    x = rng.standard_normal((n, width)) * 2.0 ** rng.integers(-20, 20, (n, 1))
    x[0] = 0
    x[1, :32] = 1e-20
    bits = _bf16_bits(x)
    bits[2, 5] = 0x7FC0   # NaN: its group reads back as NaN
    bits[3, 40] = 0xFF80  # -inf: scale byte 254, stored as -6
    slots = rng.permutation(pages * ps)[:n].astype(np.int32)
    slots[4] = -1
    kv = oracle.kv_write(bits, slots, kv0, layout, ps)
    keep = slots >= 0
    v = bf16_f64(bits)
    got = rows_of(kv, layout, ps, slots[keep])
    one = np.stack([oracle.decode_row(kv, layout, ps, s // ps, s % ps) for s in slots[keep]])
    assert np.array_equal(got, one, equal_nan=True)
    for r, row in zip(np.flatnonzero(keep), got):
        assert np.array_equal(row[nope:], v[r, nope:])
        for g in range(nope // 32):
            a, b = v[r, 32 * g:32 * g + 32], row[32 * g:32 * g + 32]
            if np.isnan(a).any():
                assert np.isnan(b).all()
                continue
            if np.isinf(a).any():
                assert b[8] == -6 * 2.0 ** 127 and r == 3 and g == 1
                continue
            e = oracle.group_exponent_fp4(max(np.abs(a).max(), float(np.float32(1e-10))))
            grid = E2M1[:8] * 2.0 ** e
            assert grid[7] >= np.abs(a).max()
            assert np.all(np.abs(np.abs(b) - np.abs(a)) == np.abs(np.abs(a)[:, None] - grid).min(1))
    untouched = np.setdiff1d(np.arange(pages * ps), slots[keep])
    rb = workloads._ROW_BYTES[layout]
    for s in untouched:
        p, o = divmod(int(s), ps)
        assert np.array_equal(kv[p, o * rb:(o + 1) * rb], kv0[p, o * rb:(o + 1) * rb])


@pytest.mark.parametrize("layout", FP4)
def test_oracle_decode_is_plain_attention(layout):
    """The oracle's paged decode over 4-bit rows against a plain float64 softmax over rows decoded in numpy."""
    w = workloads.generate(workloads.verify(batch=2, seqlens=(3, 70), len_dist="fixed", heads=4, layout=layout,
                                            page_size=16, new_rows=False))
    ref = decode(w, w.kv_cache, dense_slots(w), w.cfg.sm_scale)
    out, lse = oracle.mla_decode(w.q, w.kv_cache, layout, 16, w.block_table, w.seqlens, 4, w.cfg.sm_scale, causal=True)
    assert np.allclose(out, ref[0], rtol=1e-9, atol=1e-11)
    assert np.array_equal(np.isneginf(lse), np.isneginf(ref[1]))
    fin = ~np.isneginf(lse)
    assert np.allclose(lse[fin], ref[1][fin], rtol=1e-10)
    w = workloads.generate(workloads.sparse(batch=2, seqlens=(90, 40), heads=3, layout=layout, topk=33, page_size=8,
                                            new_rows=False))
    ref = decode(w, w.kv_cache, listed_slots(w), w.cfg.sm_scale)
    out, lse = oracle.mla_decode(w.q, w.kv_cache, layout, 8, w.block_table, w.seqlens, 1, w.cfg.sm_scale,
                                 indices=w.indices)
    assert np.allclose(out, ref[0], rtol=1e-9, atol=1e-11) and np.allclose(lse, ref[1], rtol=1e-10)


def test_plain_attention_of_equal_keys():
    k = np.ones((5, 576))
    k[:, :512] *= np.arange(5)[:, None] * 0  # equal keys: the mean of V, lse = s + ln n
    out, lse, _, _ = attend(np.ones((1, 576)), k, 0.5)
    assert np.allclose(out, 0) and np.allclose(lse, 32 + np.log(5))


@pytest.mark.parametrize("width", [512, 576])
@pytest.mark.parametrize("norm", [False, True])
def test_oracle_q_norm_rope(width, norm):
    """Against complex multiplication of the pairs and a plain RMSNorm; rows outside the table keep their bits."""
    rng = np.random.default_rng(width + norm)
    n, max_pos, eps = 20, 50, 1e-5
    bits = _bf16_bits(rng.standard_normal((n, width)))
    w = _bf16_bits(1 + 0.3 * rng.standard_normal(512))
    theta = np.outer(np.arange(max_pos), 10000.0 ** (-np.arange(32) / 32.0))
    f = np.zeros((max_pos, 64), np.float32)
    f[:, 0::2], f[:, 1::2] = np.cos(theta), np.sin(theta)
    pos = rng.integers(0, max_pos, n).astype(np.int32)
    pos[3], pos[4] = -1, max_pos
    before = rng.integers(0, 1 << 16, bits.shape, dtype=np.uint16)
    got = oracle.q_norm_rope(bits, pos, f, eps=eps if norm else None, weight_bits=w if norm else None, out=before)
    assert np.array_equal(got[3:5], before[3:5])
    ok = (pos >= 0) & (pos < max_pos)
    x = bf16_f64(bits)[ok]
    if norm:
        x[:, :512] *= bf16_f64(w) / np.sqrt((x[:, :512] ** 2).mean(1, keepdims=True) + float(np.float32(eps)))
    z = (x[:, -64::2] + 1j * x[:, -63::2]) * (f[pos[ok], 0::2].astype(np.float64) + 1j * f[pos[ok], 1::2])
    x[:, -64::2], x[:, -63::2] = z.real, z.imag
    assert np.all(np.abs(bf16_f64(got[ok]) - x) <= np.abs(x) * 2.0 ** -8 + 1e-30)


# ----------------------------------------------------------------------------- refusals
FAKE = ctypes.c_void_p(0x100000)
ODD = ctypes.c_void_p(0x100008)


def test_kv_read_refuses(lib):
    def rc(kv=FAKE, layout=4, pages=4, ps=64, slots=FAKE, n=3, rows=FAKE):
        return lib.mla_kv_read(kv, layout, pages, ps, slots, n, rows, None, None)

    assert rc(n=0, kv=None, slots=None, rows=None) == 0
    assert rc(n=-1) == -1
    assert rc(kv=None) == -1 and rc(slots=None) == -1 and rc(rows=None) == -1
    assert rc(layout=5) == -1 and rc(layout=-1) == -1
    assert rc(ps=48) == -1 and rc(pages=0) == -1
    assert rc(rows=ODD) == -1 and rc(kv=ODD) == -1
    assert b"aligned" in lib.mla_last_error()


def test_qkv_norm_rope_refuses(lib):
    # T = 3, N = 2 rows of 576: addresses far apart unless a case moves them together
    at = lambda k: ctypes.c_void_p(0x1000000 * k)  # noqa: E731

    def rc(**kw):
        a = dict(qn=at(1), qnt=1024, qnh=512, qp=at(2), qpt=128, qph=64, norm=0, qw=None, qeps=1e-6, kv_raw=at(3),
                 kvs=576, slots=at(4), pos=at(5), kw=at(6), keps=1e-6, freqs=at(7), max_pos=100, T=3, N=2, out=at(8),
                 kv=at(9), layout=4, pages=4, ps=64)
        a.update(kw)
        return lib.mla_qkv_norm_rope(a["qn"], a["qnt"], a["qnh"], a["qp"], a["qpt"], a["qph"], a["norm"], a["qw"],
                                     a["qeps"], a["kv_raw"], a["kvs"], a["slots"], a["pos"], a["kw"], a["keps"],
                                     a["freqs"], a["max_pos"], a["T"], a["N"], a["out"], a["kv"], a["layout"],
                                     a["pages"], a["ps"], None, None)

    assert rc(T=0, qn=None, kv=None) == 0
    assert rc(T=-1) == -1
    for name in ("qn", "qp", "kv_raw", "slots", "pos", "kw", "freqs", "out", "kv"):
        assert rc(**{name: None}) == -1, name
    for name in ("qn", "qp", "kv_raw", "kw", "freqs", "out", "kv"):
        assert rc(**{name: ODD}) == -1, name
    for name in ("qnt", "qnh", "qpt", "qph", "kvs"):
        assert rc(**{name: 12}) == -1 and rc(**{name: -8}) == -1, name
    assert rc(layout=9) == -1 and rc(ps=12) == -1 and rc(pages=0) == -1 and rc(max_pos=0) == -1 and rc(N=0) == -1
    assert rc(keps=-1.0) == -1 and rc(keps=float("nan")) == -1 and rc(norm=1, qeps=float("inf")) == -1
    assert rc(norm=0, qw=at(10)) == -1            # a gain without the norm
    assert rc(T=1 << 30, N=8) == -2               # row count past 31 bits
    # q_out over an input, other than row for row
    base = 0x1000000
    assert rc(out=at(1)) == -1 and b"overlaps" in lib.mla_last_error()
    assert rc(qn=at(8), qnt=1152, qnh=576, qp=ctypes.c_void_p(8 * base + 1024), qpt=1152, qph=512) == -1
    assert rc(out=at(3)) == -1
    assert rc(out=ctypes.c_void_p(2 * base + 2 * 128 * 2 + 2 * 64)) == -1   # the last pe row's last bytes


def test_binding_refuses(monkeypatch):
    """Shapes, types and layouts are checked before the call (on tensors that claim to live on the GPU)."""
    monkeypatch.setattr(mla, "_require_cuda", lambda *t: None)
    monkeypatch.setattr(mla, "_stream", lambda s: None)
    called = []

    class Lib:
        mla_page_bytes = staticmethod(mla.load().mla_page_bytes)
        mla_qkv_norm_rope = staticmethod(lambda *a: called.append(a) or 0)
        mla_kv_read = staticmethod(lambda *a: called.append(a) or 0)
        mla_decode = staticmethod(lambda *a: called.append(a) or 0)

    monkeypatch.setattr(mla, "load", lambda path=None: Lib)
    T, N, L = 3, 2, 4
    bf, i32 = torch.bfloat16, torch.int32
    good = dict(q_nope=torch.zeros(T, N, 512, dtype=bf), q_pe=torch.zeros(T, N, 64, dtype=bf),
                kv_raw=torch.zeros(T, 576, dtype=bf), slots=torch.zeros(T, dtype=i32),
                positions=torch.zeros(T, dtype=i32), kv_norm_weight=torch.ones(512, dtype=bf), kv_eps=1e-6,
                freqs=torch.zeros(9, 64), q_out=torch.zeros(T, N, 576, dtype=bf),
                kv_cache=torch.zeros(2, mla.mla_page_bytes(L, 64), dtype=torch.uint8), layout=L, page_size=64)
    mla.mla_qkv_norm_rope(**good)
    assert len(called) == 1
    bad = dict(q_nope=[torch.zeros(T, N, 448, dtype=bf), torch.zeros(T, N, 512), torch.zeros(T, N, 1024, dtype=bf)[..., ::2]],
               q_pe=[torch.zeros(T, N + 1, 64, dtype=bf), torch.zeros(T, N, 32, dtype=bf)],
               kv_raw=[torch.zeros(T, 512, dtype=bf), torch.zeros(T, 576)],
               slots=[torch.zeros(T, dtype=torch.int64), torch.zeros(T - 1, dtype=i32), torch.zeros(2 * T, dtype=i32)[::2]],
               positions=[torch.zeros(T)], kv_norm_weight=[torch.ones(576, dtype=bf)],
               freqs=[torch.zeros(9, 32), torch.zeros(9, 64, dtype=torch.float64)],
               q_out=[torch.zeros(T, N, 512, dtype=bf), torch.zeros(N, T, 576, dtype=bf).transpose(0, 1)],
               kv_cache=[torch.zeros(2, 100, dtype=torch.uint8)], q_norm_weight=[torch.ones(512)],
               status=[torch.zeros(1, dtype=torch.int64)])
    for name, values in bad.items():
        for v in values:
            with pytest.raises(ValueError):
                mla.mla_qkv_norm_rope(**{**good, name: v})
    for rows in (torch.zeros(T, 512, dtype=bf), torch.zeros(T + 1, 576, dtype=bf), torch.zeros(T, 576)):
        with pytest.raises(ValueError):
            mla.mla_kv_read(good["kv_cache"], L, 64, good["slots"], rows)
    assert len(called) == 1


def test_decode_refuses_as_other_layouts(lib):
    """The 4-bit layouts go through the decode's own checks."""
    def rc(layout, ps=64, ws=1 << 30, heads=16, sq=1, topk=0, idx=None):
        return lib.mla_decode(FAKE, FAKE, layout, 4, ps, FAKE, 2, FAKE, 2, sq, heads, 0.1, None, idx, topk, 0, FAKE, FAKE,
                              1, 2, FAKE, ws, FAKE, FAKE, 0, None)

    for layout in FP4:
        assert rc(layout, ps=4) == -2 and rc(layout, ps=48) == -2
        assert rc(layout, ws=100) == -3
        assert rc(layout, sq=2, topk=8, idx=FAKE) == -2
        assert rc(layout, topk=8) == -1
    assert rc(5) == -1


def test_decode_refuses_what_a_4_bit_cache_cannot_be(lib):
    """Its alignment, its count of slots, its page size; a cache of another layout may be so."""
    def rc(layout, kv=FAKE, pages=4, ps=64):
        return lib.mla_decode(FAKE, kv, layout, pages, ps, FAKE, 2, FAKE, 2, 1, 128, 0.1, None, None, 0, 0, FAKE, FAKE,
                              1, 2, FAKE, 100, FAKE, FAKE, 0, None)   # (a workspace of 100 bytes: -3 when all else is right)

    for layout in FP4:
        assert rc(layout) == -3
        assert rc(layout, kv=ctypes.c_void_p(0x100010)) == -1 and b"32-byte" in lib.mla_last_error()
        assert rc(layout, pages=1 << 26) == -2 and b"2^32" in lib.mla_last_error()
        assert rc(layout, pages=(1 << 26) - 2) == -3
        assert rc(layout, ps=1 << 23) == -2 and rc(layout, ps=1 << 22) == -3
    assert rc(2, kv=ctypes.c_void_p(0x100010)) == -3 and rc(2, pages=1 << 26) == -3 and rc(2, ps=1 << 23) == -3


def test_overlaps_with_the_cache_are_refused(lib):
    """Rows that are read or written inside the cache, and strides that no memory holds."""
    at = lambda k, o=0: ctypes.c_void_p(0x1000000 * k + o)  # noqa: E731
    end = mla.mla_page_bytes(4, 64) * 4

    def qkv(qn=at(1), qnt=1024, qp=at(2), kv_raw=at(3), kvs=576, out=at(8), T=3):
        return lib.mla_qkv_norm_rope(qn, qnt, 512, qp, 128, 64, 0, None, 0.0, kv_raw, kvs, at(4), at(5), at(6), 1e-6, at(7),
                                     100, T, 2, out, at(9), 4, 4, 64, None, None)

    for name in ("qn", "qp", "kv_raw", "out"):
        assert qkv(**{name: at(9, end - 16)}) == -1 and b"kv_cache overlaps" in lib.mla_last_error(), name
    assert qkv(qn=at(9, -1024)) == -1
    for name in ("qnt", "kvs"):
        assert qkv(T=1 << 20, **{name: 1 << 39}) == -1 and b"past any memory" in lib.mla_last_error(), name
    assert lib.mla_kv_read(at(9), 4, 4, 64, at(1), 3, at(9, end - 16), None, None) == -1
    assert lib.mla_kv_read(at(9), 4, 4, 64, at(1), 3, at(9, -1024), None, None) == -1
    assert b"overlaps" in lib.mla_last_error()


def test_binding_wants_one_device(monkeypatch):
    """Tensors of another device than the others', or than the current one, are refused before the call."""
    class On:
        def __init__(self, d):
            self.device, self.get_device = f"cuda:{d}", lambda: d

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(mla, "_torch_c", None)
    mla._require_one_device(On(0), None, On(0))
    for tensors in ((On(0), On(1)), (On(1), On(1)), (On(1), None, On(0))):
        with pytest.raises(ValueError):
            mla._require_one_device(*tensors)
