"""NaN through the merge of split partials: a row is empty only if every partial is (lse = -inf); a partial whose
lse is NaN makes NaN of its row, whatever stands beside it. The merge alone, its two fused forms, and 4-bit decodes
that a plan cuts into splits."""
import numpy as np
import pytest
import torch

import mla_paged_latent_gb300 as mla
import workloads
from gpu_helpers import DeviceWorkload, bf16_to_f64

pytestmark = pytest.mark.gpu
FP4 = [mla.MLA_KV_FP4_448_UE8M0, mla.MLA_KV_FP4_512_UE8M0]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_paged_latent_gb300 import build
    build.build()
    mla.load()


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _partials(rows, ns, seed):
    """Partials of one request: rows 0-2 have NaN and nothing else or empty splits, row 3 is empty, row 4 has a NaN
    among numbers, the others are ordinary. Values of an empty split are not numbers and must not count."""
    rng = np.random.default_rng(seed)
    po = rng.standard_normal((ns, rows, 512)).astype(np.float32)
    pl = rng.standard_normal((ns, rows)).astype(np.float32)
    pl[:, 0] = np.nan                               # every split
    pl[:, 1], pl[0, 1] = -np.inf, np.nan            # the first, the others empty
    pl[:, 2], pl[ns - 1, 2] = -np.inf, np.nan       # the last
    pl[:, 3] = -np.inf
    pl[ns // 2, 4] = np.nan
    po[np.isneginf(pl)] = np.nan
    return po, pl


def _check(out, lse, rows, what):
    out, lse = out.reshape(rows, -1), lse.reshape(rows)
    for r in (0, 1, 2, 4):
        assert np.isnan(lse[r]) and np.isnan(out[r]).all(), f"{what}: row {r}"
    assert np.isneginf(lse[3]) and np.all(out[3] == 0), what
    assert np.isfinite(out[5:]).all() and np.isfinite(lse[5:]).all(), what


@pytest.mark.parametrize("rows", [8, 400, 600])     # four warps a row, and one
@pytest.mark.parametrize("ns", [2, 3, 4, 5, 33])
@pytest.mark.parametrize("sink", [False, True])
def test_merge_keeps_nan(rows, ns, sink):
    po, pl = _partials(rows, ns, rows + ns)
    counts = _cuda(np.array([0, ns], np.int32))
    s = _cuda(np.zeros(rows, np.float32)) if sink else None
    out = torch.full((1, rows, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, rows), 7.0, device="cuda")
    mla.mla_combine(_cuda(po), _cuda(pl), counts, rows, rows, out, lse, sink=s)
    _check(bf16_to_f64(out), lse.cpu().numpy(), rows, "combine")
    # the fused forms merge the same rows to the same bits
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    freqs = torch.zeros(1, 64, device="cuda")
    freqs[:, 0::2] = 1                              # the identity
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_combine_inv_rope(_cuda(po), _cuda(pl), counts, 1, rows, pos, freqs, o2, l2, sink=s)
    _check(bf16_to_f64(o2), l2.cpu().numpy(), rows, "inverse RoPE")
    w = torch.randn(rows, 512, 128, device="cuda").to(torch.bfloat16)
    ov = torch.full((1, rows, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    mla.mla_combine_v_up(_cuda(po), _cuda(pl), counts, 1, rows, w, o2, l2, ov, sink=s)
    _check(bf16_to_f64(o2), l2.cpu().numpy(), rows, "up-projection")
    _check(bf16_to_f64(ov), l2.cpu().numpy(), rows, "up-projection's values")


@pytest.mark.parametrize("rows,splits", [(513, 2), (520, 5), (600, 21), (600, 33), (512, 33)])
def test_merge_of_many_rows(rows, splits):
    """One warp a row (and, at 512, the last count with four), in 64 bits; some partials empty, one row wholly."""
    rng = np.random.default_rng(rows + splits)
    po = rng.standard_normal((splits, rows, 512)).astype(np.float32)
    pl = (3 * rng.standard_normal((splits, rows))).astype(np.float32)
    empty = rng.random((splits, rows)) < 0.2
    empty[0], empty[:, 3] = False, True
    pl[empty], po[empty] = -np.inf, np.nan
    sink = rng.standard_normal(rows).astype(np.float32)
    out = torch.empty(rows, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(rows, device="cuda")
    mla.mla_combine(_cuda(po), _cuda(pl), _cuda(np.array([0, splits], np.int32)), rows, rows, out, lse, sink=_cuda(sink))
    got, glse = bf16_to_f64(out), lse.cpu().numpy().astype(np.float64)
    assert np.isneginf(glse[3]) and np.all(got[3] == 0)
    keep = np.arange(rows) != 3
    l, o = pl[:, keep].astype(np.float64), np.where(empty, 0.0, po.transpose(2, 0, 1))[:, :, keep].astype(np.float64)
    ref_lse = np.log(np.exp(l).sum(0))
    wt = np.exp(l - ref_lse) / (1 + np.exp(sink[keep] - ref_lse))
    ref, mean = np.einsum("sr,dsr->rd", wt, o), np.einsum("sr,dsr->rd", wt, np.abs(o))
    # fp32 weights: exponentials and logarithm (2 units each), their arguments (|lse| below 16: 2^-20), sums of up to 33
    # terms (33 * 2^-24 of their magnitudes); then one rounding to bf16
    assert np.all(np.abs(glse[keep] - ref_lse) <= 2.0 ** -19)
    assert np.all(np.abs(got[keep] - ref) <= 2.0 ** -17 * mean + 2.0 ** -8 * np.abs(ref))


def _nan_scales(w, request, rows):
    """Scale byte 255 in group 0 of the request's first `rows` rows."""
    layout, ps = w.cfg.layout, w.cfg.page_size
    rb = workloads._ROW_BYTES[layout]
    for j in range(rows):
        w.kv_cache[w.block_table[request, j // ps], ps * rb + 16 * (j % ps)] = 255


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("heads", [64, 128])
def test_every_split_of_a_request_is_nan(layout, heads):
    """A request of NaN rows alone, in one split and in several; its neighbour is whole."""
    w = workloads.generate(workloads.dsv4(batch=2, seqlens=(100, 100), len_dist="fixed", heads=heads, layout=layout,
                                          new_rows=False))
    _nan_scales(w, 0, 100)
    for splits in (1, 2):
        d = DeviceWorkload(w)
        assert d.make_plan(min_splits=splits).max_splits >= splits
        d.decode()
        assert mla.mla_read_status(d.ws) == 0
        assert d.out[0].isnan().all() and d.lse[0].isnan().all(), splits
        assert torch.isfinite(d.out[1].float()).all() and torch.isfinite(d.lse[1]).all(), splits


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("front", [True, False])
def test_nan_beside_empty_splits(layout, heads, front):
    """Few listed rows under a long list, one of them NaN: the splits beside it have nothing to say."""
    w = workloads.generate(workloads.sparse(batch=2, heads=heads, seqlens=(300, 300), layout=layout, topk=640,
                                            page_size=64, min_splits=5, new_rows=False))
    _nan_scales(w, 0, 1)
    w.indices[:] = -1
    at = slice(0, 60) if front else slice(580, 640)
    w.indices[0, at], w.indices[1, at] = np.arange(60), np.arange(100, 160)
    d = DeviceWorkload(w)
    assert d.make_plan().max_splits >= 5
    d.decode()
    assert mla.mla_read_status(d.ws) == 0
    assert d.out[0].isnan().all() and d.lse[0].isnan().all()
    assert torch.isfinite(d.out[1].float()).all() and torch.isfinite(d.lse[1]).all()


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("heads", [64, 128])
def test_nan_query_row(layout, heads):
    """One head's query is NaN: that row of the output in every plan, and no other."""
    w = workloads.generate(workloads.dsv4(batch=2, seqlens=(300, 40), len_dist="fixed", heads=heads, layout=layout,
                                          new_rows=False))
    w.q[0, 3] = 0x7FC0
    for splits in (1, 4):
        d = DeviceWorkload(w)
        d.make_plan(min_splits=splits)
        d.decode()
        assert mla.mla_read_status(d.ws) == 0
        nan = torch.zeros(2, heads, dtype=torch.bool, device="cuda")
        nan[0, 3] = True
        assert torch.equal(d.lse.isnan(), nan) and torch.equal(d.out.isnan().all(-1), nan), splits
        assert torch.equal(d.out.isnan().any(-1), nan), splits
