"""4-bit decodes whose running maximum moves: scores that climb past the rescale threshold (64 powers of two) tile by
tile, each time in another half and column group of the tile, so that of the threads that share a query row only
one sees the climb and all have to take it over: O is rescaled between tiles, the sums with it."""
import numpy as np
import pytest
import torch

import mla_paged_latent_gb300 as mla
import workloads
from fp4_helpers import attend, bf16_f64, dense_slots, listed_slots, rows_of
from gpu_helpers import DeviceWorkload, bf16_to_f64

pytestmark = pytest.mark.gpu
FP4 = [mla.MLA_KV_FP4_448_UE8M0, mla.MLA_KV_FP4_512_UE8M0]
STEP = 60.0                                      # > 64 ln 2 = 44.4, in every head


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_paged_latent_gb300 import build
    build.build()
    mla.load()


def _bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(
        np.uint16).copy()


def _peaks(n, tile=128):
    """Heights of rows 0 .. n - 1: in each tile of 128 a few rows of one quarter stand STEP above all before, the
    quarters in turn; over the last third they fall again."""
    j = np.arange(n)
    t, quarter = j // tile, (j % tile) // 32
    up = np.where((quarter == t % 4) & (j % 32 >= 27), STEP * (t + 1), 0.0)
    return np.where(j < 2 * n // 3, up, 10.0)


def _set_heights(w, heights, lead=None, noise=0.02):
    """The first RoPE element carries the scores: the queries' is 1 .. 2 (or `lead`, by head), the rows' height /
    scale."""
    layout, ps = w.cfg.layout, w.cfg.page_size
    rb, nope = workloads._ROW_BYTES[layout], workloads._NOPE[layout]
    rng = np.random.default_rng(11)
    q = np.zeros(w.q.shape, np.float32)
    q[..., :nope] = rng.standard_normal(q[..., :nope].shape) * noise
    q[..., nope] = 1 + rng.random(q.shape[:2]) if lead is None else lead
    w.q[:] = _bits(q)
    for b, h in enumerate(heights):
        j = np.arange(h.size)
        bits = _bits(h / w.cfg.sm_scale)
        page, col = w.block_table[b, j // ps], (j % ps) * rb + rb - 128
        w.kv_cache[page, col], w.kv_cache[page, col + 1] = bits & 255, bits >> 8


def _check(w, slots_of, single_sm, splits, what):
    c = w.cfg
    d = DeviceWorkload(w)
    p = d.make_plan(min_splits=splits, num_sms=None if splits > 1 else 2)
    assert splits == 1 or p.max_splits >= splits
    mla.mla_decode(d.q, d.kv, c.layout, c.page_size, d.bt, d.sl, c.sq, c.sm_scale, d.sched, d.ns, p.num_partitions,
                   p.total_splits, d.ws, d.out, d.lse, sink=d.sink, indices=d.idx, causal=c.causal, single_sm=single_sm)
    assert mla.mla_read_status(d.ws) == 0
    out, lse = bf16_to_f64(d.out), d.lse.cpu().numpy().astype(np.float64)
    for t in range(w.q.shape[0]):
        k = rows_of(w.kv_cache, c.layout, c.page_size, slots_of(t))
        ref, ref_lse, mean, _ = attend(bf16_f64(w.q[t]), k, float(np.float32(c.sm_scale)))
        if k.shape[0] == 0:
            assert np.all(out[t] == 0) and np.all(np.isneginf(lse[t])), what
            continue
        # S: the score of a row, at most. The RoPE element joins the sum in the last of its MMAs: four of them round it
        # (2^-23 each, as for a sum that is cut). The scale and the maximum in log2 units are rounded to 2^-24, the
        # argument of the exponential too, a split's lse twice: 1.9 * 2^-21 S in all, taken as 2^-20 S. A weight and the
        # normaliser are off by that factor each, a weight is rounded to bf16, the output too. A weight below 2^-126 is
        # zero in fp32 (e^-87.4; heads climb by up to 120 a tile), and so is a factor that small on what stands in O, whose
        # weights are below 2^4 here where the factor is that small: either takes at most 2^-122 |V| of a row's share.
        e = 2.0 ** -20 * max(1.0, float(np.abs(ref_lse).max())) + 2.0 ** -19
        gone = 2.0 ** -122 * np.abs(k[:, :512]).sum(0)
        off = np.abs(out[t] - ref)
        assert np.all(off <= (2.0 ** -8 + 2.1 * e) * mean + 2.0 ** -8 * np.abs(ref) + gone), (what, t, off.max())
        assert np.all(np.abs(lse[t] - ref_lse) <= 2 * e), (what, t)


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("heads,splits,single_sm", [(128, 1, False), (128, 1, True), (128, 3, False), (256, 1, False),
                                                    (256, 2, False), (64, 1, False), (64, 3, False)])
def test_climb_in_each_quarter(layout, heads, splits, single_sm):
    w = workloads.generate(workloads.dsv3(batch=3, seqlens=(1500, 700, 129), len_dist="fixed", heads=heads, layout=layout,
                                          new_rows=False, seed=12))
    _set_heights(w, [_peaks(int(n)) for n in w.seqlens])
    _check(w, dense_slots(w), single_sm, splits, f"{heads} heads")


def _pairs_of_tiles(layout, heads):
    lens = (384, 640, 946, 300)
    w = workloads.generate(workloads.dsv3(batch=4, seqlens=lens, len_dist="fixed", heads=heads, layout=layout,
                                          new_rows=False, seed=16))
    heights = []
    for n in lens:
        j = np.arange(n)
        t, quarter = j // 128, (j % 128) // 32
        top = np.where(t % 2 == 1, 45.0 * (t // 2) + 43.8, 45.0 * (t // 2))
        heights.append(np.where((quarter == (t // 2 + 2 * t) % 4) & (j % 32 >= 27), top, 0.0))
    return w, heights


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("heads,splits,single_sm", [(128, 1, False), (128, 1, True), (256, 1, False), (128, 2, False),
                                                    (64, 1, False)])
def test_what_a_rescale_leaves_counts(layout, heads, splits, single_sm):
    """Two tiles of nearly the same height, the first just below the threshold over the tile before them and the second
    just above it: the maximum moves by 45 (in heads whose query is 1), and three tenths of the result are what O held
    until then, with weights of e^43.8. Requests end behind different pairs. Of every four heads one has the moves at
    other tiles (twice the height), one none until late (half)."""
    w, heights = _pairs_of_tiles(layout, heads)
    _set_heights(w, heights, lead=np.array([1.0, 1.0, 2.0, 0.5])[np.arange(heads) % 4], noise=0.005)
    _check(w, dense_slots(w), single_sm, splits, f"{heads} heads")


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("heads,single_sm", [(128, False), (128, True), (64, False)])
def test_large_values_under_large_weights(layout, heads, single_sm):
    """Values up to 6 * 2^50 while O holds weights of e^43.8 = 2^63.2: five such rows a tile reach 2^119, and fp32
    holds them. (The scores come from the RoPE part alone.)"""
    w, heights = _pairs_of_tiles(layout, heads)
    ps, rb, nope = w.cfg.page_size, workloads._ROW_BYTES[layout], workloads._NOPE[layout]
    sc = w.kv_cache[:, ps * rb:ps * (rb + 16)].reshape(-1, ps, 16)
    sc[..., :nope // 32] = 127 + 50
    w.kv_cache[:, ps * rb:ps * (rb + 16)] = sc.reshape(-1, ps * 16)
    _set_heights(w, heights, lead=1.0, noise=0.0)
    _check(w, dense_slots(w), single_sm, 1, f"large values, {heads} heads")


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("heads,sq,splits", [(128, 4, 1), (64, 4, 1), (64, 4, 2), (192, 2, 1)])
def test_climb_among_draft_tokens(layout, heads, sq, splits):
    """The last rows climb too, so that each draft token has a maximum of its own, some of them in one group of query
    rows."""
    w = workloads.generate(workloads.verify(batch=3, sq=sq, heads=heads, seqlens=(900, 257, sq), len_dist="fixed",
                                            layout=layout, new_rows=False, seed=13))
    heights = [_peaks(int(n)) for n in w.seqlens]
    for h in heights:
        h[-sq:] = h.max() + STEP * (1 + np.arange(sq))
    _set_heights(w, heights)
    _check(w, dense_slots(w), False, splits, f"{sq} x {heads}")


@pytest.mark.parametrize("layout", FP4)
@pytest.mark.parametrize("heads,single_sm,splits", [(128, False, 1), (128, True, 1), (256, False, 1), (128, False, 2),
                                                    (64, False, 1)])
def test_climb_behind_an_empty_tile(layout, heads, single_sm, splits):
    """Lists whose first 128 or 192 entries are unused, with holes behind them; one list has a single row at its end."""
    topk = 896
    w = workloads.generate(workloads.sparse(batch=4, heads=heads, seqlens=(1000,) * 4, layout=layout, topk=topk,
                                            page_size=64, min_splits=1, new_rows=False, seed=14))
    _set_heights(w, [_peaks(1000)] * 4)
    rng = np.random.default_rng(15)
    w.indices[:] = -1
    for t, first in ((0, 128), (1, 192), (2, 128)):
        w.indices[t, first:] = np.arange(topk - first)       # in order, so that they climb tile by tile
    w.indices[2, 128:][rng.random(topk - 128) < 0.3] = -1
    w.indices[3, topk - 1] = 128 + 32 + 31                   # the only one
    _check(w, listed_slots(w), single_sm, splits, f"listed, {heads} heads")
