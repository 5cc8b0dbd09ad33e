"""Attention of chunks of new tokens over the paged cache against its definition in 64 bits."""
import math

import pytest
import torch

import mla_paged_latent_gb300 as mla
from chunk_helpers import Cache, chunk_reference, generator, normal, run_chunk

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(192)


def make(seed, new, lens, heads, layout=0, page=16, **kw):
    g = generator(seed)
    cache = Cache(g, lens, layout, page, **kw)
    return normal(g, sum(new), heads, 192), cache, normal(g, heads, 256, 512, scale=512 ** -0.5)


def check(q, cache, new, w, causal=True, scale=SCALE, rms=True, **kw):
    out, lse, plan, ws = run_chunk(q, cache, new, w, scale, causal, **kw)
    assert mla.mla_read_status(ws) == 0
    ref, ref_lse, bound, lse_bound = chunk_reference(q, cache, new, w, scale, causal)
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= bound).all(), f"largest error over its bound: {(err / bound).max().item():.3g}"
    empty = ref_lse == -torch.inf
    assert torch.equal(lse == -torch.inf, empty)
    assert ((lse.double() - ref_lse).abs()[~empty] <= lse_bound[~empty]).all()
    assert (out[empty] == 0).all()
    # four roundings (K, V, the weights, the result), each 0.0017 of its value in the mean square, give 0.0034
    if rms and ref.norm() > 0:
        assert (out.double() - ref).norm() / ref.norm() < 5e-3
    return out, lse, plan


@pytest.mark.parametrize("new, lens", [([1], [1]), ([1], [300]), ([37, 130], [37, 130]), ([128], [128]), ([129], [129]),
                                       ([256], [256]), ([257], [900]), ([512], [512]), ([513], [640]), ([700, 1, 90], [700, 129, 1000]),
                                       ([5, 600, 300], [261, 1500, 300])])
def test_lengths(new, lens):
    check(*make(1, new, lens, 3)[:2], new, make(1, new, lens, 3)[2])


@pytest.mark.parametrize("layout", [0, 2, 4])
@pytest.mark.parametrize("page", [8, 64, 256])
def test_layouts_and_pages(layout, page):
    new, lens = [70, 200], [333, 200]
    q, cache, w = make(2, new, lens, 5, layout, page)
    check(q, cache, new, w)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new, lens", [([0, 40], [100, 40]), ([40, 3], [0, 3]), ([300, 20], [100, 10]), ([10], [0]),
                                       ([0, 9, 0], [50, 77, 0])])
def test_empty_requests_and_queries_before_the_first_row(new, lens, causal):
    """More new tokens than rows: the first queries see nothing (causal)."""
    q, cache, w = make(3, new, lens, 2)
    check(q, cache, new, w, causal)


def test_nothing_to_do():
    q, cache, w = make(4, [1], [5], 2)
    plan = mla.mla_chunk_plan([0], [5], 2)
    out = torch.full((0, 2, 128), 1.0, dtype=torch.bfloat16, device="cuda")
    mla.mla_chunk_attention(q[:0], cache.data, 0, 16, cache.table, w, SCALE, plan, torch.from_numpy(plan.sched).cuda(),
                            mla.alloc_workspace(plan.workspace_bytes), out)


@pytest.mark.parametrize("causal", [True, False])
def test_split_over_the_context(causal):
    """Few queries over many rows: pieces of the rows, merged."""
    new, lens = [70, 300], [6000, 9000]
    q, cache, w = make(5, new, lens, 4)
    assert check(q, cache, new, w, causal)[2].slots > 0


def test_units_whose_sub_tiles_see_little_or_nothing():
    """Causal, more queries than rows, over several units."""
    new, lens = [1500, 1100], [1400, 500]
    q, cache, w = make(6, new, lens, 1)
    check(q, cache, new, w)


@pytest.mark.parametrize("heads", [1, 7, 20])
def test_groups_of_heads(heads):
    """K and V of three heads at a time, the last group shorter."""
    new, lens = [100, 260], [400, 300]
    q, cache, w = make(7, new, lens, heads)
    rows = 512 + 384
    out, lse, plan = check(q, cache, new, w, kv_budget=3 * rows * 512)
    assert plan.group <= 3
    whole = run_chunk(q, cache, new, w, SCALE)
    assert torch.equal(out, whole[0]) and torch.equal(lse, whole[1])


@pytest.mark.parametrize("num_sms", [2, 7, 64])
def test_fewer_pairs(num_sms):
    new, lens = [600, 40, 300], [1000, 40, 700]
    q, cache, w = make(8, new, lens, 3)
    check(q, cache, new, w, num_sms=num_sms)


def test_large_scores_move_the_maximum():
    """Scores of hundreds that grow along the rows: the running maximum moves past its threshold again and again."""
    new, lens = [200], [2000]
    q, cache, w = make(9, new, lens, 2)
    ramp = torch.arange(cache.pages * cache.page, device="cuda") % 97 / 8.0
    rows = normal(generator(10), cache.pages * cache.page, 576)
    rows[:, 512:] = (ramp[:, None] * torch.ones(64, device="cuda")).to(torch.bfloat16)
    mla.mla_kv_write(rows, torch.arange(rows.shape[0], dtype=torch.int32, device="cuda"), cache.data, 0, cache.page)
    q[..., 128:] = q[..., 128:].abs() * 4
    check(q, cache, new, w, rms=False)


def test_rows_of_other_requests_and_stale_memory_do_not_show():
    """NaN in every row that no request has, and in the workspace."""
    new, lens = [30, 140], [45, 333]
    q, cache, w = make(11, new, lens, 2)
    want = run_chunk(q, cache, new, w, SCALE)
    mine = torch.zeros(cache.pages * cache.page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        pos = torch.arange(n, device="cuda")
        mine[cache.table[b].long()[pos // cache.page] * cache.page + pos % cache.page] = True
    nan = torch.full((cache.pages * cache.page, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    slots = torch.where(mine, -1, torch.arange(mine.shape[0], device="cuda")).int()
    mla.mla_kv_write(nan, slots, cache.data, 0, cache.page)
    got = run_chunk(q, cache, new, w, SCALE)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_behind_the_last_token_keep_what_they_held():
    new, lens = [30, 140], [45, 333]
    q, cache, w = make(12, new, lens, 2)
    plan = mla.mla_chunk_plan(new, lens, 2)
    wide = torch.full((sum(new) + 100, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    sums = torch.full((sum(new) + 100, 2), 7.0, device="cuda")
    mla.mla_chunk_attention(q, cache.data, 0, 16, cache.table, w, SCALE, plan, torch.from_numpy(plan.sched).cuda(),
                            mla.alloc_workspace(plan.workspace_bytes), wide[:sum(new)], sums[:sum(new)])
    assert (wide[sum(new):] == 7).all() and (sums[sum(new):] == 7).all()
    want = run_chunk(q, cache, new, w, SCALE)
    assert torch.equal(wide[:sum(new)], want[0]) and torch.equal(sums[:sum(new)], want[1])


def test_the_same_pages_in_two_requests():
    """A shared prefix: both tables name the same pages."""
    new, lens = [60, 33], [200, 200]
    q, cache, w = make(13, new, lens, 2)
    cache.table[1] = cache.table[0]
    check(q, cache, new, w)


def test_bad_pages_are_reported_and_read_as_zeros():
    new, lens = [20], [100]
    q, cache, w = make(14, new, lens, 2)
    table = cache.table.clone()
    table[0, 2] = cache.pages + 5
    out, _, _, ws = run_chunk(q, cache, new, w, SCALE, table=table)
    with pytest.raises(mla.MlaError, match="block_table"):
        mla.mla_read_status(ws)
    page = int(cache.table[0, 2])
    mla.mla_kv_write(torch.zeros(16, 576, dtype=torch.bfloat16, device="cuda"),
                     torch.arange(page * 16, page * 16 + 16, dtype=torch.int32, device="cuda"), cache.data, 0, 16)
    assert torch.equal(out, run_chunk(q, cache, new, w, SCALE)[0])
    short = cache.table[:, :3].contiguous()  # the rows past its end
    _, _, _, ws = run_chunk(q, cache, new, w, SCALE, table=short)
    with pytest.raises(mla.MlaError, match="block_table"):
        mla.mla_read_status(ws)


def test_a_nan_reaches_the_queries_that_see_it():
    new, lens = [300], [300]
    q, cache, w = make(15, new, lens, 1)
    slot = int(cache.table[0, 280 // 16]) * 16 + 280 % 16
    row = torch.full((1, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    want = run_chunk(q, cache, new, w, SCALE)[0]
    mla.mla_kv_write(row, torch.tensor([slot], dtype=torch.int32, device="cuda"), cache.data, 0, 16)
    out, lse, _, _ = run_chunk(q, cache, new, w, SCALE)
    assert torch.isnan(out[280:]).all() and torch.isnan(lse[280:]).all()
    assert torch.equal(out[:128], want[:128])  # queries of whom no tile holds it


def test_another_stream_and_a_captured_call():
    new, lens = [100, 31], [500, 400]
    q, cache, w = make(16, new, lens, 4)
    want, want_lse, _, _ = run_chunk(q, cache, new, w, SCALE)
    plan = mla.mla_chunk_plan(new, lens, 4)
    sched, ws = torch.from_numpy(plan.sched).cuda(), mla.alloc_workspace(plan.workspace_bytes)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mla.mla_chunk_attention(q, cache.data, 0, 16, cache.table, w, SCALE, plan, sched, ws, out, lse, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.mla_chunk_attention(q, cache.data, 0, 16, cache.table, w, SCALE, plan, sched, ws, out, lse)
    q.copy_(normal(generator(17), *q.shape))
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    fresh = run_chunk(q, cache, new, w, SCALE)
    assert torch.equal(out, fresh[0]) and torch.equal(lse, fresh[1])


def scaled_values(seed, new, lens, heads, exponents):
    """Scores from the RoPE part alone; the latent rows of each 32 times a power of two of their own."""
    q, cache, w = make(seed, new, lens, heads)
    w[:, :128] = 0
    n = cache.pages * cache.page
    rows = normal(generator(seed + 100), n, 576)
    power = 2.0 ** exponents(n // 16).repeat_interleave(16).double()  # of a page: two of them are 32 rows of a request, or not
    rows[:, :512] = (rows[:, :512].double() * power[:, None]).to(torch.bfloat16)
    mla.mla_kv_write(rows, torch.arange(n, dtype=torch.int32, device="cuda"), cache.data, 0, cache.page)
    return q, cache, w


@pytest.mark.parametrize("lo, hi", [(-20, 20), (-70, -60), (55, 70), (-4, 60)])
def test_values_of_very_different_size(lo, hi):
    new, lens = [150, 1], [700, 333]
    exps = lambda n: torch.randint(lo, hi + 1, (n,), generator=generator(18), device="cuda")  # noqa: E731
    check(*scaled_values(19, new, lens, 2, exps)[:2], new, scaled_values(19, new, lens, 2, exps)[2], rms=False)


def test_values_that_are_zero():
    new, lens = [40], [200]
    q, cache, w = make(20, new, lens, 2)
    w[:, 128:] = 0
    out, lse, _, _ = run_chunk(q, cache, new, w, SCALE)
    assert (out == 0).all() and torch.isfinite(lse).all()


def test_an_infinite_value_stays_one():
    """One latent element infinite, in a row that all queries of its tile see: the values that it reaches are infinite or NaN (its
    key is too), queries of other requests do not change."""
    new, lens = [20, 20], [300, 200]
    q, cache, w = make(21, new, lens, 1)
    want = run_chunk(q, cache, new, w, SCALE)[0]
    rows = normal(generator(22), 1, 576)
    rows[0, 5] = float("inf")
    slot = int(cache.table[0, 0]) * cache.page
    mla.mla_kv_write(rows, torch.tensor([slot], dtype=torch.int32, device="cuda"), cache.data, 0, cache.page)
    out = run_chunk(q, cache, new, w, SCALE)[0]
    assert not torch.isfinite(out[:20]).any() and torch.equal(out[20:], want[20:])
