"""Chunk attention where a request's values differ in size by far: between its rows, and between the dims of a row."""
import math

import pytest
import torch

import mla_paged_latent_gb300 as mla
from chunk_helpers import Cache, chunk_reference, generator, normal, run_chunk

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(192)
PAGE = 32


def split_values(seed, new, lens, heads, power):
    """Value dims 0 to 63 come from the first half of the latent row, dims 64 to 127 from the other half, and the scores from the
    RoPE part alone. power(rows): the power of two of every row's first half."""
    g = generator(seed)
    cache = Cache(g, lens, 0, PAGE)
    q, w = normal(g, sum(new), heads, 192), normal(g, heads, 256, 512, scale=256 ** -0.5)
    w[:, :128] = 0
    w[:, 128:192, 256:] = 0
    w[:, 192:, :256] = 0
    n = cache.pages * PAGE
    rows = normal(generator(seed + 100), n, 576)
    # by the row's place in its request, so that groups of 32 rows and tiles of 128 are known
    place = torch.zeros(n, dtype=torch.int64, device="cuda")
    for b, length in enumerate(lens):
        at = torch.arange(-(-length // PAGE) * PAGE, device="cuda")
        place[cache.table[b].long()[at // PAGE] * PAGE + at % PAGE] = at
    rows[:, :256] = (rows[:, :256].double() * 2.0 ** power(place).double()[:, None]).to(torch.bfloat16)
    mla.mla_kv_write(rows, torch.arange(n, dtype=torch.int32, device="cuda"), cache.data, 0, PAGE)
    return q, cache, w


def check(q, cache, new, w, causal=True, **kw):
    out, lse, plan, ws = run_chunk(q, cache, new, w, SCALE, causal, **kw)
    assert mla.mla_read_status(ws) == 0
    ref, ref_lse, bound, lse_bound = chunk_reference(q, cache, new, w, SCALE, causal)
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= bound).all(), f"largest error over its bound: {(err / bound).max().item():.3g}"
    seen = ref_lse > -torch.inf
    assert ((lse.double() - ref_lse).abs()[seen] <= lse_bound[seen]).all()
    return plan


APART = {
    "every other group of 32 rows": lambda at, far: torch.where(at // 32 % 2 == 0, far, 0),
    "one group": lambda at, far: torch.where(at // 32 == 3, far, 0),
    "one row": lambda at, far: torch.where(at == 37, far, 0),
    "the first tile": lambda at, far: torch.where(at < 128, far, 0),
    "the last tiles": lambda at, far: torch.where(at >= 256, far, 0),
}


@pytest.mark.parametrize("where", APART)
@pytest.mark.parametrize("far", [10, 24, 34, 60])
def test_dims_of_some_rows_are_larger_by_far(where, far):
    """The other dims of all rows, and all dims of the other rows, keep their accuracy."""
    new, lens = [150, 3], [700, 333]
    check(*(x := split_values(1, new, lens, 2, lambda at: APART[where](at, far)))[:2], new, x[2])


@pytest.mark.parametrize("far", [-60, -20, 9, 70])
def test_all_values_of_a_size(far):
    new, lens = [150, 3], [700, 333]
    q, cache, w = split_values(2, new, lens, 2, lambda at: torch.full_like(at, 0))
    n = cache.pages * PAGE
    rows = normal(generator(3), n, 576)
    rows[:, :512] = (rows[:, :512].double() * 2.0 ** far).to(torch.bfloat16)
    mla.mla_kv_write(rows, torch.arange(n, dtype=torch.int32, device="cuda"), cache.data, 0, PAGE)
    check(q, cache, new, w)


def test_large_values_that_no_query_weighs():
    """Rows of a score far below the others', with values far above: the others keep their weights."""
    new, lens = [140], [520]
    q, cache, w = split_values(4, new, lens, 2, lambda at: torch.where(at // 32 % 3 == 1, 40, 0))
    n = cache.pages * PAGE
    rows = normal(generator(5), n, 576)
    place = torch.zeros(n, dtype=torch.int64, device="cuda")
    at = torch.arange(-(-520 // PAGE) * PAGE, device="cuda")
    place[cache.table[0].long()[at // PAGE] * PAGE + at % PAGE] = at
    far = place // 32 % 3 == 1
    rows[:, :512] = (rows[:, :512].double() * torch.where(far, 2.0 ** 40, 1.0)[:, None]).to(torch.bfloat16)
    rows[:, 512] = torch.where(far, -4.0, 4.0).to(torch.bfloat16)
    q[..., 128] = 80.0  # a score of +-23: weights of e^-46 = 2^-66
    mla.mla_kv_write(rows, torch.arange(n, dtype=torch.int32, device="cuda"), cache.data, 0, PAGE)
    check(q, cache, new, w)


@pytest.mark.parametrize("causal", [True, False])
def test_cut_units_of_values_apart(causal):
    new, lens = [70, 300], [6000, 4000]
    q, cache, w = split_values(6, new, lens, 2, lambda at: torch.where(at // 32 % 7 == 2, 30, 0))
    assert check(q, cache, new, w, causal).slots > 0


@pytest.mark.parametrize("head", [0, 3, 6])
def test_one_head_of_a_group_of_heads(head):
    """Values of one head out of fp16's range, heads expanded two at a time: every head to its own accuracy."""
    new, lens = [300, 7], [900, 333]
    q, cache, w = split_values(7, new, lens, 7, lambda at: torch.zeros_like(at))
    w[head, 128:192] *= 2.0 ** 45
    rows = sum(-(-n // 128) * 128 for n in lens)
    assert check(q, cache, new, w, kv_budget=2 * rows * 512).group == 2


@pytest.mark.parametrize("graph", [False, True])
def test_one_workspace_for_calls_of_either_kind(graph):
    """Values in fp16's range, out of it and in it again, in the same buffers: each call as in buffers of its own."""
    new, lens, heads = [300, 7], [900, 333], 3
    q, cache, small = split_values(8, new, lens, heads, lambda at: torch.zeros_like(at))
    large = small.clone()
    large[1, 128:] *= 2.0 ** 30
    want = [run_chunk(q, cache, new, w, SCALE)[:2] for w in (small, large)]
    plan = mla.mla_chunk_plan(new, lens, heads)
    sched, ws = torch.from_numpy(plan.sched).cuda(), mla.alloc_workspace(plan.workspace_bytes)
    w, out, lse = small.clone(), torch.empty_like(want[0][0]), torch.empty_like(want[0][1])

    def run():
        mla.mla_chunk_attention(q, cache.data, 0, PAGE, cache.table, w, SCALE, plan, sched, ws, out, lse)
    if graph:
        run()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            run()
        run = captured.replay
    for k in (0, 1, 0, 1, 1, 0, 0):
        w.copy_((small, large)[k])
        run()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])
    assert not torch.equal(want[0][0], want[1][0])
