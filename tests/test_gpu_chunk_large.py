"""The chunk's operators where offsets pass 32 bits, and two of their calls at once."""
import math

import pytest
import torch

import mla_paged_latent_gb300 as mla
from chunk_helpers import Cache, chunk_reference, generator, normal, run_chunk
from test_gpu_linear import check as check_linear

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(192)


def test_keys_and_values_past_32_bits():
    """131071 rows at 128 heads: 2^32 elements of K and V, in one group of heads."""
    g = generator(1)
    new, lens, heads = [130], [131071], 128
    cache = Cache(g, lens, 2, 64)
    q, w = normal(g, 130, heads, 192), normal(g, heads, 256, 512, scale=512 ** -0.5)
    out, lse, plan, ws = run_chunk(q, cache, new, w, SCALE)
    assert plan.group == heads and mla.mla_read_status(ws) == 0
    for h in (0, 127):
        ref, ref_lse, bound, lse_bound = chunk_reference(q[:, h:h + 1], cache, new, w[h:h + 1], SCALE, True)
        assert ((out[:, h:h + 1].double() - ref).abs() <= bound).all()
        assert ((lse[:, h:h + 1].double() - ref_lse).abs() <= lse_bound).all()


def test_queries_past_32_bits():
    """90 requests of 1000 tokens at 128 heads: 2.2e9 elements of q. The last requests as they are by themselves."""
    g = generator(2)
    heads, each, n = 128, 1000, 90
    cache = Cache(g, [each], 0, 8)
    q = torch.empty(n * each, heads, 192, dtype=torch.bfloat16, device="cuda")
    for i in range(n):
        q[i * each:(i + 1) * each] = normal(g, each, heads, 192)
    w = normal(g, heads, 256, 512, scale=512 ** -0.5)
    many = Cache.__new__(Cache)
    many.__dict__.update(cache.__dict__)
    many.lens, many.table = [each] * n, cache.table.repeat(n, 1)
    out, lse, _, ws = run_chunk(q, many, [each] * n, w, SCALE)
    assert mla.mla_read_status(ws) == 0
    for i in (0, n - 1):
        mine = q[i * each:(i + 1) * each]
        for h in (0, 127):
            ref, ref_lse, bound, lse_bound = chunk_reference(mine[:, h:h + 1], cache, [each], w[h:h + 1], SCALE, True)
            assert ((out[i * each:(i + 1) * each, h:h + 1].double() - ref).abs() <= bound).all()
            assert ((lse[i * each:(i + 1) * each, h:h + 1].double() - ref_lse).abs() <= lse_bound).all()


@pytest.mark.parametrize("width, layout", [(192, 0), (576, 2), (512, 3)])
def test_rotated_queries_past_32_bits(width, layout):
    """The last tokens of a call with more than 2^31 elements of queries, in place, as they are by themselves."""
    g = generator(3)
    heads, page = 128, 64
    tokens = (2 ** 31 // (heads * width)) + 300
    q = torch.zeros(tokens, heads, width, dtype=torch.bfloat16, device="cuda")
    q[-200:] = normal(g, 200, heads, width)
    raw = normal(g, tokens, mla.ROW_ELEMS[layout])
    slots = torch.arange(tokens, dtype=torch.int32, device="cuda")
    positions = torch.randint(500, (2, tokens), generator=g, device="cuda", dtype=torch.int32)
    freqs, gain = torch.randn(500, 64, generator=g, device="cuda"), normal(g, 512)
    pages = -(-tokens // page)
    caches = [torch.zeros(pages, mla.mla_page_bytes(layout, page), dtype=torch.uint8, device="cuda") for _ in range(2)]
    nope = width - 64
    want = torch.empty(200, heads, width, dtype=torch.bfloat16, device="cuda")
    mla.mla_qkv_norm_rope_axes(q[-200:, :, :nope], q[-200:, :, nope:], raw[-200:], slots[-200:], positions[:, -200:].contiguous(),
                               [0, 1] * 16, gain, 1e-6, freqs, want, caches[0], layout, page)
    mla.mla_qkv_norm_rope_axes(q[..., :nope], q[..., nope:], raw, slots, positions, [0, 1] * 16, gain, 1e-6, freqs, q, caches[1],
                               layout, page)
    assert torch.equal(q[-200:], want)
    rows = [torch.empty(200, mla.ROW_ELEMS[layout], dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for cache, back in zip(caches, rows):
        mla.mla_kv_read(cache, layout, page, slots[-200:], back)
    assert torch.equal(rows[0], rows[1])


def test_products_past_32_bits():
    g = generator(4)
    rows, inner, outer = 300000, 72, 8200
    x, w = normal(g, rows, inner), normal(g, outer, inner, scale=1 / 8)
    res = torch.zeros(rows, outer, dtype=torch.bfloat16, device="cuda")
    res[-300:] = normal(g, 300, outer)
    mla.mla_linear(x, w, res, activation="silu", residual=res)
    want = torch.empty(300, outer, dtype=torch.bfloat16, device="cuda")
    first = torch.empty(300, outer, dtype=torch.bfloat16, device="cuda")
    g2 = generator(4)
    normal(g2, rows, inner), normal(g2, outer, inner)
    check_linear(x[-300:], w, act="silu", residual=normal(g2, 300, outer), out=want)
    check_linear(x[:300], w, act="silu", out=first)
    assert torch.equal(res[-300:], want) and torch.equal(res[:300], first)


def test_two_calls_at_once():
    """Chunks and products on two streams, each with buffers of its own: as one after the other."""
    g = generator(5)
    jobs = []
    for i in range(2):
        new, lens, heads = [[300, 70], [513, 1]][i], [[2500, 600], [700, 4000]][i], 16
        cache = Cache(g, lens, [0, 4][i], 16)
        q, w = normal(g, sum(new), heads, 192), normal(g, heads, 256, 512, scale=512 ** -0.5)
        w_o = normal(g, 1000, heads * 128, scale=0.02)
        plan = mla.mla_chunk_plan(new, lens, heads)
        sched, ws = torch.from_numpy(plan.sched).cuda(), mla.alloc_workspace(plan.workspace_bytes)
        out = torch.empty(sum(new), heads, 128, dtype=torch.bfloat16, device="cuda")
        y, one = (torch.empty(n, 1000, dtype=torch.bfloat16, device="cuda") for n in (sum(new), 1))

        def run(stream, cache=cache, q=q, w=w, w_o=w_o, plan=plan, sched=sched, ws=ws, out=out, y=y, one=one):
            mla.mla_chunk_attention(q, cache.data, cache.layout, 16, cache.table, w, SCALE, plan, sched, ws, out, stream=stream)
            mla.mla_linear(out.view(out.shape[0], -1), w_o, y, activation="gelu", stream=stream)
            mla.mla_linear(out.view(out.shape[0], -1)[:1], w_o, one, stream=stream)
        jobs.append((run, out, y, one, ws))
    streams = [torch.cuda.Stream() for _ in range(2)]
    want = []
    for run, out, y, one, _ in jobs:
        run(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append([t.clone() for t in (out, y, one)])
    for _ in range(20):
        for (run, *_), s in zip(jobs, streams):
            for _ in range(3):
                run(s)
        torch.cuda.synchronize()
        for (_, out, y, one, ws), (a, b, c) in zip(jobs, want):
            assert torch.equal(out, a) and torch.equal(y, b) and torch.equal(one, c) and mla.mla_read_status(ws) == 0
            out.zero_(), y.zero_(), one.zero_()
        torch.cuda.synchronize()


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_query_without_numbers_stays_alone(value):
    g = generator(6)
    new, lens = [300, 20], [700, 40]
    cache = Cache(g, lens, 0, 16)
    q, w = normal(g, 320, 3, 192), normal(g, 3, 256, 512, scale=512 ** -0.5)
    want, want_lse, _, _ = run_chunk(q, cache, new, w, SCALE)
    q[17, 1, 40] = value
    q[310, 2, 150] = value
    out, lse, _, _ = run_chunk(q, cache, new, w, SCALE)
    hit = torch.zeros(320, 3, dtype=torch.bool, device="cuda")
    hit[17, 1] = hit[310, 2] = True
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
    assert torch.isnan(out[hit]).all()
