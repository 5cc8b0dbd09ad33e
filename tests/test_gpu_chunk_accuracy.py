"""How far a chunk's attention is from its definition in 64 bits, by what it rounds: the result and K to bf16, V and the softmax
weights to fp16; the same bits at every call; and groups of heads whose units are cut."""
import math

import pytest
import torch

import mla_paged_latent_gb300 as mla
from chunk_helpers import Cache, chunk_reference, generator, normal, run_chunk

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(192)


def make(seed, new, lens, heads, layout=0, keys=True):
    g = generator(seed)
    cache = Cache(g, lens, layout, 16)
    q, w = normal(g, sum(new), heads, 192), normal(g, heads, 256, 512, scale=512 ** -0.5)
    if not keys:
        w[:, :128] = 0
    return q, cache, w


def relative(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


# With r the relative error (of the norm) of rounding the exact result to bf16, a rounding of like numbers to fp16 makes r / 8: three
# bits more. The weights' and V's roundings are independent and pass into the sum of the weighted rows, whose terms have random
# signs, as they are: sqrt(r^2 + 2 (r / 8)^2) = 1.02 r. With both in bf16 it would be sqrt(3) r = 1.73 r.
# K's rounding, where the NoPE part of the scores is not zero, moves a score by r times the size of its 128 random terms: of
# variance 1, scaled by 192^-0.5, that is sqrt(128 / 192) r of every weight, in all sqrt(1 + 0.67 + 0.03) r = 1.30 r; in bf16
# sqrt(1 + 0.67 + 2) r = 1.92 r.
@pytest.mark.parametrize("keys, limit", [(False, 1.2), (True, 1.5)])
@pytest.mark.parametrize("layout", [0, 2, 4])
@pytest.mark.parametrize("new, lens", [([200, 37], [200, 37]), ([300], [2500]), ([70, 513], [6000, 900])])
def test_norm_of_the_error(keys, limit, layout, new, lens):
    q, cache, w = make(1, new, lens, 4, layout, keys)
    out, lse, _, ws = run_chunk(q, cache, new, w, SCALE)
    assert mla.mla_read_status(ws) == 0
    ref = chunk_reference(q, cache, new, w, SCALE, True)[0]
    r = relative(ref.to(torch.bfloat16), ref)
    assert relative(out, ref) < limit * r, (relative(out, ref), r)


@pytest.mark.parametrize("length", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("small", [0, 18, 30])
def test_every_element_of_few_rows(length, small):
    """Scores without a rounding of K: a weight is off by 2^-11, V by 2^-11 of itself or 2^-33, the exponential and the sum by
    2^-18, the result by 2^-8; sums of 64 products by 2^-17 of their magnitudes in a score of at most 2^5. V's own sum of 512
    products in fp32, taken off by 512 2^-23 of their magnitudes, is what the rows below are measured against. Half of the dims are
    smaller by 2^small."""
    new, lens = [1] * 40, [length] * 40
    q, cache, w = make(2, new, lens, 8, 0, keys=False)
    w[:, 128:192] *= 2.0 ** -small
    out, _, _, ws = run_chunk(q, cache, new, w, SCALE)
    assert mla.mla_read_status(ws) == 0
    scale = torch.tensor(SCALE, dtype=torch.float32).double().item()
    for b in range(40):
        rows = cache.rows(b)
        k, c = rows[:, 512:], rows[:, :512]
        s = q[b, :, 128:].double() @ k.T * scale
        off = 64 * 2.0 ** -23 * (q[b, :, 128:].double().abs() @ k.abs().T * scale).amax(1)
        p = torch.softmax(s, 1)
        for h in range(8):
            v = c @ w[h, 128:].double().T
            v_off = 2.0 ** -11 * v.abs() + 2.0 ** -33 + 512 * 2.0 ** -23 * (c.abs() @ w[h, 128:].double().abs().T)
            ref = p[h] @ v
            bound = (p[h] @ v.abs()) * (2.0 ** -11 + 2.0 ** -18 + 2 * off[h]) * 1.01 + (p[h] @ v_off) * 1.01
            bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
            assert ((out[b, h].double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("new, lens", [([300, 70], [2500, 6000]), ([1500, 1, 90], [1700, 333, 4000])])
def test_the_same_bits_every_time(new, lens):
    q, cache, w = make(3, new, lens, 6)
    first = run_chunk(q, cache, new, w, SCALE)
    for _ in range(10):
        again = run_chunk(q, cache, new, w, SCALE)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads, held", [(7, 3), (8, 2), (5, 1)])
def test_groups_of_heads_with_cut_units(causal, heads, held):
    """Heads in groups (the last one shorter), each group's units cut over the rows and merged."""
    new, lens = [256, 100], [7000, 5000]
    q, cache, w = make(4, new, lens, heads)
    rows = sum(-(-n // 128) * 128 for n in lens)
    out, lse, plan, ws = run_chunk(q, cache, new, w, SCALE, causal, kv_budget=held * rows * 512)
    assert plan.group <= held and plan.info.merges > 0 and mla.mla_read_status(ws) == 0
    ref, ref_lse, bound, lse_bound = chunk_reference(q, cache, new, w, SCALE, causal)
    assert ((out.double() - ref).abs() <= bound).all()
    assert ((lse.double() - ref_lse).abs() <= lse_bound).all()
