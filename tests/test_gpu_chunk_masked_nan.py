"""A NaN or an infinity in a cached row reaches the queries that see the row and no others, whichever tile it lies in."""
import math

import pytest
import torch

import mla_paged_latent_gb300 as mla
from chunk_helpers import Cache, chunk_reference, generator, normal, run_chunk

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(192)
BAD = {"a row of NaN": lambda row: row.fill_(math.nan), "one NaN": lambda row: row[:, 77].fill_(math.nan),
       "an infinity": lambda row: row[:, 5].fill_(math.inf), "a RoPE element": lambda row: row[:, 530].fill_(math.nan)}


def slot_of(cache, b, pos):
    return int(cache.table[b, pos // cache.page]) * cache.page + pos % cache.page


# (NaN in the latent part of an fp8 or 4-bit row: the next test)
@pytest.mark.parametrize("layout, bad", [(0, bad) for bad in BAD] + [(2, "a RoPE element"), (4, "a RoPE element")])
@pytest.mark.parametrize("new, lens, at", [([300, 20], [300, 40], [280]), ([300, 20], [900, 40], [605, 730, 899]),
                                           ([600, 20], [600, 40], [0]), ([129, 20], [129, 40], [128]),
                                           ([513, 20], [7000, 40], [6490])])
def test_only_the_queries_that_see_the_row(bad, layout, new, lens, at):
    g = generator(1)
    cache = Cache(g, lens, layout, 16)
    q, w = normal(g, sum(new), 3, 192), normal(g, 3, 256, 512, scale=512 ** -0.5)
    want, want_lse, _, _ = run_chunk(q, cache, new, w, SCALE)
    first = lens[0] - new[0]  # row of the first new token
    sees = torch.zeros(sum(new), dtype=torch.bool, device="cuda")
    for pos in at:
        rows = normal(generator(2), 1, 576)
        BAD[bad](rows)
        mla.mla_kv_write(rows, torch.tensor([slot_of(cache, 0, pos)], dtype=torch.int32, device="cuda"), cache.data, layout, 16)
        sees[:new[0]] |= first + torch.arange(new[0], device="cuda") >= pos
    out, lse, _, ws = run_chunk(q, cache, new, w, SCALE)
    assert mla.mla_read_status(ws) == 0
    assert torch.equal(out[~sees], want[~sees]) and torch.equal(lse[~sees], want_lse[~sees])
    assert torch.isnan(out[sees]).all() and torch.isnan(lse[sees]).all()


@pytest.mark.parametrize("layout", [2, 4])
def test_cached_groups_that_hold_no_number(layout):
    """A scale byte of 255: NaN in a group of an fp8 or 4-bit row."""
    g = generator(3)
    new, lens, pos = [200], [400], 330
    cache = Cache(g, lens, layout, 16)
    q, w = normal(g, 200, 2, 192), normal(g, 2, 256, 512, scale=512 ** -0.5)
    want, want_lse, _, _ = run_chunk(q, cache, new, w, SCALE)
    row_bytes, slot_bytes = (640, 8) if layout == 2 else (384, 16)
    cache.data[int(cache.table[0, pos // 16]), 16 * row_bytes + slot_bytes * (pos % 16) + 3] = 255
    assert torch.isnan(cache.rows(0)[pos]).any()
    out, lse, _, _ = run_chunk(q, cache, new, w, SCALE)
    before = pos - (lens[0] - new[0])
    assert torch.equal(out[:before], want[:before]) and torch.equal(lse[:before], want_lse[:before])
    assert torch.isnan(out[before:]).all() and torch.isnan(lse[before:]).all()


@pytest.mark.parametrize("new, lens, at", [([300, 20], [300, 40], 280), ([513, 20], [7000, 40], 6490)])
def test_a_row_larger_than_all_others_by_far(new, lens, at):
    """Finite, but near the end of bf16's range: queries that do not see it are as accurate as the others' sizes allow."""
    g = generator(4)
    cache = Cache(g, lens, 0, 16)
    q, w = normal(g, sum(new), 2, 192), normal(g, 2, 256, 512, scale=512 ** -0.5)
    w[:, 128:, 9] = w[:, 128:, 9].clamp(-0.25, 0.25)
    want = run_chunk(q, cache, new, w, SCALE)[0]
    row = normal(generator(5), 1, 576)
    row[0, 9] = 2.0 ** 120
    mla.mla_kv_write(row, torch.tensor([slot_of(cache, 0, at)], dtype=torch.int32, device="cuda"), cache.data, 0, 16)
    out, lse, _, _ = run_chunk(q, cache, new, w, SCALE)
    ref, ref_lse, bound, lse_bound = chunk_reference(q, cache, new, w, SCALE, True)
    sees = torch.zeros(sum(new), dtype=torch.bool, device="cuda")
    sees[:new[0]] = lens[0] - new[0] + torch.arange(new[0], device="cuda") >= at
    assert ((out.double() - ref).abs() <= bound)[~sees].all()
    assert ((lse.double() - ref_lse).abs() <= lse_bound)[~sees].all()
    assert torch.equal(out[new[0]:], want[new[0]:])  # the other request's
