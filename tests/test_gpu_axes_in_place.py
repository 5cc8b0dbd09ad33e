"""Queries prepared in their own memory by positions of several axes: what is neither rotated nor normalised stays as it is, bit
for bit, and is not written."""
import pytest
import torch

import mla_paged_latent_gb300 as mla
from chunk_helpers import generator, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width, layout", [(192, 0), (192, 4), (576, 0), (576, 2), (512, 1), (512, 3)])
@pytest.mark.parametrize("pe_elsewhere", [False, True])
def test_bits_of_the_nope_part_stay(width, layout, pe_elsewhere):
    g = generator(1)
    tokens, heads, page, nope = 21, 5, 16, width - 64
    row = mla.ROW_ELEMS[layout]
    # every bit pattern of 16 bits, quiet and signalling NaN among them
    bits = (torch.arange(tokens * heads * nope, device="cuda") * 40503 % 65536).to(torch.int32)
    q = torch.empty(tokens, heads, width, dtype=torch.bfloat16, device="cuda")
    q.view(torch.int16)[..., :nope] = torch.where(bits > 32767, bits - 65536, bits).to(torch.int16).view(tokens, heads, nope)
    pe = normal(g, tokens, heads, 64)
    q[..., nope:] = pe
    raw, slots = normal(g, tokens, row), torch.arange(tokens, dtype=torch.int32, device="cuda")
    positions = torch.randint(100, (2, tokens), generator=g, device="cuda", dtype=torch.int32)
    freqs, gain = torch.randn(100, 64, generator=g, device="cuda"), normal(g, 512)
    cache = torch.zeros(2, mla.mla_page_bytes(layout, page), dtype=torch.uint8, device="cuda")
    axes = [0, 1] * 16
    before = q.view(torch.int16).clone()
    mla.mla_qkv_norm_rope_axes(q[..., :nope], pe if pe_elsewhere else q[..., nope:], raw, slots, positions, axes, gain, 1e-6,
                               freqs, q, cache, layout, page)
    assert torch.equal(q.view(torch.int16)[..., :nope], before[..., :nope])
    turn = freqs.view(-1, 32, 2)[positions[torch.tensor(axes, device="cuda")].long(), torch.arange(32, device="cuda")[:, None]]
    cos, sin = turn.transpose(0, 1)[:, None, :, 0].double(), turn.transpose(0, 1)[:, None, :, 1].double()
    u, v = pe[..., 0::2].double(), pe[..., 1::2].double()
    want = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
    size = torch.stack([(u * cos).abs() + (v * sin).abs(), (u * sin).abs() + (v * cos).abs()], -1).flatten(-2)
    assert ((q[..., nope:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -21 * size).all()
