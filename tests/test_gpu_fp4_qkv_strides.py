"""mla_qkv_norm_rope on one token or one head: the stride of a dimension of size one says nothing about memory, and
torch gives it whatever the tensor's history left there."""
import numpy as np
import pytest
import torch

import mla_paged_latent_gb300 as mla
import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_paged_latent_gb300 import build
    build.build()
    mla.load()


def _call(layout, q_nope, q_pe, raw, out):
    T = q_nope.shape[0]
    i = torch.arange(T, dtype=torch.int32, device="cuda")
    angle = torch.arange(16, device="cuda")[:, None] * 0.3 ** torch.arange(32, device="cuda")
    freqs = torch.stack([angle.cos(), angle.sin()], -1).reshape(16, 64).float()
    ones = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(2, mla.mla_page_bytes(layout, 16), dtype=torch.uint8, device="cuda")
    mla.mla_qkv_norm_rope(q_nope, q_pe, raw, i, i + 1, ones, 1e-6, freqs, out, kv, layout, 16, q_eps=1e-6)
    return kv


@pytest.mark.parametrize("layout", [0, 1, 3, 4])
@pytest.mark.parametrize("T,N", [(1, 24), (5, 1), (1, 1)])
def test_in_place_after_a_product_over_heads(layout, T, N):
    """q comes as [N, T, width] and is prepared in its own memory through its transpose, which is contiguous when either
    count is one."""
    width = workloads._DQK[layout]
    g = torch.Generator(device="cuda").manual_seed(T + N)
    q = torch.randn(N, T, width, generator=g, device="cuda").to(torch.bfloat16).transpose(0, 1)
    raw = torch.randn(T, width, generator=g, device="cuda").to(torch.bfloat16)
    assert q.is_contiguous()
    want = torch.empty(T, N, width, dtype=torch.bfloat16, device="cuda")
    kv = _call(layout, q[..., :width - 64], q[..., width - 64:], raw, want)
    kv2 = _call(layout, q[..., :width - 64], q[..., width - 64:], raw, q)
    assert torch.equal(q, want) and torch.equal(kv, kv2)


@pytest.mark.parametrize("layout", [3, 4])
def test_strides_of_one_token_are_not_read(layout):
    width, N = workloads._DQK[layout], 8
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(1, N, width, generator=g, device="cuda").to(torch.bfloat16)
    raw = torch.randn(1, width, generator=g, device="cuda").to(torch.bfloat16)
    want, out = torch.empty_like(q), torch.empty_like(q)
    kv = _call(layout, q[..., :width - 64], q[..., width - 64:], raw, want)
    for s in (0, 3, 1 << 45):
        qn = q[..., :width - 64].as_strided((1, N, width - 64), (s, width, 1))
        qp = q[..., width - 64:].as_strided((1, N, 64), (s, width, 1))
        out.zero_()
        kv2 = _call(layout, qn, qp, raw.as_strided((1, width), (s, 1)), out)
        assert torch.equal(out, want) and torch.equal(kv, kv2), s
