"""The matrix product with bias, activation and residual against its definition in 64 bits."""
import pytest
import torch

import mla_paged_latent_gb300 as mla
from chunk_helpers import H, generator, normal

pytestmark = pytest.mark.gpu


def reference(x, w, bias, act, residual):
    """(result, its bound): fp32 sums of K products, the activation's slope at most 1.13 and its own error 2^-18 of the value
    (and of |y| e^-|y| at most, far below the bound, where it is cut to zero), one rounding."""
    xd, wd = x.double(), w.double()
    y = xd @ wd.T
    off = (x.shape[1] + 2) * 2.0 ** -23 * (xd.abs() @ wd.abs().T)
    if bias is not None:
        y = y + bias.double()
        off = off + 2.0 ** -23 * y.abs()
    if act == "silu":
        y = y * torch.sigmoid(y)
    elif act == "gelu":
        y = y * torch.special.ndtr(y)
    if act is not None:
        off = 1.13 * off + 2.0 ** -18 * y.abs()
    if residual is not None:
        y = y + residual.double()
        off = off + 2.0 ** -23 * y.abs()
    return y, off * (1 + H) + H * y.abs() + 1e-37


def check(x, w, bias=None, act=None, residual=None, out=None):
    out = torch.full((x.shape[0], w.shape[0]), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    want, bound = reference(x, w, bias, act, residual)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_linear(x, w, out, bias=bias, activation=act, residual=residual, status=status)
    err = (out.double() - want).abs()
    assert status.item() == 0
    assert (err <= bound).all(), f"largest error over its bound: {(err / bound).max().item():.3g}"
    return out


ROWS = [1, 2, 15, 16, 17, 33, 64, 65, 127, 128, 129, 200, 256, 257, 300, 511, 777, 1030]


@pytest.mark.parametrize("rows", ROWS)
def test_rows(rows):
    g = generator(rows)
    check(normal(g, rows, 512), normal(g, 384, 512, scale=512 ** -0.5))


@pytest.mark.parametrize("rows", [1, 20, 100, 300])
@pytest.mark.parametrize("inner, outer", [(8, 8), (16, 264), (64, 128), (72, 8), (136, 136), (1000, 520), (2056, 1032), (4096, 64),
                                          (200, 2600)])
def test_sizes(rows, inner, outer):
    g = generator(inner + outer)
    check(normal(g, rows, inner), normal(g, outer, inner, scale=inner ** -0.5), normal(g, outer), "gelu", normal(g, rows, outer))


@pytest.mark.parametrize("rows", [1, 40, 300])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("residual", [False, True])
def test_epilogue(rows, bias, act, residual):
    g = generator(5)
    check(normal(g, rows, 320), normal(g, 200, 320, scale=3 * 320 ** -0.5), normal(g, 200) if bias else None, act,
          normal(g, rows, 200) if residual else None)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [4, 300])
def test_activation_far_out(act, rows):
    """Sums from -300 to 300 and infinities: no NaN but where the definition has one."""
    g = generator(6)
    x = torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.linspace(-300, 300, rows, device="cuda").to(torch.bfloat16)
    w = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = 1
    check(x, w, act=act)
    bias = torch.full((64,), 3e38, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(rows, 64, dtype=torch.bfloat16, device="cuda")
    mla.mla_linear(x, w, out, bias=bias, activation=act)
    assert (out > 1e38).all()
    mla.mla_linear(x, w, out, bias=-bias, activation=act)
    assert (out == 0).all()
    x[1, 0] = float("nan")
    mla.mla_linear(x, w, out, activation=act)
    assert torch.isnan(out[1]).all() and not torch.isnan(out[0]).any() and not torch.isnan(out[2:]).any()


@pytest.mark.parametrize("rows", [3, 128, 290])
def test_strides(rows):
    """Rows apart by more than they hold; what lies between the output's rows stays."""
    g = generator(7)
    x, res = normal(g, rows, 520)[:, 8:264], normal(g, rows, 400)[:, 16:16 + 328]
    wide = torch.full((rows, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    check(x, normal(g, 328, 256, scale=1 / 16), None, "silu", res, out=wide[:, 64:64 + 328])
    assert (wide[:, :64] == 7).all() and (wide[:, 64 + 328:] == 7).all()


@pytest.mark.parametrize("rows", [3, 128, 290])
def test_residual_in_place(rows):
    g = generator(8)
    x, w, res = normal(g, rows, 256), normal(g, 256, 256, scale=1 / 16), normal(g, rows, 256)
    want = check(x, w, residual=res)
    mla.mla_linear(x, w, res, residual=res)
    assert torch.equal(res, want)


@pytest.mark.parametrize("rows", [5, 64, 400])
def test_the_same_result_every_time_and_captured(rows):
    g = generator(9)
    x, w = normal(g, rows, 4096), normal(g, 1024, 4096, scale=1 / 64)
    want = check(x, w)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    mla.mla_linear(x, w, out)
    with torch.cuda.graph(graph):
        mla.mla_linear(x, w, out)
    for _ in range(5):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


def test_a_row_does_not_depend_on_its_neighbours():
    """NaN rows beside a row, and past the last row of a wider buffer."""
    g = generator(10)
    x, w = normal(g, 300, 256), normal(g, 512, 256, scale=1 / 16)
    for rows in (40, 290):
        want = check(x[:rows], w)
        y = x.clone()
        y[rows:] = float("nan")
        y[3] = float("nan")
        out = torch.empty_like(want)
        mla.mla_linear(y[:rows], w, out)
        assert torch.isnan(out[3]).all()
        out[3] = want[3]
        assert torch.equal(out, want)
