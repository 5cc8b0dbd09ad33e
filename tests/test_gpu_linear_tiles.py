"""The matrix product where a pair of SMs takes several tiles, of every width: both accumulators, the residual that is asked for
ahead, tails of 32 columns, more than one band of row tiles."""
import pytest
import torch

import mla_paged_latent_gb300 as mla
from chunk_helpers import generator, normal
from test_gpu_linear import check

pytestmark = pytest.mark.gpu

# rows, outer: columns of a tile and rounds over 76 pairs (152 SMs)
SIZES = {"160 wide": (200, 9984), "160 wide, ends in the tail": (200, 10056), "160, two rounds": (1000, 5096),
         "192, two rounds": (1001, 6152), "224, two rounds": (1003, 7368), "224, three bands": (5000, 648),
         "256, two rounds": (1001, 8712), "192, three rounds and two bands": (2309, 4104),
         "256, two rounds and two bands": (2600, 2920), "224, three rounds": (777, 12000)}
EPILOGUES = {"plain": (False, None, False), "bias and residual": (True, None, True), "silu": (False, "silu", True),
             "gelu": (True, "gelu", True)}


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("epilogue", EPILOGUES)
@pytest.mark.parametrize("inner", [72, 456])
def test_tiles(size, epilogue, inner):
    """Strided operands; what lies beside the output stays."""
    rows, outer = SIZES[size]
    bias, act, residual = EPILOGUES[epilogue]
    g = generator(rows + outer + inner)
    x = normal(g, rows, inner + 64)[:, 64:]
    w = normal(g, outer, inner, scale=inner ** -0.5)
    wide = torch.full((rows + 2, outer + 32), 7.0, dtype=torch.bfloat16, device="cuda")
    check(x, w, normal(g, outer) if bias else None, act, normal(g, rows, outer + 8)[:, 8:] if residual else None,
          out=wide[1:-1, 16:-16])
    assert (wide[:, :16] == 7).all() and (wide[:, -16:] == 7).all() and (wide[0] == 7).all() and (wide[-1] == 7).all()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_residual_in_place(size, act):
    rows, outer = SIZES[size]
    g = generator(rows + outer)
    x, w, res = normal(g, rows, 136), normal(g, outer, 136, scale=1 / 12), normal(g, rows, outer)
    want = torch.empty_like(res)
    mla.mla_linear(x, w, want, activation=act, residual=res)
    for _ in range(3):
        again = res.clone()
        mla.mla_linear(x, w, again, activation=act, residual=again)
        assert torch.equal(again, want)


@pytest.mark.parametrize("rows", [3, 50, 300, 1001])
@pytest.mark.parametrize("act", [None, "silu", "gelu"])
def test_infinite_sums(rows, act):
    """+inf stays, -inf times 0 is NaN with an activation (y / (1 + e^-y) and y Phi(y) as they stand), and neither leaves its row."""
    outer = 136 if rows < 1000 else 6152
    g = generator(3)
    x, w = normal(g, rows, 72), normal(g, outer, 72, scale=1 / 8)
    w[:, 5] = 1
    want = torch.empty(rows, outer, dtype=torch.bfloat16, device="cuda")
    mla.mla_linear(x, w, want, activation=act)
    x[0, 5], x[2, 5] = float("inf"), float("-inf")
    out = torch.empty_like(want)
    mla.mla_linear(x, w, out, activation=act)
    assert (out[0] == float("inf")).all()
    assert (out[2] == float("-inf")).all() if act is None else torch.isnan(out[2]).all()
    rest = [i for i in range(rows) if i not in (0, 2)]
    assert torch.equal(out[rest], want[rest])
