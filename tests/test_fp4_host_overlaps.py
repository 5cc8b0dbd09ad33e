"""mla_qkv_norm_rope refuses outputs that lie over any of its inputs, the small ones too (host checks, made before any
device work)."""
import ctypes

import pytest

import mla_paged_latent_gb300 as mla
from mla_paged_latent_gb300 import build as mla_build


@pytest.fixture(scope="module")
def lib():
    mla_build.build()
    return mla.load()


def _at(k, o=0):
    return ctypes.c_void_p(0x1000000 * k + o)


# 3 tokens of 2 heads of 576; bytes of each small input
INPUTS = {"slots": 12, "pos": 12, "kw": 1024, "qw": 1024, "freqs": 100 * 256}


@pytest.mark.parametrize("name", INPUTS)
@pytest.mark.parametrize("output,size", [("out", 3 * 2 * 576 * 2), ("kv", None)])
def test_outputs_over_small_inputs_are_refused(lib, name, output, size):
    size = 4 * mla.mla_page_bytes(4, 64) if size is None else size
    base = 8 if output == "out" else 9
    for place in (0, size - 16, -((INPUTS[name] - 1) // 16 * 16)):      # over the first bytes, the last, by its own end
        a = dict(slots=_at(4), pos=_at(5), kw=_at(6), qw=_at(10), freqs=_at(7))
        a[name] = _at(base, place)
        rc = lib.mla_qkv_norm_rope(_at(1), 1024, 512, _at(2), 128, 64, 1, a["qw"], 1e-6, _at(3), 576, a["slots"], a["pos"],
                                   a["kw"], 1e-6, a["freqs"], 100, 3, 2, _at(8), _at(9), 4, 4, 64, None, None)
        assert rc == -1 and b"overlaps" in lib.mla_last_error(), place
