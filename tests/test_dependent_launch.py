"""Every kernel is launched so that it may be on its SMs before the kernel ahead of it on the stream has ended
(programmatic dependent launch, `launch_pdl`), and what that kernel writes is what it reads. The non-coherent load
path is for memory that nothing writes while a kernel lives, so no kernel source takes it, nor declares a pointer
free of aliases, from which the compiler may take it by itself; and each kernel waits before its first load."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_paged_latent_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def _code(path):
    src = re.sub(r"/\*.*?\*/", " ", open(path, encoding="utf-8").read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", src)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_non_coherent_loads(path):
    code = _code(path)
    for form in (r"ld\.global(\.\w+)*\.nc\b", r"__ldg\b", r"__restrict__", r"__restrict\b"):
        found = re.search(form, code)
        assert found is None, f"{os.path.basename(path)}: {found.group(0)}"


@pytest.mark.parametrize("path", [p for p in SOURCES if p.endswith(".cu")], ids=os.path.basename)
def test_kernels_wait_for_the_grid_ahead(path):
    code = _code(path)
    kernels = re.split(r"__global__", code)[1:]
    for k in kernels:
        assert "pdl_wait()" in k, re.search(r"(\w+)\s*\(", k).group(1)
