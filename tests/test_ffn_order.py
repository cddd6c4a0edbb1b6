"""Order of memory under programmatic dependent launch. A kernel launched that way starts before the
kernel ahead of it has written what it reads, so after grid_wait() it may read only through loads
that the compiler keeps behind the wait and that do not ask for data that nobody writes during the
kernel's life: no .nc load (by name, by __ldg, or by a const __restrict__ pointer, which lets the
compiler choose one), and no asm without `volatile` and a memory clobber."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gemv_w4a16_w8a8_b200", "csrc")


def source(path):
    """A source without its comments."""
    with open(path) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


DEPENDENT = sorted(p for p in glob.glob(os.path.join(CSRC, "*.cu")) if "launch_dependent" in source(p))


def test_files_with_dependent_launches():
    assert {"act_quant.cu", "ffn.cu", "ffn_small.cu", "ffn_tile.cu"} <= {os.path.basename(p) for p in DEPENDENT}


@pytest.mark.parametrize("path", DEPENDENT, ids=os.path.basename)
def test_no_read_only_loads(path):
    text = source(path)
    for pattern in (r"\bld_stream_\w+", r"\bld_cached_\w+", r"__ldg", r"\.nc\b",
                    r"const\s+\w+\s*\*\s*__restrict__"):
        assert not re.findall(pattern, text), (os.path.basename(path), pattern)


@pytest.mark.parametrize("path", DEPENDENT, ids=os.path.basename)
def test_every_kernel_waits(path):
    """Every kernel of these files holds the wait that its dependent launch asks for."""
    text = source(path)
    kernels = re.split(r"__global__", text)[1:]
    assert kernels and all("grid_wait()" in k.split("cudaError_t")[0] for k in kernels)


def test_loads_behind_the_wait_are_ordered():
    """The loads that those files use instead: volatile, with a clobber, not .nc."""
    text = source(os.path.join(CSRC, "ffn.cuh"))
    loads = re.findall(r"asm([^;]*?\(\s*\"ld\.global.*?)\);", text, flags=re.S)
    assert len(loads) >= 4
    for body in loads:
        assert body.lstrip().startswith("volatile") and '"memory"' in body and ".nc" not in body, body
