"""What the kernels that are launched early promise, read from their sources (no GPU).

A kernel launched with launch_early() may be resident while the kernel ahead of it still writes.
So it may not have the compiler take any global data for constant (the read-only path needs that
for the kernel's whole life), nor use loads that the wait for the kernels ahead does not hold back."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_video_diffusion_b200", "csrc")


def _code(name):
    """The source without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


EARLY = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu") and re.search(r"\blaunch_(early|items)\(", _code(f)))


def test_the_sources_are_found():
    assert {"dp_mx4.cu", "dp_mx4_gemm.cu", "dp_packed.cu", "dp_packed_few.cu", "dp_packed_tc.cu"} <= set(EARLY)


@pytest.mark.parametrize("name", EARLY)
def test_no_global_data_is_taken_for_constant(name):
    found = re.findall(r"__ld[a-z]+\b|\.nc\b|__restrict__|ld\.global(?!\.cs\.v4)[.a-z0-9]*", _code(name))
    assert not found, found


@pytest.mark.parametrize("name", EARLY)
def test_every_kernel_waits_for_the_ones_ahead(name):
    kernels = re.split(r"__global__", _code(name))[1:]
    assert kernels and all("wait_for_earlier_kernels();" in k for k in kernels)


@pytest.mark.parametrize("name", EARLY)
def test_the_next_kernel_starts_behind_the_wait(name):
    """A kernel behind may read, before a wait of its own, what its predecessor does not write: it
    must not start while kernels ahead of this one still run."""
    for kernel in re.split(r"__global__", _code(name))[1:]:
        at = kernel.find("let_next_kernel_start();")
        assert at < 0 or 0 <= kernel.find("wait_for_earlier_kernels();") < at
