"""Kernels that are set up while the kernel before them runs, on the CPU: what their sources hold."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "free_block_sparse_means_b200", "csrc")


def code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


EARLY = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu") and "spr_launch_early(" in code(f))


def test_there_are_such_sources():
    assert EARLY == ["k_attend_masked.cu", "k_norm_rotate.cu", "k_project.cu"]


@pytest.mark.parametrize("name", EARLY)
def test_no_load_on_the_read_only_path(name):
    """The data may be written by the kernel before, while this one is resident: no __ldg, no
    ld.global.nc, and no pointer that lets the compiler choose them."""
    found = [w for w in ("__ldg", "ld.global.nc", ".nc.", "__restrict__") if w in code(name)]
    assert not found, found


@pytest.mark.parametrize("name", EARLY)
def test_every_kernel_waits_for_the_one_before(name):
    text = code(name)
    kernels = re.split(r"__global__", text)[1:]
    assert kernels
    for k in kernels:
        body = k[k.index("{"):]
        assert "after_previous();" in body, k[:200]
