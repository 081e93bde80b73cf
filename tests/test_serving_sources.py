"""What the serving kernels' sources have to keep to, read from the files."""
import os
import re

import pytest

from gated_deltanet_recurrent_la_b200 import lastate as L

CSRC = os.path.join(os.path.dirname(os.path.abspath(L.__file__)), "csrc")
SERVING = ("la_tree.cu", "la_tree.cuh", "la_tree_tc.cuh", "la_beam.cu", "la_slots.cu")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", SERVING)
def test_dependent_kernels_do_not_load_through_the_read_only_path(name):
    """They start before the kernel that wrote their inputs has completed, so their inputs are not
    read-only for their whole life, which __ldg and ld.global.nc ask for."""
    assert "__ldg" not in code(name) and ".global.nc" not in code(name)


@pytest.mark.parametrize("name", SERVING)
def test_dependent_kernels_wait_before_they_read(name):
    """Every kernel of these files waits for the one before it."""
    for kernel in re.split(r"__global__", code(name))[1:]:
        body = kernel.split("\n}\n")[0]
        assert "griddep_wait();" in body, kernel[:120]
