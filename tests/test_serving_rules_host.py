"""Rules of the few-token serving operators that need no GPU to be checked: the
order of synchronisation in the kernels' sources, launch plans, size limits,
and the state of the modules."""
import os
import re

import pytest

from backward_tcgen05_tma_gb300 import build

KERNELS = ["w4_stream.cuh", "w4_tensor.cuh", "experts.cuh"]


def source(name):
    """A serving source without comments."""
    with open(os.path.join(build.CSRC_SERVING, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", KERNELS)
def test_barriers_are_initialised_for_the_whole_block(name):
    # an mbarrier that one thread initialises may be waited on by the others
    # only past a barrier of the block
    text = source(name)
    text = text[text.index("__global__"):]
    begin = text.rindex("fence_mbar_init();")
    wait = min(m.start() for m in re.finditer(r"mbar_(try_)?wait(_bounded)?\(", text) if m.start() > begin)
    assert re.search(r"__syncthreads\(\)|ft_build_lists<", text[begin:wait])
    assert not re.search(r"mbar_(try_)?wait(_bounded)?\(", text[:begin])


def test_list_building_synchronises_the_block():
    # what the rule above takes for a barrier of the block in experts.cuh
    text = source("fewtok.cuh")
    for name in ("ft_build_lists_warp", "ft_build_lists"):
        body = text[text.index("void %s(" % name):]
        body = body[:body.index("\n}\n")]
        assert body.rstrip().endswith("__syncthreads();")


@pytest.mark.parametrize("name", KERNELS + ["moe_route.cuh", "fewtok.cuh"])
def test_no_read_only_loads(name):
    # every launch is a programmatic dependent: what it reads may still be
    # written while it runs, which the read-only path does not allow
    text = source(name)
    assert "__ldg(" not in text and "ld.global.nc" not in text
