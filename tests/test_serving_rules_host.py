"""Rules of the few-token serving operators that need no GPU to be checked: the
order of synchronisation in the kernels' sources, launch plans, size limits,
and the state of the modules."""
import ctypes
import os
import re

import pytest

from backward_tcgen05_tma_gb300 import api, build

UNSUP = 3
P = ctypes.c_void_p(0x10000)  # an aligned fake device address (never dereferenced)
N = ctypes.c_void_p(0)
BIG = 1 << 50

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


def test_rows_copies_are_waited_for_before_the_block_goes():
    # after a wait for the token rows ran out: no further copy on their barrier,
    # and the one under way is waited for (with the same limit) at the end
    text = source("w4_stream.cuh")
    stage = text[text.index("auto stage_rows"):]
    stage = stage[:stage.index("\n  };")]
    assert "warp == 0 && xlive" in stage and "__syncthreads_and(xlive)" in stage
    end = text[text.rindex("cluster_wait();"):]
    assert re.search(r"if \(!xlive\) mbar_wait_bounded\(xbar", end)


@pytest.mark.parametrize("name", KERNELS + ["moe_route.cuh", "fewtok.cuh"])
def test_no_read_only_loads(name):
    # every launch is a programmatic dependent: what it reads may still be
    # written while it runs, which the read-only path does not allow
    text = source(name)
    assert "__ldg(" not in text and "ld.global.nc" not in text


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def test_sizes_beyond_the_indexes_are_refused(L):
    # before any CUDA call: the plans and the kernels count in 32 bits
    lin = lambda M, rows, K: L.swiglu_mlp_w4_linear(P, P, P, M, rows, K, 128, 0, 0, P, BIG, N)
    mlp = lambda D, H: L.swiglu_mlp_fwd_nograd_w4(P, P, P, P, P, 1, D, H, 128, 0, 0, N, P, BIG, N)
    moe = lambda D, H: L.swiglu_mlp_moe_fwd_nograd(P, P, P, P, P, P, P, 64, D, H, 512, 16, 1, 1.0, N, 0,
                                                   N, P, BIG, N)
    for M in (1, 8, 32, 64):
        assert lin(M, 16, (1 << 27) + 8) == UNSUP and lin(M, 16, 1 << 30) == UNSUP
        assert lin(M, (1 << 31) - 8, 64) == UNSUP
    assert mlp((1 << 27) + 8, 64) == UNSUP and mlp(64, (1 << 27) + 8) == UNSUP
    assert moe((1 << 24) + 8, 64) == UNSUP and moe(64, (1 << 24) + 8) == UNSUP
    assert L.swiglu_mlp_w4_pack(P, P, N, P, 1, 16, (1 << 27) + 8, 128, 0, 0, N) == UNSUP
    assert L.swiglu_mlp_w4_unpack(P, P, 1, 16, (1 << 27) + 8, 128, 0, 0, 0, N) == UNSUP
    assert L.swiglu_mlp_w4_quantize(P, P, P, N, 16, (1 << 27) + 8, 128, 0, N) == UNSUP
    # the largest ones that are not are taken (there is no GPU here: not by these checks)
    assert L.swiglu_mlp_w4_packed_bytes(1, (1 << 31) - 264, 64, 128, 0, 0) > 0
    assert L.swiglu_mlp_w4_packed_bytes(1, 16, 1 << 27, 128, 0, 0) > 0
    assert L.swiglu_mlp_w4_packed_bytes(1, 16, (1 << 27) + 8, 128, 0, 0) == 0
