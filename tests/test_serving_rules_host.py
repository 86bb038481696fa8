"""Rules of the few-token serving operators that need no GPU to be checked: the
order of synchronisation in the kernels' sources, launch plans, size limits,
and the state of the modules."""
import copy
import ctypes
import io
import os
import re
import subprocess
import sys

import pytest
import torch

from backward_tcgen05_tma_gb300 import api, build
from backward_tcgen05_tma_gb300.serving import MoESwiGLU, PackedW4, W4SwiGLUMLP

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


def test_packed_bytes_of_what_packing_refuses(L):
    for n in (8, 24, 40):  # a pair's H is a multiple of 8
        assert L.swiglu_mlp_w4_pack(P, P, N, P, 1, n, 64, 64, 1, 0, N) == 2
        assert L.swiglu_mlp_w4_packed_bytes(1, n, 64, 64, 0, 1) == 0
    assert L.swiglu_mlp_w4_packed_bytes(1, 48, 64, 64, 0, 1) == 3 * 544


def test_no_type_is_an_invalid_argument(L):
    # fp32 is a type that these calls do not support; 7 is none
    for dt, status in ((2, UNSUP), (7, 1)):
        assert L.swiglu_mlp_w4_linear(P, P, P, 4, 16, 64, 64, 0, dt, P, BIG, N) == status
        assert L.swiglu_mlp_fwd_nograd_w4(P, P, P, P, P, 4, 64, 64, 64, 0, dt, N, P, BIG, N) == status
        assert L.swiglu_mlp_w4_quantize(P, P, P, N, 16, 64, 64, dt, N) == status
        assert L.swiglu_mlp_w4_pack(P, P, N, P, 1, 16, 64, 64, 0, dt, N) == status
        assert L.swiglu_mlp_w4_unpack(P, P, 1, 16, 64, 64, 0, 0, dt, N) == status
        assert L.swiglu_mlp_moe_route(P, P, P, P, 4, 64, 8, 2, 1, 1.0, dt, N) == status


# ---------------------------------------------------------------------------
# modules: quantised weights are state
# ---------------------------------------------------------------------------
def w4(seed, n, k, pair, experts=None, group=64, zeros=True):
    """Packed weights of random bytes (nothing on the host reads them)."""
    n_bytes = api.lib().swiglu_mlp_w4_packed_bytes(experts or 1, n, k, group, int(zeros), int(pair))
    g = torch.Generator().manual_seed(seed)
    packed = torch.randint(0, 256, (n_bytes,), dtype=torch.uint8, generator=g)
    return api.W4Weights(packed, n, k, group, zeros, pair, torch.float16, experts)


def through_a_file(state):
    f = io.BytesIO()
    torch.save(state, f)
    f.seek(0)
    return torch.load(f, weights_only=True)


def alike(a, b):
    keys = ("N", "K", "group", "zeros", "gate_up", "experts", "dtype", "shape")
    return all(getattr(a, k) == getattr(b, k) for k in keys) and torch.equal(a.packed, b.packed)


@pytest.fixture
def quantized(L):
    """A 4-bit MLP and a mixture with 4-bit experts, as quantising leaves them."""
    mlp = W4SwiGLUMLP()
    mlp.gate_up_w4, mlp.down_w4 = PackedW4(w4(1, 32, 72, True)), PackedW4(w4(2, 72, 16, False))
    mlp.gate_multiplier, mlp.down_multiplier = 0.3, 1.7
    moe = MoESwiGLU(72, 16, 4, 2, dtype=torch.float16)
    moe._experts_w4(PackedW4(w4(3, 32, 72, True, 4)), PackedW4(w4(4, 72, 16, False, 4)))
    return mlp, moe


def test_quantized_modules_keep_their_weights_in_their_state(quantized):
    mlp, moe = quantized
    new_mlp, new_moe = W4SwiGLUMLP(), MoESwiGLU(72, 16, 4, 2, dtype=torch.float16)
    new_mlp.load_state_dict(through_a_file(mlp.state_dict()))
    assert alike(new_mlp.gate_up, mlp.gate_up) and alike(new_mlp.down, mlp.down)
    assert (new_mlp.gate_multiplier, new_mlp.down_multiplier) == (0.3, 1.7)
    new_moe.load_state_dict(through_a_file(moe.state_dict()))  # replaces the 16-bit experts
    assert new_moe.gate_up_weight is None and torch.equal(new_moe.router_weight, moe.router_weight)
    for name in ("gate_up_w4", "down_w4"):
        assert alike(getattr(new_moe, name).weights, getattr(moe, name).weights)
        assert getattr(new_moe, name).packed is not getattr(moe, name).packed
    # and again, into modules that hold other 4-bit weights, as parts of a model
    other = copy.deepcopy(moe)
    other.gate_up_w4 = PackedW4(w4(5, 32, 72, True, 4, group=32, zeros=False))
    model = torch.nn.Sequential(other, W4SwiGLUMLP())
    model.load_state_dict(through_a_file(torch.nn.Sequential(moe, mlp).state_dict()))
    assert alike(other.gate_up_w4.weights, moe.gate_up_w4.weights) and alike(model[1].down, mlp.down)


def test_quantized_modules_refuse_a_state_without_the_weights(quantized):
    mlp, moe = quantized
    with pytest.raises(RuntimeError, match="gate_up_w4.packed"):
        moe.load_state_dict(MoESwiGLU(72, 16, 4, 2, dtype=torch.float16).state_dict())
    with pytest.raises(RuntimeError, match="router_weight"):
        MoESwiGLU(72, 16, 4, 2, dtype=torch.float16).load_state_dict(
            {k: v for k, v in moe.state_dict().items() if k != "router_weight"})
    with pytest.raises(RuntimeError, match="no 4-bit weights"):
        W4SwiGLUMLP().gate_up


def test_quantized_modules_move_with_their_weights(quantized):
    for m in quantized:
        moved = copy.deepcopy(m).to("meta")
        assert moved.gate_up_w4.packed.is_meta and moved.down_w4.weights.device.type == "meta"
        assert moved.gate_up_w4.weights.shape == m.gate_up_w4.weights.shape
        cast = copy.deepcopy(m).to(torch.bfloat16)  # the bytes are no numbers of the module's type
        assert alike(cast.gate_up_w4.weights, m.gate_up_w4.weights)


def test_modules_before_quantizing_have_their_old_state(L):
    m = MoESwiGLU(64, 32, 4, 2, dtype=torch.float16)
    assert set(m.state_dict()) == {"router_weight", "gate_up_weight", "down_weight"}
    n = MoESwiGLU(64, 32, 4, 2, dtype=torch.float16)
    n.load_state_dict(m.state_dict())
    assert torch.equal(n.down_weight, m.down_weight)


def test_the_binding_imports_on_a_torch_without_cuda():
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
            "    del torch._C._cuda_getCurrentRawStream\n"
            "from backward_tcgen05_tma_gb300 import api, serving\n"
            "try:\n"
            "    api.swiglu_mlp_w4_quantize(torch.zeros(16, 64, dtype=torch.bfloat16))\n"
            "except ValueError:\n"
            "    print('refused')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=build.ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr


PLANS = r"""
#include <cstdio>
#include <initializer_list>
#include "experts_plan.h"
int main() {
  using namespace swiglu;
  // warps and stage bytes of the experts kernels: 16-bit (2 units of 2 KB), 4-bit (8 or 4 records)
  struct { int warps, nt, stage; } f[] = {{16, 1, 4096}, {16, 2, 4096}, {12, 1, 8 * 608}, {12, 2, 4 * 608},
                                          {12, 1, 8 * 544}, {12, 2, 4 * 544}};
  for (auto k : f)
    for (int combine = 0; combine < 2; ++combine)
      for (int M = 1; M <= 64; ++M)
        for (int E : {1, 2, 8, 27, 64, 128, 130, 512})
          for (int topk = 1; topk <= 16 && topk <= E; ++topk)
            for (int most : {1, 7, 1000000}) {
              const WxPlan p = wx_plan(k.warps, k.nt, k.stage, combine, M, topk, E, most);
              const int used = p.ring_off + 1024 + p.stages * k.warps * k.stage;
              if (p.stages < 2 || p.stages > WX_MAX_STAGES || used > p.bytes || p.bytes > WX_SMEM_MOST ||
                  p.ring_off % 16 != 0 || (p.stages > 2 && p.bytes > WX_SMEM + 1024)) {
                printf("warps %d nt %d combine %d M %d E %d topk %d: %d stages, %d bytes\n", k.warps, k.nt,
                       combine, M, E, topk, p.stages, p.bytes);
                return 1;
              }
            }
  return 0;
}
"""


def test_experts_rings_fetch_ahead_at_every_size(tmp_path):
    # a ring of one stage fetches nothing while its stage is in use
    (tmp_path / "plans.cpp").write_text(PLANS)
    exe = str(tmp_path / "plans")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC_SERVING, "-o", exe,
                    str(tmp_path / "plans.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
