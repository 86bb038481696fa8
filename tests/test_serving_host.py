"""Host-side checks of the few-token serving operators (no GPU): sizes, and
the refusals of the C entry points and of the binding, which come before any
CUDA call."""
import ctypes

import pytest
import torch

from backward_tcgen05_tma_gb300 import api, build
from backward_tcgen05_tma_gb300.serving import MoESwiGLU, W4SwiGLUMLP

OK, INVALID, ALIGN, UNSUP, WSERR = 0, 1, 2, 3, 4
P = ctypes.c_void_p(0x10000)  # an aligned fake device address (never dereferenced)
P_MIS = ctypes.c_void_p(0x10008)
N = ctypes.c_void_p(0)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


@pytest.mark.parametrize("group,zeros,record", [(128, 0, 544), (64, 0, 544), (32, 0, 576),
                                                (128, 1, 560), (32, 1, 608)])
def test_packed_sizes(L, group, zeros, record):
    f = L.swiglu_mlp_w4_packed_bytes
    assert f(1, 16, 64, group, zeros, 0) == record
    assert f(1, 17, 72, group, zeros, 0) == 2 * 2 * record      # ragged rows and columns
    assert f(1, 32, 64, group, zeros, 1) == 2 * record          # gate/up: tiles of 8 hidden units
    assert f(3, 4096, 11008, group, zeros, 0) == 3 * 256 * 172 * record
    assert f(1, 16, 60, group, zeros, 0) == 0 and f(0, 16, 64, group, zeros, 0) == 0
    assert f(1, 17, 64, group, zeros, 1) == 0 and f(1, 16, 64, 48, zeros, 0) == 0
    assert f(1, 16, 64, group, 2, 0) == 0


def test_workspace_sizes(L):
    assert L.swiglu_mlp_w4_workspace_bytes(1, 4096, 4096) >= 256
    assert L.swiglu_mlp_fwd_nograd_w4_workspace_bytes(64, 4096, 11008) >= 256
    # the assignments' hidden values
    assert L.swiglu_mlp_moe_workspace_bytes(64, 2048, 1024, 64, 8) >= 256 + 64 * 8 * 1024 * 2
    assert L.swiglu_mlp_moe_workspace_bytes(-1, 2048, 1024, 64, 8) == 0


def _linear(L, X=P, W=P, Y=P, M=4, Nn=24, K=64, group=64, zeros=0, dt=0, ws=P, wsb=BIG):
    return L.swiglu_mlp_w4_linear(X, W, Y, M, Nn, K, group, zeros, dt, ws, wsb, N)


def test_w4_linear_refuses(L):
    assert _linear(L, X=N) == INVALID and _linear(L, Y=N) == INVALID and _linear(L, W=N) == INVALID
    assert _linear(L, W=P_MIS) == ALIGN and _linear(L, ws=P_MIS) == ALIGN
    assert _linear(L, M=-1) == INVALID and _linear(L, Nn=0) == INVALID and _linear(L, K=0) == INVALID
    assert _linear(L, K=60) == ALIGN
    assert _linear(L, group=48) == INVALID and _linear(L, zeros=2) == INVALID
    assert _linear(L, dt=2) == UNSUP and _linear(L, M=65) == UNSUP
    assert _linear(L, ws=N) == WSERR and _linear(L, wsb=8) == WSERR
    assert _linear(L, M=0) == OK and L.swiglu_mlp_last_launch_count() == 0


def _mlp(L, X=P, Wgu=P, Wd=P, Y=P, A=P, M=4, D=64, H=128, group=64, zeros=0, dt=0, o=N, ws=P,
         wsb=BIG):
    return L.swiglu_mlp_fwd_nograd_w4(X, Wgu, Wd, Y, A, M, D, H, group, zeros, dt, o, ws, wsb, N)


def test_w4_mlp_refuses(L):
    for k in ("X", "Wgu", "Wd", "Y", "A"):
        assert _mlp(L, **{k: N}) == INVALID and _mlp(L, **{k: P_MIS}) == ALIGN
    assert _mlp(L, D=60) == ALIGN and _mlp(L, H=60) == ALIGN
    assert _mlp(L, M=65) == UNSUP and _mlp(L, dt=2) == UNSUP
    assert _mlp(L, group=0) == INVALID and _mlp(L, wsb=100) == WSERR
    nan, acc = api.Options(float("nan"), 1.0, 0), api.Options(1.0, 1.0, 1)
    assert _mlp(L, o=ctypes.byref(nan)) == INVALID and _mlp(L, o=ctypes.byref(acc)) == INVALID
    assert _mlp(L, M=0) == OK and L.swiglu_mlp_last_launch_count() == 0


def test_w4_layout_calls_refuse(L):
    q, p, u = L.swiglu_mlp_w4_quantize, L.swiglu_mlp_w4_pack, L.swiglu_mlp_w4_unpack
    assert q(N, P, P, N, 16, 64, 64, 0, N) == INVALID and q(P, P, P, P_MIS, 16, 64, 64, 0, N) == ALIGN
    assert q(P, P, P, N, 16, 60, 64, 0, N) == ALIGN and q(P, P, P, N, 16, 64, 64, 2, N) == UNSUP
    assert p(P, P, N, N, 1, 16, 64, 64, 0, 0, N) == INVALID
    assert p(P, P, N, P, 1, 24, 64, 64, 1, 0, N) == ALIGN  # gate/up: H a multiple of 8
    assert p(P, P, N, P, 0, 16, 64, 64, 0, 0, N) == INVALID
    assert u(P, N, 1, 16, 64, 64, 0, 0, 0, N) == INVALID and u(P, P, 1, 16, 64, 65, 0, 0, 0, N) == INVALID


def _moe(L, X=P, Wr=P, Wgu=P, Wd=P, Y=P, idx=P, w=P, T=4, D=64, H=128, E=8, k=2, norm=1, scale=1.0,
         f=N, dt=0, o=N, ws=P, wsb=BIG):
    return L.swiglu_mlp_moe_fwd_nograd(X, Wr, Wgu, Wd, Y, idx, w, T, D, H, E, k, norm, scale, f, dt,
                                       o, ws, wsb, N)


def test_moe_refuses(L):
    for n in ("X", "Wr", "Wgu", "Wd", "Y", "idx", "w"):
        assert _moe(L, **{n: N}) == INVALID and _moe(L, **{n: P_MIS}) == ALIGN
    assert _moe(L, T=-1) == INVALID and _moe(L, k=0) == INVALID and _moe(L, k=9) == INVALID
    assert _moe(L, E=0) == INVALID and _moe(L, norm=2) == INVALID
    assert _moe(L, scale=float("inf")) == INVALID and _moe(L, dt=7) == INVALID
    assert _moe(L, D=60) == ALIGN and _moe(L, H=4) == ALIGN
    assert _moe(L, T=65) == UNSUP and _moe(L, E=513) == UNSUP and _moe(L, E=64, k=17) == UNSUP
    assert _moe(L, dt=2) == UNSUP
    bad = api.W4Format(16, 0)
    assert _moe(L, f=ctypes.byref(bad)) == INVALID
    need = L.swiglu_mlp_moe_workspace_bytes(4, 64, 128, 8, 2)
    assert _moe(L, wsb=need - 1) == WSERR and _moe(L, ws=N) == WSERR
    assert _moe(L, T=0) == OK and L.swiglu_mlp_last_launch_count() == 0
    r, e = L.swiglu_mlp_moe_route, L.swiglu_mlp_moe_experts
    assert r(P, N, P, P, 4, 64, 8, 2, 1, 1.0, 0, N) == INVALID
    assert r(P, P, P, P, 4, 64, 8, 2, 3, 1.0, 0, N) == INVALID
    assert r(P, P, P, P, 0, 64, 8, 2, 1, 1.0, 0, N) == OK
    assert e(P, N, P, P, P, P, 4, 64, 128, 8, 2, N, 0, N, P, BIG, N) == INVALID
    assert e(P, P, P, P, P, P, 4, 64, 128, 8, 2, N, 0, N, P, 100, N) == WSERR


def test_binding_refuses_cpu_tensors_and_mismatches():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = api.W4Weights(torch.zeros(16, dtype=torch.uint8), 16, 64, 64, False, False, torch.bfloat16)
    gu = api.W4Weights(torch.zeros(16, dtype=torch.uint8), 32, 64, 64, False, True, torch.bfloat16)
    with pytest.raises(ValueError):
        api.swiglu_mlp_w4_linear(x, w)                      # not on a GPU
    with pytest.raises(ValueError):
        api.swiglu_mlp_w4_linear(x, gu)                     # a gate/up pair
    with pytest.raises(ValueError):
        api.swiglu_mlp_w4_linear(x.half(), w)               # scales of another type
    with pytest.raises(ValueError):
        api.swiglu_mlp_w4_linear(x[:, :32], w)              # another K
    with pytest.raises(ValueError):
        api.swiglu_mlp_fwd_nograd_w4(x, gu, w)              # [32, 64] pair with [16, 64]
    with pytest.raises(ValueError):
        api.swiglu_mlp_moe_fwd_nograd(x, x, gu, torch.zeros(1, 64, 16), 1)  # formats mixed
    with pytest.raises(ValueError):
        api.swiglu_mlp_moe_fwd_nograd(x, torch.zeros(3, 64, dtype=x.dtype),
                                      torch.zeros(2, 32, 64, dtype=x.dtype),
                                      torch.zeros(2, 64, 16, dtype=x.dtype), 1)  # Wr of 3 experts
    with pytest.raises(ValueError):
        api.swiglu_mlp_moe_experts(x, torch.zeros(4, 1), torch.zeros(4, 1),
                                   torch.zeros(2, 32, 64, dtype=x.dtype),
                                   torch.zeros(2, 64, 16, dtype=x.dtype))  # idx not int32


def test_modules_on_the_host():
    m = MoESwiGLU(64, 32, 4, 2, dtype=torch.float16)
    assert m.router_weight.shape == (4, 64) and m.gate_up_weight.shape == (4, 64, 64)
    assert m.down_weight.shape == (4, 64, 32) and not m.down_weight.requires_grad
    assert set(m.state_dict()) == {"router_weight", "gate_up_weight", "down_weight"}
    x = torch.zeros(1, 64, requires_grad=True)
    for module in (m, W4SwiGLUMLP()):
        with pytest.raises(RuntimeError, match="no backward"):
            module(x)
