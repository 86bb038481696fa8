"""Host side of the layer norm and the linear layers: argument errors before any
launch, sizes, modules' state.  No GPU needed."""
import ctypes
import os
import re

import pytest
import torch

from backward_tcgen05_tma_gb300 import api, block, build

OK, INVALID, ALIGN, UNSUP, WSERR = 0, 1, 2, 3, 4
P = ctypes.c_void_p(0x10000)  # an aligned fake device address (never dereferenced)
MIS = ctypes.c_void_p(0x10008)
N = ctypes.c_void_p(0)
BIG = 1 << 40
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def ln_fwd(L, X=P, R=N, w=P, b=P, S=N, Y=P, mean=P, rstd=P, M=4, D=64, eps=1e-5, dt=0, ws=N, n=0):
    return L.swiglu_mlp_layer_norm_fwd(X, R, w, b, S, Y, mean, rstd, M, D, eps, dt, ws, n, N)


def ln_bwd(L, dY=P, S=P, w=P, mean=P, rstd=P, dS=N, dX=P, dw=P, db=P, M=4, D=64, acc=0, dt=0, ws=P, n=BIG):
    return L.swiglu_mlp_layer_norm_bwd(dY, S, w, mean, rstd, dS, dX, dw, db, M, D, acc, dt, ws, n, N)


def lin_fwd(L, X=P, W=P, b=P, R=N, Z=N, Y=P, M=4, n=64, k=128, act=0, dt=0, ws=P, nb=BIG):
    return L.swiglu_mlp_linear_fwd(X, W, b, R, Z, Y, M, n, k, act, dt, ws, nb, N)


def lin_bwd(L, dY=P, X=P, W=P, Z=N, act=0, pre=N, xact=0, dZ=N, dX=P, dW=P, db=P, M=4, n=64, k=128, acc=0, dt=0,
            ws=P, nb=BIG):
    return L.swiglu_mlp_linear_bwd(dY, X, W, Z, act, pre, xact, dZ, dX, dW, db, M, n, k, acc, dt, ws, nb, N)


def test_layer_norm_refusals(L):
    for f, need, opt in ((ln_fwd, ("X", "Y"), ("R", "w", "b", "S", "mean", "rstd")),
                         (ln_bwd, ("dY", "S", "mean", "rstd", "dX"), ("w", "dS", "dw", "db"))):
        for name in need:
            assert f(L, **{name: N}) == INVALID
            assert f(L, **{name: MIS}) == ALIGN
        for name in opt:
            assert f(L, **{name: MIS, **({"S": P} if name == "R" else {"R": P} if name == "S" and f is ln_fwd else {})}) == ALIGN
        assert f(L, M=-1) == INVALID and f(L, D=0) == INVALID and f(L, dt=7) == INVALID
        assert f(L, D=60) == ALIGN and f(L, D=62, dt=2) == ALIGN
        assert f(L, D=16392) == UNSUP and f(L, D=16388, dt=2) == UNSUP and f(L, M=2 ** 31) == UNSUP
        assert f(L, M=2 ** 31 - 256) == UNSUP
    # a residual needs a place for the sum, and none else
    assert ln_fwd(L, R=P) == INVALID and ln_fwd(L, S=P) == INVALID
    for eps in (-1e-5, NAN, float("inf")):
        assert ln_fwd(L, eps=eps) == INVALID
    assert ln_fwd(L, ws=P, n=255) == WSERR and ln_fwd(L, ws=MIS, n=256) == ALIGN
    assert ln_bwd(L, acc=2) == INVALID and ln_bwd(L, ws=N) == WSERR and ln_bwd(L, ws=MIS) == ALIGN
    need = L.swiglu_mlp_layer_norm_workspace_bytes(4, 64, 0)
    assert need > 256 and ln_bwd(L, n=need - 1) == WSERR
    assert L.swiglu_mlp_layer_norm_workspace_bytes(4, 60, 0) == 0
    assert L.swiglu_mlp_layer_norm_workspace_bytes(4, 64, 9) == 0
    assert ln_fwd(L, M=0) == OK and L.swiglu_mlp_last_launch_count() == 0
    assert ln_bwd(L, M=0, dw=N, db=N) == OK and L.swiglu_mlp_last_launch_count() == 0


def test_linear_refusals(L):
    for f, need, opt in ((lin_fwd, ("X", "W", "Y"), ("b", "R", "Z")),
                         (lin_bwd, ("dY", "X", "W"), ("Z", "pre", "dZ", "dX", "dW", "db"))):
        for name in need:
            assert f(L, **{name: N}) == INVALID
            assert f(L, **{name: MIS}) == ALIGN
        for name in opt:
            assert f(L, **{name: MIS}) == ALIGN
        assert f(L, M=-1) == INVALID and f(L, n=0) == INVALID and f(L, k=-8) == INVALID
        assert f(L, dt=3) == INVALID and f(L, act=5) == INVALID and f(L, act=-1) == INVALID
        assert f(L, n=60) == ALIGN and f(L, k=60) == ALIGN and f(L, n=62, dt=2) == ALIGN
        assert f(L, M=2 ** 31) == UNSUP and f(L, n=2 ** 31) == UNSUP and f(L, k=2 ** 31) == UNSUP
        assert f(L, M=2 ** 30, n=2 ** 20) == UNSUP  # tiles beyond 32 bits
        assert f(L, ws=N) == WSERR and f(L, ws=MIS) == ALIGN and f(L, nb=256) == WSERR
    for op in (0, 2):
        for dt in (0, 1, 2):
            for M in (1, 64, 65, 4096):
                need = L.swiglu_mlp_linear_workspace_bytes(M, 512, 256, dt, op)
                assert need >= 1280
                f = lin_fwd if op == 0 else lin_bwd
                assert f(L, M=M, n=512, k=256, dt=dt, nb=need - 1) == WSERR
    assert L.swiglu_mlp_linear_workspace_bytes(4, 64, 64, 0, 1) == 0
    assert L.swiglu_mlp_linear_workspace_bytes(4, 60, 64, 0, 0) == 0
    # an activation needs what its derivative is taken at
    assert lin_bwd(L, act=1) == INVALID and lin_bwd(L, act=1, Z=P) == INVALID and lin_bwd(L, act=1, dZ=P) == INVALID
    assert lin_bwd(L, xact=2) == INVALID and lin_bwd(L, xact=9) == INVALID and lin_bwd(L, acc=3) == INVALID
    assert lin_fwd(L, M=0) == OK and L.swiglu_mlp_last_launch_count() == 0
    assert lin_bwd(L, M=0, dW=N, db=N) == OK and L.swiglu_mlp_last_launch_count() == 0


def test_header_and_binding_name_the_activations_alike(L):
    with open(api.HEADER_PATH) as f:
        found = dict(re.findall(r"SWIGLU_ACT_(\w+) = (\d)", f.read()))
    assert {k.lower(): int(v) for k, v in found.items()} == api.ACTIVATIONS
    with pytest.raises(ValueError):
        api.activation_code("tanh")
    assert set(block.HIDDEN_ACTS.values()) <= set(api.ACTIVATIONS)


def test_kernels_wait_before_they_read():
    # every launch is a programmatic dependent: nothing is read before the wait,
    # and not through the read-only path
    for name, kernels in (("layer_norm.cuh", 2), ("column_sums.cuh", 2)):
        with open(os.path.join(build.CSRC_BLOCK, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        assert "__ldg(" not in text and "ld.global.nc" not in text and "__restrict__" not in text
        bodies = text.split("__global__")[1:]
        assert len(bodies) == kernels
        for b in bodies:
            head = b[b.index("{"):b.index("pdl_wait();")]
            assert "a.x" not in head and "ld_stream" not in head and "cp16" not in head


def test_cpu_tensors_and_shapes_are_refused_by_the_binding():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.swiglu_mlp_layer_norm_fwd(x)
    with pytest.raises(ValueError):
        api.swiglu_mlp_linear_fwd(x, w)
    with pytest.raises(ValueError):
        block.linear(x[:, :32], w)
    with pytest.raises(ValueError):
        block.linear(x, w, residual=x)
    with pytest.raises(ValueError):
        block.layer_norm(x, residual=x[:2])
    with pytest.raises(ValueError):
        block.LayerNorm(32)(x)
    with pytest.raises(ValueError):
        block.mlp(x, w, None, w.T.contiguous(), None, "tanh")


def test_modules_load_other_blocks_state():
    ref = torch.nn.LayerNorm(64)
    torch.nn.init.normal_(ref.weight)
    m = block.LayerNorm(64, dtype=torch.float32)
    m.load_state_dict(ref.state_dict())
    assert torch.equal(m.weight, ref.weight) and m.eps == ref.eps
    for names in (("fc1", "fc2"), ("up_proj", "down_proj")):
        lins = torch.nn.Linear(64, 96), torch.nn.Linear(96, 64)
        state = {"%s.%s" % (n, p): getattr(l, p) for n, l in zip(names, lins) for p in ("weight", "bias")}
        m = block.MLP(64, 96, dtype=torch.float32)
        m.load_state_dict(state)
        assert torch.equal(m.up_weight, lins[0].weight) and torch.equal(m.down_bias, lins[1].bias)
        b = block.MLPBlock(block.MLP(64, 96, dtype=torch.float32))
        assert b.norm.weight.dtype == torch.float32
        b.load_state_dict({"norm.weight": ref.weight, "norm.bias": ref.bias,
                           **{"mlp." + k: v for k, v in state.items()}})
        assert torch.equal(b.mlp.down_weight, lins[1].weight)

    class Config:
        hidden_size, intermediate_size, hidden_act = 64, 96, "gelu_new"
    assert block.MLP(Config).activation == "gelu_tanh" and block.MLP(Config, activation="relu").activation == "relu"
    assert block.MLP(64, 96, bias=False).up_bias is None
    with pytest.raises(ValueError):
        block.MLP(64, 96, activation="tanh")
