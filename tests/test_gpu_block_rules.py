"""Layer norm and linear layers where a call's form, rather than its formula, can
go wrong.  Tolerances as in test_gpu_block.py, whose restatements are used."""
import math

import pytest
import torch

from backward_tcgen05_tma_gb300 import api, block, build
from backward_tcgen05_tma_gb300.module import SwiGLUMLP
from backward_tcgen05_tma_gb300.serving import MoESwiGLU, W4SwiGLUMLP
from test_gpu_block import DT, TINY, U, dact64, gen, normal, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    api.lib()


@pytest.mark.parametrize("dtn", list(DT))
@pytest.mark.parametrize("N,K", [(2816, 1024), (1024, 2816), (520, 12000), (8, 2048)])
def test_an_empty_batch_of_wide_layers(dtn, N, K):
    # sizes whose plans share tiles: there is none to share here
    dt, g = DT[dtn], gen(N)
    for op in (api.SWIGLU_OP_FWD, api.SWIGLU_OP_BWD):
        assert api.linear_workspace(0, N, K, dt, op, "cuda").numel() >= 1280
    X, dY, W = (torch.empty(0, K, dtype=dt, device="cuda"), torch.empty(0, N, dtype=dt, device="cuda"),
                normal(g, N, K, dtype=dt))
    b = normal(g, N, dtype=dt)
    assert api.swiglu_mlp_linear_fwd(X, W, b, "gelu")[0].shape == (0, N)
    dX, dW, db = api.swiglu_mlp_linear_bwd(dY, X, W, dY, "gelu", X_pre=X, x_activation="silu")
    assert dX.shape == (0, K) and dW.shape == (N, K) and not dW.any() and not db.any()
    held = {"dW": W.clone(), "dbias": b.clone()}
    api.swiglu_mlp_linear_bwd(dY, X, W, out=held, accumulate=True)
    assert torch.equal(held["dW"], W) and torch.equal(held["dbias"], b)
    x = torch.empty(2, 0, K, dtype=dt, device="cuda", requires_grad=True)
    m = block.MLPBlock(block.MLP(K, N, dtype=dt, device="cuda"))
    m(x).sum().backward()
    assert x.grad.shape == x.shape and all(not p.grad.any() for p in m.parameters())
    w = W.clone().requires_grad_()
    block.linear(x, w, None, "relu").sum().backward()
    assert not w.grad.any()


@pytest.mark.parametrize("dtn", ["bf16", "f16"])
def test_sublayers_of_serving_modules_go_by_their_weights(dtn):
    # without a word on type, place or size
    dt, D = DT[dtn], 256
    torch.manual_seed(1)
    with torch.no_grad():
        x = normal(gen(1), 5, D, dtype=dt)
        for mlp in (W4SwiGLUMLP(SwiGLUMLP(D, 704, dtype=dt, device="cuda"), group=64),
                    MoESwiGLU(D, 128, 8, 2, dtype=dt, device="cuda")):
            m = block.MLPBlock(mlp)
            assert torch.equal(m(x), x + mlp(block.layer_norm(x)))


@pytest.mark.parametrize("dtn", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 40, 130])
def test_gelu_keeps_its_digits_far_left(dtn, M):
    # Every 16-bit value as z, exactly (X is one-hot).  Phi's error relative to
    # itself: its fit 8e-6 up to |z| = 6 and 8e-4 beyond; z^2 / 2, rounded twice,
    # 18 * 2^-23 = 2.1e-6 there (87 * 2^-23 = 1.0e-5 at most beyond); 2^-20 for the
    # exponential, the reciprocal and seven operations: 1.2e-5 < 2^-16 and 8.3e-4 <
    # 2^-10.  Exponentials below 2^-126 become 0: 13.3 * 2^-126.  fp16's steps below
    # 2^-14 are absolute.  The slope adds z phi(z), which has the exponential's error.
    dt = DT[dtn]
    v = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(dt)
    v = v[v.isfinite() & (v <= 0) & (v >= -20)]
    v = v[: v.numel() // 8 * 8].clone()
    N = v.numel()
    z = v.double()
    phi = 0.5 * torch.erfc(-z / math.sqrt(2))
    bell = z.abs() * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    rel = torch.where(z >= -6, 2.0 ** -16, 2.0 ** -10)
    least = TINY[dtn] + 2.0 ** -122
    W = torch.zeros(N, 8, dtype=dt, device="cuda")
    W[:, 0] = v
    X = torch.zeros(M, 8, dtype=dt, device="cuda")
    X[:, 0] = 1
    Y, Z = api.swiglu_mlp_linear_fwd(X, W, None, "gelu", keep=True)
    assert torch.equal(Z, v.expand(M, N))
    within(Y[M - 1], z * phi, U[dtn], 1.0, rel * (z * phi).abs() + least)
    dZ = torch.empty(M, N, dtype=dt, device="cuda")
    api.swiglu_mlp_linear_bwd(torch.ones_like(dZ), X, W, Z, "gelu", need_dX=False, need_dW=False, out={"dZ": dZ})
    within(dZ[M - 1], dact64("gelu", z), U[dtn], 1.0, rel * (phi + bell) + least)
