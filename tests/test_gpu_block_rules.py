"""Layer norm and linear layers where a call's form, rather than its formula, can
go wrong.  Tolerances as in test_gpu_block.py, whose restatements are used."""
import math

import pytest
import torch

from backward_tcgen05_tma_gb300 import api, block, build, module
from backward_tcgen05_tma_gb300.module import SwiGLUMLP
from backward_tcgen05_tma_gb300.serving import MoESwiGLU, W4SwiGLUMLP
from conftest import device_status
import test_gpu_block as base
from test_gpu_block import DT, TINY, U, act_slack, dact64, gen, normal, within

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


@pytest.fixture
def large_forms():
    """set(pairs, wide): the kernels that large sizes take, on small ones."""
    old = api.swiglu_mlp_set_cta_pairs(1), api.swiglu_mlp_set_wide_tiles(1)

    def choose(pairs, wide):
        api.swiglu_mlp_set_cta_pairs(pairs)
        api.swiglu_mlp_set_wide_tiles(wide)
    yield choose
    choose(*old)


# N a multiple of 16: outputs leave by whole sectors; rows and columns that end inside a tile
@pytest.mark.parametrize("dtn", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(65, 16, 328), (257, 272, 1032), (300, 1040, 264), (513, 2816, 1024), (2500, 528, 136)])
@pytest.mark.parametrize("wide", [0, 2])
def test_linear_on_sm_pairs_in_sectors_and_wide_tiles(large_forms, dtn, M, N, K, wide):
    large_forms(2, wide)
    if not wide:
        base.test_linear_forward(dtn, M, N, K)
    base.test_linear_backward(dtn, M, N, K)
    # dW and the bias gradient added to what is there
    g, dt = gen(M), DT[dtn]
    dY, X, W = normal(g, M, N, std=0.5, dtype=dt), normal(g, M, K, dtype=dt), normal(g, N, K, std=0.1, dtype=dt)
    hW, hb = normal(g, N, K, dtype=dt), normal(g, N, dtype=dt)
    out = {"dW": hW.clone(), "dbias": hb.clone()}
    for _ in range(2):  # (twice the same, on what the first one left)
        out["dW"].copy_(hW)
        out["dbias"].copy_(hb)
        api.swiglu_mlp_linear_bwd(dY, X, W, out=out, accumulate=True)
        y = dY.double()
        within(out["dW"], hW.double() + y.T @ X.double(), U[dtn], act_slack(M),
               (y.square().T @ X.double().square()).sqrt() + hW.double().abs())
        within(out["dbias"], hb.double() + y.sum(0), U[dtn], act_slack(M), y.square().sum(0).sqrt() + hb.double().abs())


@pytest.mark.parametrize("dtn", ["bf16", "f16"])
@pytest.mark.parametrize("pairs", [0, 2])
@pytest.mark.parametrize("M,N,K", [(9, 48, 264), (70, 272, 328), (300, 1040, 264), (2100, 528, 136)])
def test_buffers_that_start_inside_a_sector(large_forms, dtn, pairs, M, N, K):
    # 16-byte aligned, as asked for: not by whole sectors, the same arithmetic
    large_forms(pairs, 1)
    g, dt = gen(N), DT[dtn]
    X, W, b = normal(g, M, K, dtype=dt), normal(g, N, K, std=K ** -0.5, dtype=dt), normal(g, N, dtype=dt)

    def inside(t=None):
        v = torch.empty(M * N + 8, dtype=dt, device="cuda")[8:].view(M, N)
        assert v.data_ptr() % 32 == 16
        return v if t is None else v.copy_(t)
    R = normal(g, M, N, dtype=dt)
    for act, keep in (("none", False), ("gelu", True)):
        ref = api.swiglu_mlp_linear_fwd(X, W, b, act, R, keep=keep)
        for r, y, z in ((inside(R), None, None), (R, inside(), None), (R, None, inside()), (inside(R), inside(), inside())):
            got = api.swiglu_mlp_linear_fwd(X, W, b, act, r, keep=keep, out={"Y": y, "Z": z})
            assert torch.equal(got[0], ref[0]) and (not keep or torch.equal(got[1], ref[1]))


def chain(dt, M, wait, ws, seed):
    """Calls whose inputs are the outputs of those before them, each an early launch
    on the one before: all outputs that later calls read."""
    D, N, g = 264, 528, gen(seed)
    x, r = normal(g, M, D, dtype=dt), normal(g, M, D, dtype=dt)
    W1, b1, W2 = (normal(g, *s, std=0.06, dtype=dt) for s in ((N, D), (N,), (D, N)))
    w, b = normal(g, D, std=0.1, mean=1, dtype=dt), normal(g, D, dtype=dt)
    kept = []
    for _ in range(4):
        y, s, mean, rstd = wait(api.swiglu_mlp_layer_norm_fwd(x, w, b, residual=r))
        a, z = wait(api.swiglu_mlp_linear_fwd(y, W1, b1, "gelu", keep=True, ws=ws))
        r, _ = wait(api.swiglu_mlp_linear_fwd(a, W2, b, "none", s, ws=ws))
        da, dw2, db2 = wait(api.swiglu_mlp_linear_bwd(r, a, W2, X_pre=z, x_activation="gelu", ws=ws))
        dy, dw1, db1 = wait(api.swiglu_mlp_linear_bwd(da, y, W1, z, "silu", ws=ws))
        x, dw, db = wait(api.swiglu_mlp_layer_norm_bwd(dy, s, w, mean, rstd, dS=r, ws=ws))
        # the gradients are the next weights, brought to their size by a norm
        W1 = wait(api.swiglu_mlp_layer_norm_fwd(dw1, dw, db, stats=False))[0]
        W2 = wait(api.swiglu_mlp_layer_norm_fwd(dw2, db1, stats=False))[0]
        W1, W2 = (wait(api.swiglu_mlp_layer_norm_fwd(v, stats=False))[0].mul_(0.06) for v in (W1, W2))
        b = wait(api.swiglu_mlp_layer_norm_fwd(db2.view(1, D), stats=False))[0].view(D)
        kept += [y, s, mean, rstd, a, z, r, da, dw2, db2, dy, dw1, db1, x, dw, db, W1, W2, b]
        x, r = (wait(api.swiglu_mlp_layer_norm_fwd(v, stats=False))[0] for v in (x, r))
    return kept


def bits(t):
    """As whole numbers, so that what is no number compares too."""
    return t.view(torch.int32 if t.dtype is torch.float32 else torch.int16)


@pytest.mark.parametrize("dtn", list(DT))
@pytest.mark.parametrize("M", [1, 5, 40, 200, 1500])
def test_calls_in_a_row_read_what_the_one_before_wrote(large_forms, dtn, M):
    # (fp16: the weights' gradients of later rounds exceed 65504, in 64 bits in the same
    # places, and their norms are then no numbers)
    dt = DT[dtn]
    ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")

    def slowly(out):
        torch.cuda.synchronize()
        return out
    for pairs, wide in ((1, 1), (2, 2)) if dtn != "f32" and M > 64 else ((1, 1),):
        large_forms(pairs, wide)
        ref = chain(dt, M, slowly, ws, M)
        assert dtn == "f16" or all(bool(t.isfinite().all()) for t in ref)
        for _ in range(10):
            got = chain(dt, M, lambda out: out, ws, M)
            assert all(torch.equal(bits(p), bits(q)) for p, q in zip(got, ref))


@pytest.mark.parametrize("dtn", ["bf16", "f16"])
def test_debug_build_checks_the_large_forms(large_forms, dtn):
    # accesses by sectors, on pairs and on single SMs, and 512-column tiles
    M, N, K, g, dt = 1100, 272, 1032, gen(1), DT[dtn]
    X, W, b, R = (normal(g, *s, std=0.3, dtype=dt) for s in ((M, K), (N, K), (N,), (M, N)))
    for pairs in (0, 2):
        large_forms(pairs, 2)
        ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
        run = lambda: (*api.swiglu_mlp_linear_fwd(X, W, b, "gelu", R, keep=True, ws=ws),
                       *api.swiglu_mlp_linear_bwd(R, X, W, R, "gelu", X_pre=X, x_activation="silu", ws=ws))
        release = run()
        prev = api.use_debug_library(True)
        try:
            large_forms(pairs, 2)  # (the debug library keeps its own)
            debug = run()  # (raises on a failed check)
            api.lib().swiglu_mlp_debug_narrow_once(1)
            assert device_status(lambda: api.swiglu_mlp_linear_fwd(X, W, b, "gelu", R, ws=ws), ws) == 7
            large_forms(1, 1)
        finally:
            api.use_debug_library(prev)
        assert all(torch.equal(p, q) for p, q in zip(release, debug))


@pytest.mark.parametrize("dtn", list(DT))
def test_outputs_changed_in_place_have_their_gradients(dtn):
    dt, g = DT[dtn], gen(6)
    w, x = normal(g, 64, 64, std=0.2, dtype=dt).requires_grad_(), normal(g, 3, 5, 64, dtype=dt).requires_grad_()
    layers = [lambda v: block.layer_norm(v), lambda v: block.layer_norm(v, residual=v)[0],
              lambda v: block.linear(v, w, None, "gelu"), lambda v: block.mlp(v, w, None, w, None)]
    if dtn != "f32":
        pair, down = normal(g, 192, 64, std=0.2, dtype=dt), normal(g, 64, 96, std=0.2, dtype=dt)
        layers.append(lambda v: module.swiglu_mlp(v, pair, down))
    for f in layers:
        y = f(x)
        y *= 2
        got = torch.autograd.grad(y.sum(), x)[0]
        assert torch.equal(got, torch.autograd.grad((f(x) * 2).sum(), x)[0])
    # the sum is what backward reads: changing it is noticed
    y, s = block.layer_norm(x, residual=x)
    s += 1
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y.sum(), x)


@pytest.mark.parametrize("dtn", list(DT))
def test_layers_take_inputs_and_gradients_that_start_anywhere(dtn):
    dt, g, M, D = DT[dtn], gen(7), 6, 64
    w = normal(g, D, D, std=0.2, dtype=dt).requires_grad_()
    pair, down = normal(g, 192, 64, std=0.2, dtype=dt), normal(g, 64, 96, std=0.2, dtype=dt)
    a, c = normal(g, 3, dtype=dt), normal(g, 3 + M * D, dtype=dt)
    x = normal(g, 3 + M * D, dtype=dt)[3:].view(M, D)  # contiguous, inside 16 bytes
    assert x.data_ptr() % 16
    layers = [lambda v: block.layer_norm(v), lambda v: block.layer_norm(v, residual=v)[1], lambda v: block.linear(v, w, None, "gelu"),
              lambda v: block.linear(v, w, None, "none", v), lambda v: block.mlp(v, w, None, w, None),
              lambda v: sum(block.layer_norm(v, residual=v)), lambda v: module.swiglu_mlp(v, pair, down)]
    if dtn != "f32":
        with torch.no_grad():
            layers.append(W4SwiGLUMLP(SwiGLUMLP(D, 96, dtype=dt, device="cuda"), group=32))
            layers.append(MoESwiGLU(D, 64, 4, 2, dtype=dt, device="cuda"))
    for f in layers:
        with torch.no_grad():
            assert torch.equal(f(x), f(x.clone()))
        if isinstance(f, torch.nn.Module):
            continue
        grads = []
        for v in (x, x.clone()):
            v = v.detach().requires_grad_()
            # the gradient of the second part of a row of values starts behind three others
            joined = torch.cat([a, f(v).flatten()])
            grads.append(torch.autograd.grad(joined, v, c)[0])
        v = x.clone().requires_grad_()
        grads.append(torch.autograd.grad(f(v), v, c[3:].view(M, D).clone())[0])
        assert torch.equal(grads[0], grads[1]) and torch.equal(grads[1], grads[2])


@pytest.mark.parametrize("dtn", list(DT))
def test_input_gradients_without_the_input(dtn):
    g, dt = gen(8), DT[dtn]
    dY, X, W, Z = (normal(g, *s, dtype=dt) for s in ((40, 136), (40, 264), (136, 264), (40, 136)))
    dX, _, db = api.swiglu_mlp_linear_bwd(dY, X, W, Z, "gelu")
    got = api.swiglu_mlp_linear_bwd(dY, None, W, Z, "gelu", need_dW=False)
    assert torch.equal(got[0], dX) and got[1] is None and torch.equal(got[2], db)


def test_relus_slope_where_there_is_no_number():
    # 1, as its other side gives: the gradient passes
    for dt in DT.values():
        for M in (3, 300):
            z = torch.full((M, 16), float("nan"), dtype=dt, device="cuda")
            dY, W = normal(gen(1), M, 16, dtype=dt), torch.zeros(16, 8, dtype=dt, device="cuda")
            pre = torch.full((M, 8), float("nan"), dtype=dt, device="cuda")
            W[:8] = torch.eye(8)
            dZ = torch.empty_like(dY)
            dX, _, _ = api.swiglu_mlp_linear_bwd(dY, None, W, z, "relu", X_pre=pre, x_activation="relu", need_dW=False,
                                                 out={"dZ": dZ})
            assert torch.equal(dZ, dY) and torch.equal(dX, dY[:, :8])


# ---------------------------------------------------------------------------
# offsets that pass 32 bits: the last rows are what a call on them alone gives
# ---------------------------------------------------------------------------
def large(rows, columns, dt=torch.bfloat16, seed=0):
    """Rows of 2^20 different values, repeated (quickly made)."""
    n = 1 << 20
    v = normal(gen(seed), n, dtype=dt)
    return v.repeat((rows * columns + n - 1) // n + 1)[: rows * columns].view(rows, columns)


TAIL = 40


def test_norms_of_more_than_2_to_the_31_elements():
    M, D = 140_000, 16384
    x, dy = large(M, D, seed=1), large(M, D, seed=2)
    w = normal(gen(3), D, dtype=x.dtype)
    Y, S, mean, rstd = api.swiglu_mlp_layer_norm_fwd(x, w, None, residual=dy)
    dX, dw, _ = api.swiglu_mlp_layer_norm_bwd(dy, S, w, mean, rstd, dS=x, need_dbias=False)
    t = slice(M - TAIL, M)
    y2, s2, m2, r2 = api.swiglu_mlp_layer_norm_fwd(x[t], w, None, residual=dy[t])
    d2, _, _ = api.swiglu_mlp_layer_norm_bwd(dy[t], s2, w, m2, r2, dS=x[t])
    for a, b in ((Y[t], y2), (S[t], s2), (mean[t], m2), (rstd[t], r2), (dX[t], d2)):
        assert torch.equal(a, b)
    # dw, by parts of the rows
    ref, size = torch.zeros(D, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    for i in range(0, M, 4000):
        h = dy[i:i + 4000].double() * (S[i:i + 4000].double() - mean[i:i + 4000, None]) * rstd[i:i + 4000, None]
        ref += h.sum(0)
        size += h.square().sum(0)
    within(dw, ref, U["bf16"], 4 * math.sqrt(M) * 2.0 ** -24 + 2.0 ** -20, size.sqrt())


@pytest.mark.parametrize("dtn", ["bf16", "f32"])
def test_outputs_of_more_than_2_to_the_31_elements(dtn):
    M, N, K, dt = 600_000, 4096, 64, DT[dtn]
    X, W, b = large(M, K, dt), normal(gen(1), N, K, std=0.1, dtype=dt), normal(gen(2), N, dtype=dt)
    Y, Z = api.swiglu_mlp_linear_fwd(X, W, b, "silu", keep=True)
    assert Y.numel() > 2 ** 31
    t = slice(M - 1200, M)  # (as many as take the same kernel)
    y2, z2 = api.swiglu_mlp_linear_fwd(X[t], W, b, "silu", keep=True)
    assert torch.equal(Y[t], y2) and torch.equal(Z[t], z2)
    dZ = torch.empty_like(Y)
    dX, _, db = api.swiglu_mlp_linear_bwd(Y, X, W, Z, "silu", need_dW=False, out={"dZ": dZ})
    e2 = torch.empty_like(y2)
    d2, _, _ = api.swiglu_mlp_linear_bwd(y2, X[t], W, z2, "silu", need_dW=False, out={"dZ": e2})
    assert torch.equal(dZ[t], e2)
    u, n = U[dtn], act_slack(N)
    ref = e2.double() @ W.double()
    within(dX[t], ref, u, n, (e2.double().square() @ W.double().square()).sqrt())
    # db: the rows come again and again, so the terms of a column add up and their
    # roundings do not go like a random walk.  A warp adds every eighth row of a part
    # one after another (4096 columns: 32 strips of fp32, 19 parts, 3948 rows; 16 strips
    # of bf16, 38 parts, 1974 rows), each sum rounded by up to 2^-24 of itself, which is
    # at most the sum of all absolute values; a slope is off by up to 2^-18 of |Y|
    ref, size = torch.zeros(N, dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
    for i in range(0, M, 20_000):
        v = Y[i:i + 20_000].double() * dact64("silu", Z[i:i + 20_000].double())
        ref += v.sum(0)
        size += v.abs().sum(0) + 2.0 ** -18 / (4100 * 2.0 ** -24) * Y[i:i + 20_000].double().abs().sum(0)
    within(db, ref, u, 4100 * 2.0 ** -24, size)


@pytest.mark.parametrize("dtn,M", [("bf16", 1), ("f16", 16), ("bf16", 64), ("bf16", 200), ("f32", 1), ("f32", 8), ("f32", 40)])
def test_weights_of_more_than_2_to_the_31_elements(dtn, M):
    N, K, dt = 300_000, 8192, DT[dtn]
    X, W = normal(gen(M), M, K, dtype=dt), large(N, K, dt)
    Y, _ = api.swiglu_mlp_linear_fwd(X, W)
    for t in (slice(0, 64), slice(N - 64, N)):
        x, w = X.double(), W[t].double()
        within(Y[:, t], x @ w.T, U[dtn], act_slack(K), (x.square() @ w.square().T).sqrt())
