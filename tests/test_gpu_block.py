"""Layer norm and linear layers against restatements of their definitions in 64
bits, their gradients against the formulas and against differences.

Tolerances, fixed before any run.  u: half a step of the storage type (2^-8 bf16,
2^-11 fp16, 2^-24 fp32), the largest relative error of the one rounding of an
output.  What comes before it is fp32:
 * a sum of n terms in any order is within n 2^-24 of the sum of their absolute
   values, and no order here adds more than a few hundred terms in a row per
   partial sum of products (products: K in blocks through the tensor core or
   one FMA at a time); its errors add like a random walk, so a slack of
   4 sqrt(n) 2^-24, relative to the root of the sum of squares of the terms,
   covers all but one element in thousands of millions;
 * exponentials, reciprocals and Phi are within 2^-20 of their value (Phi:
   1.5e-7 absolutely); 2^-18 stands for the handful of them in an activation.
Elements are compared as |got - ref| <= u |ref| + slack * scale, the scale being
the root of the sum of squares of what was added up for that element.
dW and dX of a layer with an activation are products of the rounded dZ: each
of its terms is off by up to u, which adds u * scale (a random walk, times 4)."""
import itertools
import math

import pytest
import torch

from backward_tcgen05_tma_gb300 import api, block, build
from backward_tcgen05_tma_gb300.module import SwiGLUMLP
from backward_tcgen05_tma_gb300.serving import MoESwiGLU, W4SwiGLUMLP
from conftest import device_status

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 0.0, "f16": 2.0 ** -24, "f32": 0.0}  # fp16's subnormal step
ACTS = list(api.ACTIVATIONS)


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    api.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def within(got, ref, u, slack, scale):
    """|got - ref| <= u |ref| + slack * scale everywhere."""
    d = (got.double() - ref).abs()
    bad = ~(d <= u * ref.abs() + slack * scale)
    assert not bool(bad.any()), "%d of %d off, worst by %.3g at %.3g" % (
        int(bad.sum()), bad.numel(), float(d[bad].max()), float(ref[bad].abs().max()))


def act64(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z) if name == "silu" else z


def dact64(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
LN_SHAPES = [(1, 8), (3, 16), (2, 248), (5, 256), (7, 264), (130, 512), (33, 520), (1, 1024), (64, 1032),
             (257, 2048), (9, 2056), (100, 4096), (31, 4104), (3, 8192), (611, 1000), (2, 8200), (5, 16384)]
FWD_SLACK = 2.0 ** -17  # (mean, centre, two sums over D <= 16384, root, product)


def ln64(s, w, b, eps):
    mean = s.mean(1, keepdim=True)
    var = ((s - mean) ** 2).mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    h = (s - mean) * rstd
    return h * (1 if w is None else w.double()) + (0 if b is None else b.double()), mean[:, 0], rstd[:, 0], h


@pytest.mark.parametrize("dtn", list(DT))
@pytest.mark.parametrize("M,D", LN_SHAPES)
def test_layer_norm_forward(dtn, M, D):
    g, dt = gen(M * 131 + D), DT[dtn]
    x, r = normal(g, M, D, std=2, mean=0.5, dtype=dt), normal(g, M, D, dtype=dt)
    w, b = normal(g, D, std=0.3, mean=1, dtype=dt), normal(g, D, std=0.3, dtype=dt)
    x[0] = 3.0  # a row without deviation: rstd = eps^-1/2
    r[0] = 0
    for res, ww, bb in ((None, w, b), (r, w, b), (r, None, None), (None, w, None)):
        Y, S, mean, rstd = api.swiglu_mlp_layer_norm_fwd(x, ww, bb, 1e-5, residual=res)
        s = x if res is None else (x.double() + r.double()).to(dt)
        assert (S is x) if res is None else torch.equal(S, s)
        ry, rm, rr, h = ln64(s.double(), ww, bb, 1e-5)
        wide = h.abs() * (1 if ww is None else w.double().abs()) + (0 if bb is None else b.double().abs())
        within(Y, ry, U[dtn], FWD_SLACK, wide + 1)
        within(mean, rm, 2.0 ** -24, FWD_SLACK, s.double().abs().mean(1) + 1e-30)
        within(rstd, rr, 2.0 ** -20, 0, 0 * rr)
        Y2, _, m2, r2 = api.swiglu_mlp_layer_norm_fwd(x, ww, bb, 1e-5, residual=res, stats=False)
        assert torch.equal(Y, Y2) and m2 is None and r2 is None


@pytest.mark.parametrize("dtn", list(DT))
def test_layer_norm_far_from_zero(dtn):
    # a mean of 100 deviations: squares about zero would lose the deviation in fp32
    g, dt = gen(5), DT[dtn]
    x = normal(g, 40, 1024, std=1.0, mean=100.0, dtype=dt)
    Y, _, _, _ = api.swiglu_mlp_layer_norm_fwd(x)
    ry, _, _, h = ln64(x.double(), None, None, 1e-5)
    # the mean is within 64 2^-24 of itself: 100 times that against the deviation
    within(Y, ry, U[dtn], 64 * 2.0 ** -24 * 100, h.abs() + 1)


@pytest.mark.parametrize("dtn", list(DT))
@pytest.mark.parametrize("M,D", LN_SHAPES + [(5000, 264), (3000, 1024)])
def test_layer_norm_backward(dtn, M, D):
    g, dt = gen(M * 17 + D), DT[dtn]
    x, dy, ds = (normal(g, M, D, std=s, mean=m, dtype=dt) for s, m in ((2, 0.5), (0.1, 0), (0.1, 0.05)))
    w = normal(g, D, std=0.3, mean=1, dtype=dt)
    _, _, mean, rstd = api.swiglu_mlp_layer_norm_fwd(x)
    for d, ww in ((None, w), (ds, w), (ds, None)):
        dX, dw, db = api.swiglu_mlp_layer_norm_bwd(dy, x, ww, mean, rstd, dS=d)
        y, r = dy.double(), rstd.double()[:, None]
        h = (x.double() - mean.double()[:, None]) * r
        t = y * (1 if ww is None else w.double())
        c = (t * h).mean(1, keepdim=True)
        ref = r * (t - t.mean(1, keepdim=True) - h * c) + (0 if d is None else ds.double())
        scale = r * (t.abs() + t.abs().mean(1, keepdim=True) + h.abs() * (t * h).abs().mean(1, keepdim=True)) + 1e-30
        within(dX, ref, U[dtn], 2.0 ** -18, scale)
        n = 4 * math.sqrt(M) * 2.0 ** -24 + 2.0 ** -20
        within(dw, (y * h).sum(0), U[dtn], n, (y * h).square().sum(0).sqrt() + TINY[dtn] / n)
        within(db, y.sum(0), U[dtn], n, y.square().sum(0).sqrt() + TINY[dtn] / n)
        # only what is wanted
        a, b, c2 = api.swiglu_mlp_layer_norm_bwd(dy, x, ww, mean, rstd, dS=d, need_dweight=False)
        assert torch.equal(a, dX) and b is None and torch.equal(c2, db)
        a, b, c2 = api.swiglu_mlp_layer_norm_bwd(dy, x, ww, mean, rstd, dS=d, need_dweight=False, need_dbias=False)
        assert torch.equal(a, dX) and b is None and c2 is None


def test_layer_norm_gradients_are_those_of_differences():
    # the formula above, in 64 bits, against central differences of the definition
    g = gen(3)
    M, D, e = 3, 24, 1e-5
    x, w, b, c = (torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)
                  for s in ((M, D), (D,), (D,), (M, D)))
    f = lambda x, w, b: float((ln64(x, w, b, e)[0] * c).sum())
    _, mean, rstd, h = ln64(x, w, b, e)
    t = c * w
    dx = rstd[:, None] * (t - t.mean(1, keepdim=True) - h * (t * h).mean(1, keepdim=True))
    for grad, at in ((dx, 0), ((c * h).sum(0), 1), (c.sum(0), 2)):
        for i in range(0, grad.numel(), 5):
            args = [[v.clone() for v in (x, w, b)] for _ in range(2)]
            args[0][at].view(-1)[i] += 1e-5
            args[1][at].view(-1)[i] -= 1e-5
            diff = (f(*args[0]) - f(*args[1])) / 2e-5
            assert abs(diff - float(grad.reshape(-1)[i])) <= 1e-6 * (1 + abs(diff))


@pytest.mark.parametrize("dtn", list(DT))
def test_layer_norm_accumulates_and_handles_no_rows(dtn):
    g, dt = gen(9), DT[dtn]
    x, dy = normal(g, 70, 264, dtype=dt), normal(g, 70, 264, dtype=dt)
    _, _, mean, rstd = api.swiglu_mlp_layer_norm_fwd(x)
    hw, hb = normal(g, 264, dtype=dt), normal(g, 264, dtype=dt)
    out = {"dweight": hw.clone(), "dbias": hb.clone()}
    api.swiglu_mlp_layer_norm_bwd(dy, x, None, mean, rstd, out=out, accumulate=True)
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for got, held, new in ((out["dweight"], hw, dy.double() * h), (out["dbias"], hb, dy.double())):
        within(got, held.double() + new.sum(0), U[dtn], 2.0 ** -18, new.square().sum(0).sqrt() + held.double().abs())
    none = torch.empty(0, 264, dtype=dt, device="cuda")
    Y, _, m0, r0 = api.swiglu_mlp_layer_norm_fwd(none)
    assert Y.shape == (0, 264) and m0.numel() == 0
    keep = {"dweight": hw.clone(), "dbias": hb.clone()}
    api.swiglu_mlp_layer_norm_bwd(none, none, None, m0, r0, out=keep, accumulate=True)
    assert torch.equal(keep["dweight"], hw) and torch.equal(keep["dbias"], hb)
    _, dw, db = api.swiglu_mlp_layer_norm_bwd(none, none, None, m0, r0, out=keep)
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("dtn", list(DT))
def test_layer_norm_rows_keep_to_themselves(dtn):
    # NaN and infinities in a row stay in it, and in the sums over rows
    g, dt = gen(11), DT[dtn]
    x, dy = normal(g, 50, 1032, dtype=dt), normal(g, 50, 1032, dtype=dt)
    clean, _, mean, rstd = api.swiglu_mlp_layer_norm_fwd(x)
    gx = api.swiglu_mlp_layer_norm_bwd(dy, x, None, mean, rstd)[0]
    x2 = x.clone()
    x2[7, 1000], x2[20, 0], x2[20, 1] = float("nan"), float("inf"), 1.0
    Y, _, m2, r2 = api.swiglu_mlp_layer_norm_fwd(x2)
    ok = torch.ones(50, dtype=torch.bool, device="cuda")
    ok[7] = ok[20] = False
    assert torch.equal(Y[ok], clean[ok]) and bool(Y[~ok].isnan().all())
    dX, dw, db = api.swiglu_mlp_layer_norm_bwd(dy, x2, None, m2, r2)
    assert torch.equal(dX[ok], gx[ok]) and bool(dX[~ok].isnan().all())
    assert bool(dw.isnan().all()) and not bool(db.isnan().any())


@pytest.mark.parametrize("M,D", [(37, 264), (300, 4096)])
def test_layer_norm_in_place(M, D):
    g = gen(M)
    x, r, dy, ds = (normal(g, M, D, dtype=torch.bfloat16) for _ in range(4))
    Y, S, mean, rstd = api.swiglu_mlp_layer_norm_fwd(x, residual=r)
    a, b = x.clone(), r.clone()
    Y2, S2, _, _ = api.swiglu_mlp_layer_norm_fwd(a, residual=b, out={"Y": a, "S": b})
    assert torch.equal(Y2, Y) and torch.equal(S2, S) and Y2 is a and S2 is b
    dX = api.swiglu_mlp_layer_norm_bwd(dy, S, None, mean, rstd, dS=ds)[0]
    for which in (0, 1):
        p = [dy.clone(), ds.clone()]
        got = api.swiglu_mlp_layer_norm_bwd(p[0], S, None, mean, rstd, dS=p[1], out={"dX": p[which]})[0]
        assert got is p[which] and torch.equal(got, dX)


# ---------------------------------------------------------------------------
# linear
# ---------------------------------------------------------------------------
LIN_SHAPES = [(1, 8, 8), (1, 2816, 1024), (3, 136, 72), (16, 128, 64), (17, 264, 1032), (33, 5640, 200),
              (48, 136, 2056), (49, 392, 320), (64, 1024, 4096), (65, 264, 328), (127, 136, 64),
              (129, 520, 1032), (300, 392, 2824), (1024, 2816, 1024), (2500, 264, 136)]


def act_slack(K):
    return 4 * math.sqrt(K) * 2.0 ** -24 + 2.0 ** -18


@pytest.mark.parametrize("dtn", list(DT))
@pytest.mark.parametrize("M,N,K", LIN_SHAPES)
def test_linear_forward(dtn, M, N, K):
    g, dt = gen(M + 3 * N + 7 * K), DT[dtn]
    X, W = normal(g, M, K, dtype=dt), normal(g, N, K, std=K ** -0.5, dtype=dt)
    b, R = normal(g, N, dtype=dt), normal(g, M, N, dtype=dt)
    xw = X.double() @ W.double().T
    root = (X.double().square() @ W.double().square().T).sqrt()
    combos = [("none", True, True, False), ("gelu", True, False, True), ("relu", False, True, True),
              ("gelu_tanh", True, True, True), ("silu", False, False, False), ("none", False, False, True)]
    for act, bias, res, keep in combos:
        Y, Z = api.swiglu_mlp_linear_fwd(X, W, b if bias else None, act, R if res else None, keep)
        z = xw + (b.double() if bias else 0)
        size = root + (b.double().abs() if bias else 0)
        # (no activation's slope is above 1.2)
        within(Y, act64(act, z) + (R.double() if res else 0), U[dtn], act_slack(K),
               1.2 * size + z.abs() + (R.double().abs() if res else 0) + TINY[dtn] / act_slack(K))
        assert (Z is not None) == keep
        if keep:
            within(Z, z, U[dtn], act_slack(K), size + TINY[dtn] / act_slack(K))


@pytest.mark.parametrize("dtn", list(DT))
@pytest.mark.parametrize("M,N,K", LIN_SHAPES)
def test_linear_backward(dtn, M, N, K):
    g, dt = gen(M + 5 * N + 11 * K), DT[dtn]
    dY, Z, pre = (normal(g, M, n, std=s, dtype=dt) for n, s in ((N, 0.1), (N, 1.5), (K, 1.5)))
    W = normal(g, N, K, std=K ** -0.5, dtype=dt)
    for act, x_act in (("none", "none"), ("gelu", "none"), ("none", "gelu_tanh"), ("relu", "silu"), ("silu", "relu"),
                       ("gelu_tanh", "gelu")):
        X = act64(x_act, pre.double()).to(dt)
        dZ = torch.empty(M, N, dtype=dt, device="cuda")
        dX, dW, db = api.swiglu_mlp_linear_bwd(dY, X, W, Z if act != "none" else None, act,
                                               X_pre=pre if x_act != "none" else None, x_activation=x_act,
                                               out={"dZ": dZ} if act != "none" else None)
        dz = dY.double() * dact64(act, Z.double())
        if act != "none":
            within(dZ, dz, U[dtn], 2.0 ** -18, dY.double().abs() + TINY[dtn] * 2.0 ** 18)
        off = 4 * U[dtn] if act != "none" else 0.0  # of the rounded dZ
        # a term's size: dZ itself is off by up to 2^-18 |dY| (the line above), which
        # where the slope is near 0 is more than 2^-18 |dZ|; slopes are below 1.2
        sq = dz.square() if act == "none" else dz.square() + dY.double().square()
        sx, sw, sb = act_slack(N) + off, act_slack(M) + off, act_slack(M)
        s = dact64(x_act, pre.double()) if x_act != "none" else torch.ones(M, K, dtype=torch.float64, device="cuda")
        size = (sq @ W.double().square()).sqrt() + TINY[dtn] * math.sqrt(N) / sx
        within(dX, (dz @ W.double()) * s, U[dtn], sx, size * (s.abs() + 2.0 ** -18 / sx) + (dz @ W.double()).abs() * 2.0 ** -18 / sx)
        within(dW, dz.T @ X.double(), U[dtn], sw, (sq.T @ X.double().square()).sqrt() + TINY[dtn] * math.sqrt(M) * 4 / sw)
        within(db, dz.sum(0), U[dtn], sb, sq.sum(0).sqrt() + TINY[dtn] / sb)


@pytest.mark.parametrize("dtn", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(65, 264, 328), (129, 520, 1032), (257, 392, 2824), (300, 40, 136), (2500, 1032, 264)])
def test_linear_on_sm_pairs(dtn, M, N, K):
    # the kernels that large sizes take, on ragged ones
    old = api.swiglu_mlp_set_cta_pairs(2)
    try:
        test_linear_forward(dtn, M, N, K)
        test_linear_backward(dtn, M, N, K)
    finally:
        api.swiglu_mlp_set_cta_pairs(old)


@pytest.mark.parametrize("dtn", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(64, 136, 16392), (40, 264, 23000), (1, 24, 120000), (33, 5640, 8200), (64, 2056, 9000),
                                   (7, 2456, 40), (5, 16, 264), (20, 40, 8)])
def test_linear_few_tokens_both_forms(dtn, M, N, K):
    # long contractions whose token rows do not fit a cluster's blocks, and short
    # ones with fewer 32-k blocks than a cluster has parts
    g, dt = gen(K), DT[dtn]
    X, W = normal(g, M, K, dtype=dt), normal(g, N, K, std=K ** -0.5, dtype=dt)
    b, R = normal(g, N, dtype=dt), normal(g, M, N, dtype=dt)
    z = X.double() @ W.double().T + b.double()
    root = (X.double().square() @ W.double().square().T).sqrt() + b.double().abs()
    Y, Z = api.swiglu_mlp_linear_fwd(X, W, b, "silu", R, keep=True)
    slack = act_slack(K)
    within(Z, z, U[dtn], slack, root)
    within(Y, act64("silu", z) + R.double(), U[dtn], slack, 1.2 * root + z.abs() + R.double().abs())


@pytest.mark.parametrize("dtn", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(17, 8, 8), (24, 40, 72), (33, 264, 520), (64, 2816, 1024), (63, 1032, 2056), (65, 24, 64),
                                   (128, 4104, 264), (129, 16, 5640), (200, 1032, 2824), (520, 5640, 136), (1000, 2056, 264),
                                   (1024, 8, 8), (1025, 272, 136), (2500, 1040, 264)])
def test_linear_some_tokens(dtn, M, N, K):
    # whole tiles and tiles of two and four blocks, boxes of fewer tokens than a tile,
    # one block of k, columns and tokens that end inside a tile; then the larger form
    test_linear_forward(dtn, M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 4, 4), (2, 12, 20), (4, 1004, 132), (5, 44, 20004), (8, 2060, 516), (9, 44, 5004),
                                   (32, 132, 9004), (2500, 1500, 2052), (1500, 2500, 36)])
def test_linear_in_fp32(M, N, K):
    # up to 8 rows, sizes that are odd multiples of 4, and last rounds in many parts
    test_linear_forward("f32", M, N, K)
    test_linear_backward("f32", M, N, K)


def test_activation_slopes_are_those_of_differences():
    z = torch.linspace(-6, 6, 997, dtype=torch.float64)
    for act in ACTS:
        if act == "relu":
            continue
        d = (act64(act, z + 1e-5) - act64(act, z - 1e-5)) / 2e-5
        assert float((d - dact64(act, z)).abs().max()) < 1e-8


@pytest.mark.parametrize("dtn", ["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS[1:])
def test_activations_over_the_whole_range(dtn, act):
    # X = one-hot rows: z is any 16-bit value exactly, on every path
    dt = DT[dtn]
    v = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(dt)
    v = v[v.isfinite() & (v.abs() <= (3e38 if dtn == "bf16" else 65504))]
    v = v[: v.numel() // 8 * 8].clone()
    N = v.numel()
    W = torch.zeros(N, 8, dtype=dt, device="cuda")
    W[:, 0] = v
    z = v.double()
    ref, slope = act64(act, z), dact64(act, z.clamp(-1e4, 1e4))
    for M in (1, 130):
        X = torch.zeros(M, 8, dtype=dt, device="cuda")
        X[:, 0] = 1
        Y, Z = api.swiglu_mlp_linear_fwd(X, W, None, act, keep=True)
        assert torch.equal(Z, v.expand(M, N))
        # near-zero values of z Phi(z) and z sigma(z) far left: Phi within 1.5e-7
        within(Y[M - 1], ref, U[dtn], 1.0, 2.0 ** -20 * ref.abs() + 1.6e-7 * z.abs().clamp(max=16) + TINY[dtn]
               + 2.0 ** -126)  # (values below are rounded by absolute steps)
        one = torch.ones(M, N, dtype=dt, device="cuda")
        dZ = torch.empty(M, N, dtype=dt, device="cuda")
        api.swiglu_mlp_linear_bwd(one, X, W, v.expand(M, N).contiguous(), act, need_dX=False, need_dW=False,
                                  out={"dZ": dZ})
        within(dZ[M - 1], slope, U[dtn], 1.0, 2.0 ** -18 + TINY[dtn] + 0 * slope)


@pytest.mark.parametrize("M", [4, 200])
@pytest.mark.parametrize("dtn", list(DT))
def test_infinities_and_nan(dtn, M):
    dt, inf, nan = DT[dtn], float("inf"), float("nan")
    b = torch.tensor([inf, -inf, nan, 1.0, 0, 0, 0, 0], dtype=dt, device="cuda")
    X, W = torch.zeros(M, 8, dtype=dt, device="cuda"), torch.zeros(8, 8, dtype=dt, device="cuda")
    z = b.double()
    for act in ACTS:
        Y, _ = api.swiglu_mlp_linear_fwd(X, W, b, act)
        ref = act64(act, z) if act != "gelu" else z * torch.special.ndtr(z)
        got = Y[M - 1].double()
        assert torch.equal(got.isnan(), ref.isnan()), (act, got, ref)
        assert torch.equal(got[:1], ref[:1]) and bool(got[2].isnan())
        if act != "none":
            dZ = torch.empty(M, 8, dtype=dt, device="cuda")
            api.swiglu_mlp_linear_bwd(torch.ones_like(dZ), X, W, b.expand(M, 8).contiguous(), act, out={"dZ": dZ})
            assert float(dZ[0, 0]) == 1 and float(dZ[0, 1]) == 0  # the slopes' limits
            assert act == "relu" or bool(dZ[0, 2].isnan())
    # a token's NaN touches no other token
    X[1, 3] = nan
    W[:, 3] = 1
    Y, _ = api.swiglu_mlp_linear_fwd(X, W, None, "silu")
    assert bool(Y[1].isnan().all()) and not bool(Y[2:].isnan().any()) and not bool(Y[0].isnan().any())


@pytest.mark.parametrize("dtn", list(DT))
@pytest.mark.parametrize("M", [20, 333])
def test_linear_accumulates_aliases_and_handles_no_rows(dtn, M):
    g, dt, N, K = gen(M), DT[dtn], 136, 264
    dY, Z, pre, R = (normal(g, M, n, std=0.5, dtype=dt) for n in (N, N, K, N))
    X, W, b = normal(g, M, K, dtype=dt), normal(g, N, K, std=0.1, dtype=dt), normal(g, N, dtype=dt)
    hW, hb = normal(g, N, K, dtype=dt), normal(g, N, dtype=dt)
    out = {"dW": hW.clone(), "dbias": hb.clone()}
    api.swiglu_mlp_linear_bwd(dY, X, W, out=out, accumulate=True)
    y = dY.double()
    within(out["dW"], hW.double() + y.T @ X.double(), U[dtn], act_slack(M),
           (y.square().T @ X.double().square()).sqrt() + hW.double().abs())
    within(out["dbias"], hb.double() + y.sum(0), U[dtn], act_slack(M), y.square().sum(0).sqrt() + hb.double().abs())
    # Y over the residual; dZ over dY or Z; dX over X_pre
    Y, _ = api.swiglu_mlp_linear_fwd(X, W, b, "silu", R)
    r = R.clone()
    assert torch.equal(api.swiglu_mlp_linear_fwd(X, W, b, "silu", r, out={"Y": r})[0], Y)
    ref = api.swiglu_mlp_linear_bwd(dY, X, W, Z, "gelu", X_pre=pre, x_activation="silu")
    for which in (0, 1):
        p = [dY.clone(), Z.clone()]
        q = pre.clone()
        got = api.swiglu_mlp_linear_bwd(p[0], X, W, p[1], "gelu", X_pre=q, x_activation="silu",
                                        out={"dZ": p[which], "dX": q})
        assert all(torch.equal(a, c) for a, c in zip(got, ref))
    # parts of the backward pass give what the whole gives
    for need in itertools.product((False, True), repeat=3):
        got = api.swiglu_mlp_linear_bwd(dY, X, W, Z, "gelu", X_pre=pre, x_activation="silu", need_dX=need[0],
                                        need_dW=need[1], need_dbias=need[2])
        assert all((a is None) if not n else torch.equal(a, c) for a, c, n in zip(got, ref, need))
    none = torch.empty(0, K, dtype=dt, device="cuda")
    assert api.swiglu_mlp_linear_fwd(none, W, b)[0].shape == (0, N)
    g0 = torch.empty(0, N, dtype=dt, device="cuda")
    api.swiglu_mlp_linear_bwd(g0, none, W, out=out, accumulate=True)
    dX, dW, db = api.swiglu_mlp_linear_bwd(g0, none, W)
    assert dX.shape == (0, K) and not dW.any() and not db.any() and bool(out["dW"].any())


def guarded(shape, dtype, fill=-7.0):
    """A tensor inside a larger buffer of known values, and a check of those."""
    n = math.prod(shape)
    buf = torch.full((n + 512,), fill, dtype=dtype, device="cuda")
    t = buf[256:256 + n].view(shape)
    return t, lambda: bool((buf[:256] == fill).all()) and bool((buf[256 + n:] == fill).all())


@pytest.mark.parametrize("dtn", list(DT))
@pytest.mark.parametrize("M,N,K", [(13, 264, 136), (77, 136, 200), (300, 1032, 392)])
def test_nothing_is_written_outside_the_outputs(dtn, M, N, K):
    g, dt = gen(N), DT[dtn]
    X, W, dY, Z = (normal(g, *s, dtype=dt) for s in ((M, K), (N, K), (M, N), (M, N)))
    shapes = {"Y": (M, N), "Z": (M, N), "dZ": (M, N), "dX": (M, K), "dW": (N, K), "dbias": (N,)}
    out, checks = {}, []
    for k, s in shapes.items():
        out[k], c = guarded(s, dt)
        checks.append(c)
    api.swiglu_mlp_linear_fwd(X, W, None, "gelu", dY, keep=True, out=out)
    api.swiglu_mlp_linear_bwd(dY, X, W, Z, "gelu", X_pre=X, x_activation="silu", out=out)
    ln = {k: guarded(s, d) for k, s, d in (("Y", (M, K), dt), ("S", (M, K), dt), ("mean", (M,), torch.float32),
                                           ("rstd", (M,), torch.float32), ("dX", (M, K), dt), ("dweight", (K,), dt),
                                           ("dbias", (K,), dt))}
    lo = {k: v[0] for k, v in ln.items()}
    Y, S, mean, rstd = api.swiglu_mlp_layer_norm_fwd(X, residual=X, out=lo)
    api.swiglu_mlp_layer_norm_bwd(X, S, None, mean, rstd, out=lo)
    torch.cuda.synchronize()
    assert all(c() for c in checks) and all(v[1]() for v in ln.values())
    assert not any(bool((t == -7.0).all()) for t in list(out.values()) + list(lo.values()))


# ---------------------------------------------------------------------------
# as they are used
# ---------------------------------------------------------------------------
def all_calls(ws=None, seed=0, dt=torch.bfloat16, stream=None):
    """Every kind of call in turn, on one workspace if given: their outputs."""
    g = gen(seed)
    got = []
    for M, N, K in ((5, 5640, 264), (64, 264, 1032), (200, 520, 1032), (700, 1032, 264)):
        X, W, b, R = (normal(g, *s, dtype=dt) for s in ((M, K), (N, K), (N,), (M, N)))
        Y, Z = api.swiglu_mlp_linear_fwd(X, W, b, "gelu", R, keep=True, ws=ws)
        got += [Y, Z, *api.swiglu_mlp_linear_bwd(R, X, W, Z, "gelu", ws=ws)]
        H, S, mean, rstd = api.swiglu_mlp_layer_norm_fwd(R, b, b, residual=Y)
        got += [H, S, *api.swiglu_mlp_layer_norm_bwd(R, S, b, mean, rstd, dS=Y, ws=ws)]
    return got


def test_one_workspace_serves_all_calls_in_turn():
    n = max(api.linear_workspace(M, N, K, torch.bfloat16, op, "cuda").numel()
            for M, N, K in ((5, 5640, 264), (64, 264, 1032), (200, 520, 1032), (700, 1032, 264))
            for op in (api.SWIGLU_OP_FWD, api.SWIGLU_OP_BWD))
    n = max(n, api.layer_norm_workspace(700, 5640, torch.bfloat16, "cuda").numel())
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    ref = all_calls()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(all_calls(ws), ref))
        assert api.swiglu_mlp_query_error(ws) == 0


def test_calls_on_two_streams_at_once():
    refs = [all_calls(seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in refs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, st in zip((1, 2), streams):
            with torch.cuda.stream(st):
                got.append(all_calls(seed=s))
        torch.cuda.synchronize()
        for a, r in zip(got, refs):
            assert all(torch.equal(x, y) for x, y in zip(a, r))


def reference_block(x, delta, p, act, eps=1e-5):
    """The sublayer in 64 bits with autograd, roundings left out."""
    s = x if delta is None else x + delta
    mean = s.mean(-1, keepdim=True)
    h = (s - mean) * ((s - mean).square().mean(-1, keepdim=True) + eps).rsqrt() * p["norm.weight"] + p["norm.bias"]
    z = h @ p["mlp.up_weight"].T + p["mlp.up_bias"]
    return s + act64(act, z) @ p["mlp.down_weight"].T + p["mlp.down_bias"]


@pytest.mark.parametrize("dtn,B,S,D,H,act", [("f32", 2, 16, 64, 176, "gelu"), ("bf16", 2, 150, 320, 1032, "gelu_tanh"),
                                             ("f16", 1, 40, 256, 520, "silu"), ("bf16", 3, 7, 1024, 2816, "relu")])
def test_pre_norm_block_trains_like_its_definition(dtn, B, S, D, H, act):
    # Frobenius: each tensor passes at most five roundings on its way (norm, A
    # or Z, dZ, the LN's gradient, its own), Z's as the place where the slope
    # is taken: 5 u, and as much again for products of roundings and fp32 sums.
    # relu's slope jumps: z, whose terms' roundings make it off by up to u / sqrt 3
    # of its deviation, has the other sign than in 64 bits with a probability of
    # E|e| phi(0) = 0.8 u / sqrt 3 * 0.4 = 0.18 u, and then its whole gradient is
    # off, half of all being 0: sqrt(2 * 0.18 u) < sqrt u of the norm
    g, dt = gen(D), DT[dtn]
    torch.manual_seed(D)
    m = block.MLPBlock(block.MLP(D, H, activation=act, dtype=dt, device="cuda"), dtype=dt, device="cuda")
    with torch.no_grad():
        m.norm.weight.copy_(normal(g, D, std=0.2, mean=1))
        m.norm.bias.copy_(normal(g, D, std=0.2))
    x, delta = (normal(g, B, S, D, dtype=dt).requires_grad_() for _ in range(2))
    dy = normal(g, B, S, D, std=0.1, dtype=dt)
    p = {k: v.detach().double().requires_grad_() for k, v in m.named_parameters()}
    x64, d64 = x.detach().double().requires_grad_(), delta.detach().double().requires_grad_()
    ref = reference_block(x64, d64, p, act)
    ref.backward(dy.double())
    out = m(x, delta)
    leaves = dict(m.named_parameters(), x=x, delta=delta)
    grads = torch.autograd.grad(out, list(leaves.values()), dy, retain_graph=True)
    again = torch.autograd.grad(out, list(leaves.values()), dy)
    tol = 10 * max(U[dtn], 2.0 ** -20)
    rel = lambda a, b: float((a.detach().double() - b).norm() / b.norm())
    assert rel(out, ref.detach()) <= tol
    if act == "relu":
        tol += U[dtn] ** 0.5
    for (name, _), a, b in zip(leaves.items(), grads, again):
        want = {"x": x64, "delta": d64}.get(name, p.get(name)).grad
        assert torch.equal(a, b) and rel(a, want) <= tol, name
    with torch.no_grad():
        assert torch.equal(m(x, delta), out)
    # without delta, and with a part of the leaves
    m.mlp.up_weight.requires_grad_(False)
    m.norm.weight.requires_grad_(False)
    xi = x.detach().clone().requires_grad_()
    m(xi).sum().backward()  # an expanded gradient
    assert xi.grad.isfinite().all() and m.mlp.up_weight.grad is None and m.mlp.down_bias.grad is not None
    with pytest.raises(RuntimeError):
        torch.autograd.grad(torch.autograd.grad(m(xi).sum(), xi, create_graph=True)[0].sum(), xi)


def test_block_of_a_gated_mlp():
    D, H = 320, 904
    g = gen(2)
    torch.manual_seed(2)
    m = block.MLPBlock(SwiGLUMLP(D, H, device="cuda"), device="cuda")
    x = normal(g, 70, D, dtype=torch.bfloat16).requires_grad_()
    out = m(x)
    y = block.layer_norm(x, m.norm.weight, m.norm.bias, m.norm.eps)
    assert torch.equal(out, x + m.mlp(y))
    out.sum().backward()
    assert x.grad.isfinite().all() and m.norm.weight.grad.isfinite().all() and m.mlp.down_weight.grad.isfinite().all()


def test_sublayers_pass_their_sums_on():
    # two sublayers as a server runs them, 4-bit and mixture of experts among
    # them: each sum in the next norm's kernel
    D, g = 256, gen(3)
    torch.manual_seed(3)
    with torch.no_grad():
        mlps = [block.MLP(D, 520, device="cuda"), W4SwiGLUMLP(SwiGLUMLP(D, 704, device="cuda"), group=64),
                MoESwiGLU(D, 128, 8, 2, device="cuda")]
        blocks = [block.MLPBlock(m, hidden_size=D, device="cuda") for m in mlps]
        x = normal(g, 5, D, dtype=torch.bfloat16)
        s, d = x, None
        for b in blocks:
            s, d = b(s, d, join=False)
        joined = x
        for b in blocks:
            joined = b(joined)
        # the MLP's sum is rounded once in its epilogue, else its product before it too
        assert float(((s + d).double() - joined.double()).norm() / joined.double().norm()) <= 6 * U["bf16"]
        if api._use_debug:  # (which waits for every call: nothing to capture)
            return
        # as one captured step
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            blocks[0](x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            t, e = x, None
            for b in blocks:
                t, e = b(t, e, join=False)
        x.copy_(normal(g, 5, D, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        s, d = x, None
        for b in blocks:
            s, d = b(s, d, join=False)
        assert torch.equal(t, s) and torch.equal(e, d)


def test_layers_take_views_and_odd_batches():
    g = gen(8)
    x = normal(g, 4, 6, 264, dtype=torch.bfloat16)
    w, b = normal(g, 136, 264, dtype=torch.bfloat16), normal(g, 136, dtype=torch.bfloat16)
    t = x.transpose(0, 1)  # rows that do not follow one another
    assert torch.equal(block.linear(t, w, b, "relu"), block.linear(t.contiguous(), w, b, "relu"))
    assert torch.equal(block.layer_norm(t), block.layer_norm(x).transpose(0, 1))
    assert torch.equal(block.layer_norm(x[:, :1].expand(4, 6, 264)), block.layer_norm(x)[:, :1].expand(4, 6, 264))
    assert block.linear(x[:0], w, b).shape == (0, 6, 136)
    assert block.linear(x[0, 0], w, b).shape == (136,)
    s = x.clone().requires_grad_()
    block.linear(s[:0], w, b).sum().backward()
    assert not s.grad.any()


def test_captured_training_step():
    if api._use_debug:
        pytest.skip("the debug build's session waits for every call")
    g = gen(4)
    torch.manual_seed(4)
    m = block.MLPBlock(block.MLP(256, 520, device="cuda"), device="cuda")
    params = list(m.parameters())
    x, dy = (normal(g, 200, 256, dtype=torch.bfloat16) for _ in range(2))
    step = lambda: [m_out := m(x, x), *torch.autograd.grad(m_out, params, dy)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (5, 6):
        h = gen(seed)
        x.copy_(normal(h, 200, 256, dtype=torch.bfloat16))
        dy.copy_(normal(h, 200, 256, dtype=torch.bfloat16))
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        ref = step()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("dtn", list(DT))
def test_debug_build_checks_every_access(dtn):
    release = all_calls(dt=DT[dtn])
    prev = api.use_debug_library(True)
    try:
        debug = all_calls(dt=DT[dtn])  # (raises on a failed check)
        x = normal(gen(1), 40, 264, dtype=DT[dtn])
        w = normal(gen(2), 136, 264, dtype=DT[dtn])
        for call in ("layer_norm_bwd", "linear_fwd", "linear_bwd"):
            L = api.lib()
            ws = torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")
            st = torch.ones(40, device="cuda")
            run = {"layer_norm_bwd": lambda: api.swiglu_mlp_layer_norm_bwd(x, x, None, st, st, ws=ws),
                   "linear_fwd": lambda: api.swiglu_mlp_linear_fwd(x, w, ws=ws),
                   "linear_bwd": lambda: api.swiglu_mlp_linear_bwd(x[:, :136].contiguous(), x, w, need_dbias=False, ws=ws)}[call]
            L.swiglu_mlp_debug_narrow_once(1)
            assert device_status(run, ws) == 7, call
            assert device_status(run, ws) == 0, call
    finally:
        api.use_debug_library(prev)
    assert all(torch.equal(a, b) for a, b in zip(release, debug))


@pytest.mark.parametrize("M", [8, 40, 300, 2000])
def test_a_wait_that_runs_out_is_reported(M):
    g = gen(M)
    X, W = normal(g, M, 1032, dtype=torch.bfloat16), normal(g, 264, 1032, dtype=torch.bfloat16)
    ref = api.swiglu_mlp_linear_fwd(X, W)[0]
    old = api.swiglu_mlp_set_wait_limit_ns(20_000_000)
    try:
        ws = api.linear_workspace(M, 264, 1032, torch.bfloat16, api.SWIGLU_OP_FWD, "cuda")
        api.swiglu_mlp_inject_stall_once(True)
        call = lambda: api.swiglu_mlp_linear_fwd(X, W, ws=ws)
        assert device_status(call, ws) == 6
        ws.zero_()
        api.swiglu_mlp_inject_stall_once(False)
        assert device_status(call, ws) == 0 and torch.equal(call()[0], ref)
    finally:
        api.swiglu_mlp_inject_stall_once(False)
        api.swiglu_mlp_set_wait_limit_ns(old)


def test_refusals_of_the_binding():
    g = gen(1)
    X, W = normal(g, 8, 264, dtype=torch.bfloat16), normal(g, 136, 264, dtype=torch.bfloat16)
    Y = normal(g, 8, 136, dtype=torch.bfloat16)
    bad = [lambda: api.swiglu_mlp_linear_fwd(X, W.half()), lambda: api.swiglu_mlp_linear_fwd(X, W.T),
           lambda: api.swiglu_mlp_linear_fwd(X, W, bias=X[0]), lambda: api.swiglu_mlp_linear_fwd(X, W, residual=X),
           lambda: api.swiglu_mlp_linear_fwd(X, W, activation="tanh"),
           lambda: api.swiglu_mlp_linear_fwd(X, W, out={"Y": X}),
           lambda: api.swiglu_mlp_linear_fwd(X, W, ws=torch.zeros(1 << 20, device="cuda")),
           lambda: api.swiglu_mlp_linear_fwd(X, W, ws=torch.zeros(1 << 20, dtype=torch.uint8)),
           lambda: api.swiglu_mlp_linear_fwd(X.T, W), lambda: api.swiglu_mlp_linear_bwd(Y, X, W, activation="gelu"),
           lambda: api.swiglu_mlp_linear_bwd(Y, X, W, x_activation="gelu"),
           lambda: api.swiglu_mlp_linear_bwd(Y, X, W, accumulate=True),
           lambda: api.swiglu_mlp_layer_norm_fwd(X, residual=Y), lambda: api.swiglu_mlp_layer_norm_fwd(X, weight=Y[0]),
           lambda: api.swiglu_mlp_layer_norm_bwd(X, X, None, X[:, 0], X[:, 0]),
           lambda: api.swiglu_mlp_layer_norm_bwd(X, Y, None, X[:, 0].float(), X[:, 0].float())]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: api.swiglu_mlp_linear_fwd(X, W, ws=torch.zeros(64, dtype=torch.uint8, device="cuda")),
              lambda: api.swiglu_mlp_linear_fwd(X[:, :260].contiguous(), W[:, :260].contiguous()),
              lambda: api.swiglu_mlp_layer_norm_fwd(X, eps=float("nan"))):
        with pytest.raises(api.SwigluError):
            f()
