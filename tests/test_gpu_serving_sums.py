"""Sums of the few-token products where elements of a token differ widely in
size, or are not finite.

Tolerances, fixed before any run.  A product's sum is a sum of whole numbers
q - z times elements, scaled group by group: no term is larger than the
formula's own.  Along the longest path of additions there are at most 64 within
a unit of 64 elements (the tensor core's order), one per group of at least 32,
and those that join warps and blocks (at most 32); each is off by at most 2^-23
(truncation) of the sum of the terms' magnitudes.  So an output lies within
    u |y| + (96 + K / 32) 2^-23 sum_k |W| |x|
of the formula's, with u one rounding to the output's type: an element that a
weight of 0 meets adds nothing to either side, however large it is."""
import pytest
import torch

from backward_tcgen05_tma_gb300 import api, build

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    api.lib()


def quantized(g, lead, N, K, group, zeros, dtype, nothing_at):
    """Random codes, scales and zero points (None: 8), with weights of 0 at the
    columns `nothing_at` in every other row: codes equal to the zero point."""
    ng = -(-K // group)
    rand = lambda *s: torch.randint(0, 16, s, generator=g, device="cuda", dtype=torch.uint8)
    q, z = rand(*lead, N, K), rand(*lead, N, ng) if zeros else None
    for k in nothing_at:
        q[..., ::2, k] = 8 if z is None else z[..., ::2, k // group]
    s = (torch.rand(*lead, N, ng, generator=g, device="cuda") + 0.5).mul_(0.2 * K ** -0.5).to(dtype)
    w = (q.double() - (8.0 if z is None else z.double().repeat_interleave(group, -1)[..., :K]))
    w *= s.double().repeat_interleave(group, -1)[..., :K]
    return ((q[..., 0::2] | q[..., 1::2] << 4).contiguous(), s, z), w


def tokens(g, M, K, dtype, large, at):
    X = torch.randn(M, K, generator=g, device="cuda")
    for i, k in enumerate(at):
        X[:, k] = large * (-1) ** i
    return X.to(dtype)


# one token, the columns of every form of the products, and the tensor-core form
TOKENS = [1, 8, 12, 24, 40]
LARGE = [("f16", 30000.0), ("bf16", 30000.0), ("bf16", 2.0 ** 30)]


@pytest.mark.parametrize("dtn,large", LARGE)
@pytest.mark.parametrize("group,zeros", [(128, False), (64, True), (32, False), (32, True)])
@pytest.mark.parametrize("M", TOKENS)
def test_elements_that_meet_weights_of_zero_do_not_matter(M, group, zeros, dtn, large):
    g, N, K, at = torch.Generator(device="cuda").manual_seed(M + group), 200, 520, (3, 70, 517)
    w, ref = quantized(g, (), N, K, group, zeros, DT[dtn], at)
    X = tokens(g, M, K, DT[dtn], large, at)
    Y = api.swiglu_mlp_w4_linear(X, api.swiglu_mlp_w4_pack(*w, group)).double()
    x = X.double()
    y, terms = x @ ref.T, x.abs() @ ref.abs().T
    tol = U[dtn] * y.abs() + (96 + K / 32) * 2.0 ** -23 * terms
    ok = torch.isfinite(y.to(DT[dtn]))  # fp16: the rows with other weights may pass 65504
    assert bool(ok[:, ::2].all()) and bool(((Y - y).abs() <= tol)[ok].all())


@pytest.mark.parametrize("dtn,large", LARGE)
@pytest.mark.parametrize("group,zeros", [(128, False), (64, True), (32, True)])
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (20, 4, 2), (64, 3, 3)])
def test_experts_and_elements_that_meet_weights_of_zero(T, E, k, group, zeros, dtn, large):
    # one hidden unit's rows are even rows of both Wg and Wu (H even): its value
    # is an ordinary one; the other units' weights in Wd are 0
    g, D, H, at, dt = torch.Generator(device="cuda").manual_seed(T + group), 136, 48, (5, 100), DT[dtn]
    gu, rgu = quantized(g, (E,), 2 * H, D, group, zeros, dt, at)
    dn, rdn = quantized(g, (E,), D, H, group, zeros, dt, ())
    rest = torch.arange(1, H, 2).tolist()
    q = torch.stack((dn[0] & 15, dn[0] >> 4), -1).flatten(-2)
    for c in rest:
        q[..., c] = 8 if dn[2] is None else dn[2][..., c // group]
        rdn[..., c] = 0
    dn = ((q[..., 0::2] | q[..., 1::2] << 4).contiguous(), *dn[1:])
    X = tokens(g, T, D, dt, large, at)
    X[:, list(at)] = torch.where(torch.rand(T, 1, generator=g, device="cuda") < 0.5, X[:, list(at)], 0)
    # odd units would overflow: their rows' weights at the large columns are taken out too
    q = torch.stack((gu[0] & 15, gu[0] >> 4), -1).flatten(-2)
    for c in at:
        q[..., c] = 8 if gu[2] is None else gu[2][..., c // group]
        rgu[..., c] = 0
    gu = ((q[..., 0::2] | q[..., 1::2] << 4).contiguous(), *gu[1:])
    idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    wt = torch.rand(T, k, generator=g, device="cuda")
    Y = api.swiglu_mlp_moe_experts(X, idx, wt, api.swiglu_mlp_w4_pack(*gu, group, gate_up=True),
                                   api.swiglu_mlp_w4_pack(*dn, group)).double()
    want, spread = torch.zeros_like(Y), torch.zeros_like(Y)
    x = X.double()
    for j in range(k):
        e = idx[:, j].long()
        gate, up = (rgu[e] @ x[:, :, None])[:, :, 0].chunk(2, 1)
        terms_g, terms_u = (rgu[e].abs() @ x.abs()[:, :, None])[:, :, 0].chunk(2, 1)
        a = gate * torch.sigmoid(gate) * up
        # the hidden value's own errors: its rounding, the sums of gate and up
        # (SiLU grows by at most 1.1 per unit of gate) and the exponential
        n = (96 + D / 32) * 2.0 ** -23
        da = (U[dtn] + 2.0 ** -20) * a.abs() + n * (1.1 * terms_g * up.abs() + terms_u * gate.abs())
        w = wt[:, j].double()[:, None]
        want += w * (rdn[e] @ a[:, :, None])[:, :, 0]
        spread += w * (rdn[e].abs() @ (da + (96 + H / 32) * 2.0 ** -23 * a.abs())[:, :, None])[:, :, 0]
    assert bool(((Y - want).abs() <= U[dtn] * want.abs() + 1.01 * spread + 1e-30).all())


def classes(t):
    return torch.isnan(t), torch.isposinf(t), torch.isneginf(t)


@pytest.mark.parametrize("dtn", ["bf16", "f16"])
@pytest.mark.parametrize("M", TOKENS)
def test_infinities_give_what_the_formula_gives(M, dtn):
    # inf times q - z: an infinity of its sign, or NaN for 0; whatever the form
    g, N, K, group, at = torch.Generator(device="cuda").manual_seed(M), 72, 264, 64, (6, 131)
    w, ref = quantized(g, (), N, K, group, True, DT[dtn], at)
    X = tokens(g, M, K, DT[dtn], 1.0, at)
    W = api.swiglu_mlp_w4_pack(*w, group)
    clean = api.swiglu_mlp_w4_linear(X, W)
    X[M // 2, at[0]] = float("inf")
    X[M - 1, at[1]] = -float("inf")  # M = 1: both in one row
    Y, want = api.swiglu_mlp_w4_linear(X, W), X.double() @ ref.T
    assert torch.isnan(want[M // 2]).any() and torch.isinf(want[M // 2]).any()
    for got, exp in zip(classes(Y.double()), classes(want)):
        assert torch.equal(got, exp)
    keep = [i for i in range(M) if i not in (M // 2, M - 1)]
    assert torch.equal(Y[keep], clean[keep])


@pytest.mark.parametrize("fmt", [None, (64, True)])
@pytest.mark.parametrize("T", [1, 20])
def test_infinities_in_experts(T, fmt):
    # 16-bit and 4-bit experts alike: NaN where a gate, an up value or the sum of
    # the hidden values' products is NaN; a token without one keeps its bits
    g, D, H, E, dt = torch.Generator(device="cuda").manual_seed(T), 72, 40, 3, torch.bfloat16
    if fmt is None:
        gu = torch.randn(E, 2 * H, D, generator=g, device="cuda").to(dt)
        dn = torch.randn(E, D, H, generator=g, device="cuda").to(dt)
        gu[:, ::2, 6] = 0
        args, rgu, rdn = (gu, dn), gu.double(), dn.double()
    else:
        (gu, rgu), (dn, rdn) = (quantized(g, (E,), n, k, *fmt, dt, c) for n, k, c in ((2 * H, D, (6,)), (D, H, ())))
        args = (api.swiglu_mlp_w4_pack(*gu, fmt[0], gate_up=True), api.swiglu_mlp_w4_pack(*dn, fmt[0]))
    X = torch.randn(T, D, generator=g, device="cuda").to(dt)
    idx = (torch.arange(T, device="cuda")[:, None] % E).int()
    wt = torch.ones(T, 1, device="cuda")
    clean = api.swiglu_mlp_moe_experts(X, idx, wt, *args)
    X[T - 1, 6] = float("inf")
    Y = api.swiglu_mlp_moe_experts(X, idx, wt, *args)
    e = int(idx[T - 1, 0])
    gate, up = (rgu[e] @ X[T - 1].double()).chunk(2)
    want = rdn[e] @ (gate * torch.sigmoid(gate) * up)
    for got, exp in zip(classes(Y[T - 1].double()), classes(want)):
        assert torch.equal(got, exp)
    assert torch.equal(Y[:T - 1], clean[:T - 1])
