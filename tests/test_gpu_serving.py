"""The few-token serving operators against restatements of their definitions
in 64 bits: 4-bit weights (rounding, layout, linear, MLP) and mixtures of
experts (router, experts, whole layer).

Tolerances, fixed before any run.  u is the largest relative error of one
rounding to the output's type (2^-8 bf16, 2^-11 fp16), so outputs that are
rounded once from nearly exact sums are within u of the reference in the
Frobenius norm; SLACK = 2^-13 covers the fp32 sums (fp16: the magic number
1024 against code values of about 4.6 leaves 2^-24 * 1024 / 4.6 * a few
additions = 2^-14 of a unit's sum) and the exponential.  The hidden values A
are rounded to the type before the down product; references of Y use the
rounded A, whose own differences (a rounding that falls the other way) are
again within u: 2 u.  Elements are held to the same bounds relative to the
larger of the element and the row's root mean square, times 8 (a deviation of
8 times the Frobenius one)."""
import ctypes

import numpy as np
import pytest
import torch

from backward_tcgen05_tma_gb300 import api, build
from backward_tcgen05_tma_gb300.module import SwiGLUMLP
from backward_tcgen05_tma_gb300.serving import MoESwiGLU, W4SwiGLUMLP

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SLACK = 2.0 ** -13


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    api.lib()


def near(got, ref, tol):
    g, r = got.double().cpu(), ref.double().cpu()
    assert g.shape == r.shape and torch.isfinite(g).all()
    rms = r.square().mean(-1, keepdim=True).sqrt()
    assert float((g - r).norm()) <= tol * float(r.norm()) + 1e-30
    assert bool(((g - r).abs() <= 8 * tol * torch.maximum(r.abs(), rms) + 1e-30).all())


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def codes(g, lead, N, K, group, zeros, dtype):
    """Random codes, scales and zero points: every code value occurs."""
    ng = -(-K // group)
    q = torch.randint(0, 16, (*lead, N, K), generator=g, device="cuda", dtype=torch.uint8)
    c = (q[..., 0::2] | q[..., 1::2] << 4).contiguous()
    s = (torch.rand(*lead, N, ng, generator=g, device="cuda") + 0.5).mul_(0.2 * K ** -0.5).to(dtype)
    z = torch.randint(0, 16, (*lead, N, ng), generator=g, device="cuda", dtype=torch.uint8)
    return c, s, z if zeros else None


def weights64(c, s, z, group):
    q = torch.stack((c & 15, c >> 4), -1).flatten(-2).double()
    K = q.shape[-1]
    zz = 8.0 if z is None else z.double().repeat_interleave(group, -1)[..., :K]
    return (q - zz) * s.double().repeat_interleave(group, -1)[..., :K]


def hidden64(x, wgu, gm=1.0):
    H = wgu.shape[0] // 2
    g = gm * (x @ wgu[:H].T)
    return g * torch.sigmoid(g) * (x @ wgu[H:].T)


# ---------------------------------------------------------------------------
# 4-bit weights: rounding and layout
# ---------------------------------------------------------------------------
def quantize_ref(W, group, zeros, dtype):
    w = W.float().cpu().numpy()
    N, K = w.shape
    ng = -(-K // group)
    s, z, q = np.zeros((N, ng), np.float32), np.full((N, ng), 8, np.uint8), np.zeros((N, K), np.uint8)
    for i in range(ng):
        p = w[:, i * group:(i + 1) * group]
        lo, hi = np.minimum(p.min(1), 0), np.maximum(p.max(1), 0)
        raw = (hi - lo) / np.float32(15) if zeros else np.maximum(hi, -lo) / np.float32(7)
        si = torch.from_numpy(raw.astype(np.float32)).to(dtype).float().numpy()
        ok = si != 0
        d = np.where(ok, si, 1).astype(np.float32)
        zi = np.full(N, 8, np.float32)
        if zeros:
            zi = np.where(ok, np.clip(np.rint(-lo / d), 0, 15), 8).astype(np.float32)
        qi = np.where(ok[:, None], np.clip(np.rint(p / d[:, None]) + zi[:, None], 0, 15), zi[:, None])
        s[:, i], z[:, i], q[:, i * group:(i + 1) * group] = si, zi, qi
    return q, s, z


@pytest.mark.parametrize("dtn", ["bf16", "f16"])
@pytest.mark.parametrize("N,K,group,zeros", [(5, 72, 32, False), (33, 200, 64, True),
                                             (16, 256, 128, False), (7, 8, 128, True),
                                             (64, 1024, 32, True)])
def test_quantize_is_the_definition(dtn, N, K, group, zeros):
    g = gen(N * K)
    W = normal(g, N, K, dtype=DT[dtn])
    W[1] = 0                       # scale 0
    W[2] = W[2].abs() + 0.1        # one sign
    W[3, : K // 2] = 5.0
    q, s, z = quantize_ref(W, group, zeros, DT[dtn])
    c, gs, gz = api.swiglu_mlp_w4_quantize(W, group, zeros)
    got = torch.stack((c & 15, c >> 4), -1).flatten(-2).cpu().numpy()
    assert np.array_equal(got, q) and np.array_equal(gs.float().cpu().numpy(), s)
    assert (gz is None) == (not zeros) and (gz is None or np.array_equal(gz.cpu().numpy(), z))
    # a stack of matrices is rounded matrix by matrix
    c3, s3, _ = api.swiglu_mlp_w4_quantize(torch.stack((W, W)), group, zeros)
    assert torch.equal(c3[1], c) and torch.equal(s3[0], gs)


def pack_ref(c, s, z, group, gate_up):
    """The packed layout written out (numpy, uint8)."""
    q = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], -1)
    N, K = q.shape
    nk, sets, H = -(-K // 64), 2 if group == 32 else 1, N // 2
    tiles = -(-H // 8) if gate_up else -(-N // 16)
    rec = 512 + sets * (32 if z is None else 48)
    out = np.zeros((tiles, nk, rec), np.uint8)
    for t in range(tiles):
        rows = [(t * 8 + r % 8 + (H if r >= 8 else 0) if t * 8 + r % 8 < H else None) if gate_up
                else (t * 16 + r if t * 16 + r < N else None) for r in range(16)]
        for b in range(nk):
            for lane in range(32):
                gg, tt = lane // 4, lane % 4
                for ch in range(2):
                    for r in range(2):
                        k, row = b * 64 + ch * 32 + tt * 8, rows[gg + 8 * r]
                        e = [8] * 8 if k >= K or row is None else [int(v) for v in q[row, k:k + 8]]
                        word = 0
                        for at, el in enumerate((0, 4, 2, 6, 1, 5, 3, 7)):
                            word |= e[el] << (4 * at)
                        at = lane * 16 + (2 * ch + r) * 4
                        out[t, b, at:at + 4] = np.frombuffer(np.uint32(word).tobytes(), np.uint8)
            for h in range(sets):
                for slot in range(16):
                    row, gr = rows[slot // 2 + 8 * (slot % 2)], (b * 64 + h * 32) // group
                    inside = row is not None and gr < s.shape[1]
                    at = 512 + (h * 16 + slot) * 2
                    v = s[row, gr] if inside else np.uint16(0)
                    out[t, b, at:at + 2] = np.frombuffer(np.uint16(v).tobytes(), np.uint8)
                    if z is not None:
                        out[t, b, 512 + 32 * sets + h * 16 + slot] = z[row, gr] if inside else 8
    return out.reshape(-1)


@pytest.mark.parametrize("dtn,N,K,group,zeros,gate_up", [
    ("bf16", 16, 64, 128, False, False), ("f16", 21, 72, 32, True, False),
    ("bf16", 48, 200, 64, True, True), ("f16", 32, 136, 32, False, True),
    ("bf16", 1, 8, 128, False, False)])
def test_pack_layout_and_unpack(dtn, N, K, group, zeros, gate_up):
    c, s, z = codes(gen(N + K), (), N, K, group, zeros, DT[dtn])
    W = api.swiglu_mlp_w4_pack(c, s, z, group, gate_up)
    want = pack_ref(c.cpu().numpy(), s.cpu().view(torch.int16).numpy().view(np.uint16),
                    None if z is None else z.cpu().numpy(), group, gate_up)
    assert np.array_equal(W.packed.cpu().numpy(), want)
    assert torch.equal(api.swiglu_mlp_w4_unpack(W), weights64(c, s, z, group).to(DT[dtn]))


def test_pack_and_unpack_of_experts():
    c, s, z = codes(gen(1), (3,), 24, 88, 64, True, torch.bfloat16)
    W = api.swiglu_mlp_w4_pack(c, s, z, 64)
    one = [api.swiglu_mlp_w4_pack(c[e], s[e], z[e], 64).packed for e in range(3)]
    assert torch.equal(W.packed, torch.cat(one)) and W.shape == (3, 24, 88)
    assert torch.equal(api.swiglu_mlp_w4_unpack(W), weights64(c, s, z, 64).to(torch.bfloat16))


# ---------------------------------------------------------------------------
# 4-bit products
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtn,M,N,K,group,zeros", [
    ("bf16", 1, 1, 8, 128, False), ("f16", 1, 15, 64, 32, True), ("bf16", 2, 16, 72, 32, False),
    ("bf16", 7, 250, 520, 64, True), ("f16", 8, 4096, 1032, 128, True),
    ("bf16", 8, 2500, 4096, 128, False), ("f16", 9, 33, 2056, 32, True),
    ("bf16", 13, 1000, 11008, 128, False), ("f16", 16, 5000, 640, 64, False),
    ("bf16", 17, 47, 136, 32, True), ("f16", 33, 700, 2816, 128, False),
    ("bf16", 64, 5632, 2048, 64, True), ("f16", 64, 100, 5632, 32, False),
    ("bf16", 5, 40000, 64, 64, False), ("bf16", 29, 8208, 4104, 32, True),
    ("f16", 25, 16400, 2056, 128, False), ("bf16", 40, 70001, 72, 64, True),
    ("f16", 50, 20000, 1096, 64, False)])
def test_w4_linear(dtn, M, N, K, group, zeros):
    g = gen(M * 7 + N)
    w = codes(g, (), N, K, group, zeros, DT[dtn])
    X = normal(g, M, K, dtype=DT[dtn])
    X[0, : K // 2] *= 30.0  # unlike magnitudes in one row
    Y = api.swiglu_mlp_w4_linear(X, api.swiglu_mlp_w4_pack(*w, group))
    near(Y, X.double() @ weights64(*w, group).T, U[dtn] + SLACK)


@pytest.mark.parametrize("dtn,M,D,H,group,zeros,muls", [
    ("bf16", 1, 64, 176, 128, False, (1.0, 1.0)), ("f16", 3, 72, 40, 32, True, (1.0, 1.0)),
    ("bf16", 6, 2048, 5632, 64, True, (1.0, 1.0)), ("f16", 8, 1024, 2816, 128, False, (0.5, 2.0)),
    ("bf16", 11, 264, 1416, 32, False, (1.25, 0.75)), ("f16", 40, 520, 1032, 128, True, (1.0, 1.0)),
    ("bf16", 64, 1024, 2816, 128, False, (1.0, 1.0))])
def test_w4_mlp(dtn, M, D, H, group, zeros, muls):
    g = gen(M + D + H)
    gu, dn = codes(g, (), 2 * H, D, group, zeros, DT[dtn]), codes(g, (), D, H, group, zeros, DT[dtn])
    X = normal(g, M, D, dtype=DT[dtn])
    Y, A = api.swiglu_mlp_fwd_nograd_w4(X, api.swiglu_mlp_w4_pack(*gu, group, gate_up=True),
                                        api.swiglu_mlp_w4_pack(*dn, group), gate_mul=muls[0],
                                        down_mul=muls[1])
    near(A, hidden64(X.double(), weights64(*gu, group), muls[0]), U[dtn] + 4 * SLACK)
    near(Y, muls[1] * (A.double() @ weights64(*dn, group).T), U[dtn] + SLACK)  # on the stored A


@pytest.mark.parametrize("M", [12, 45])
def test_w4_zero_tokens_and_non_finite_tokens(M):
    g = gen(3)
    w = codes(g, (), 48, 128, 64, True, torch.bfloat16)
    W = api.swiglu_mlp_w4_pack(*w, 64)
    assert api.swiglu_mlp_w4_linear(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), W).shape == (0, 48)
    X = normal(g, M, 128, dtype=torch.bfloat16)
    clean = api.swiglu_mlp_w4_linear(X, W)
    X[3, 5], X[9, 100] = float("nan"), float("inf")
    Y = api.swiglu_mlp_w4_linear(X, W)
    assert torch.isnan(Y[3]).all() and not torch.isfinite(Y[9]).any()
    keep = [i for i in range(M) if i not in (3, 9)]  # no token reaches another
    assert torch.equal(Y[keep], clean[keep])


# ---------------------------------------------------------------------------
# mixture of experts
# ---------------------------------------------------------------------------
def route64(X, Wr, k, norm, scale):
    p = torch.softmax(X.double() @ Wr.double().T, 1)
    lg = X.double() @ Wr.double().T
    idx = torch.sort(lg, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, idx)
    return idx, scale * (w / w.sum(1, keepdim=True) if norm else w)


@pytest.mark.parametrize("dtn", ["bf16", "f16"])
@pytest.mark.parametrize("T,D,E,k,norm,scale", [
    (1, 64, 8, 2, True, 1.0), (1, 8, 1, 1, True, 1.0), (5, 72, 3, 3, False, 1.0),
    (8, 2048, 64, 8, True, 2.5), (9, 136, 65, 16, False, 0.5), (64, 264, 130, 4, True, 1.0),
    (33, 4096, 512, 6, False, 1.0)])
def test_route(dtn, T, D, E, k, norm, scale):
    # small whole numbers: the logits are exact in 32 bits in any order, so the
    # choice, with its many ties, is too
    g = gen(T + E)
    X = torch.randint(-3, 4, (T, D), generator=g, device="cuda").to(DT[dtn])
    Wr = (torch.randint(-2, 3, (E, D), generator=g, device="cuda") / 16).to(DT[dtn])
    if E > 2:
        Wr[E - 1] = Wr[1]  # ties: the lower index first
    idx, w = api.swiglu_mlp_moe_route(X, Wr, k, norm, scale)
    ri, rw = route64(X, Wr, k, norm, scale)
    assert torch.equal(idx.long(), ri)
    # expf and the division: a few units in the last place, sums of E terms
    assert bool(((w.double() - rw).abs() <= 2.0 ** -19 * rw + 1e-37).all())


def test_route_nan_and_order():
    X = torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
    X[1, 7] = float("nan")
    Wr = torch.arange(8, device="cuda")[:, None].expand(8, 64).contiguous().to(torch.bfloat16) / 64
    idx, w = api.swiglu_mlp_moe_route(X, Wr, 3)
    assert idx[0].tolist() == idx[2].tolist() == [7, 6, 5]
    assert torch.isnan(w[1]).all() and torch.isfinite(w[[0, 2]]).all()
    i = idx[1].tolist()
    assert len(set(i)) == 3 and all(0 <= e < 8 for e in i)


def experts64(X, idx, w, gu, dn, dtype, gm=1.0, dm=1.0):
    """sum_j w MLP(x), the hidden values rounded to the type; gu, dn: a
    function of the expert's number."""
    y = torch.zeros(X.shape, dtype=torch.float64, device=X.device)
    for e in idx.unique().tolist():
        if not 0 <= e < 1 << 20:
            continue
        at, slot = (idx == e).nonzero(as_tuple=True)
        wgu, wd = gu(e), dn(e)
        if wgu is None:
            continue
        a = hidden64(X[at].double(), wgu, gm).to(dtype).double()
        y.index_put_((at,), dm * w[at, slot].double()[:, None] * (a @ wd.T), accumulate=True)
    return y


FMT = [None, (128, False), (32, True), (64, False)]


def expert_weights(g, E, D, H, fmt, dtype):
    """(Wgu, Wd) as the operators take them, and the matrices in 64 bits."""
    if fmt is None:
        wgu, wd = normal(g, E, 2 * H, D, std=D ** -0.5, dtype=dtype), normal(g, E, D, H, std=H ** -0.5, dtype=dtype)
        return (wgu, wd), lambda e: wgu[e].double(), lambda e: wd[e].double()
    group, zeros = fmt
    gu, dn = codes(g, (E,), 2 * H, D, group, zeros, dtype), codes(g, (E,), D, H, group, zeros, dtype)
    one = lambda t, e: [v if v is None else v[e] for v in t]
    return ((api.swiglu_mlp_w4_pack(*gu, group, gate_up=True), api.swiglu_mlp_w4_pack(*dn, group)),
            lambda e: weights64(*one(gu, e), group), lambda e: weights64(*one(dn, e), group))


@pytest.mark.parametrize("dtn,T,D,H,E,k,fmt", [
    ("bf16", 1, 64, 32, 1, 1, 0), ("f16", 1, 72, 40, 5, 5, 1), ("bf16", 1, 1024, 2816, 8, 2, 0),
    ("bf16", 2, 136, 520, 27, 3, 2), ("f16", 4, 520, 264, 16, 8, 3), ("bf16", 7, 1032, 1416, 27, 3, 3),
    ("f16", 16, 256, 128, 64, 8, 0), ("bf16", 16, 2048, 512, 64, 8, 1), ("f16", 33, 264, 72, 9, 4, 2),
    ("bf16", 64, 512, 264, 4, 2, 0), ("f16", 64, 520, 136, 4, 3, 1), ("bf16", 64, 1024, 256, 130, 6, 2),
    ("f16", 64, 128, 64, 512, 16, 0)])
def test_moe_layer(dtn, T, D, H, E, k, fmt):
    g, dt = gen(T * E + H), DT[dtn]
    (Wgu, Wd), gu, dn = expert_weights(g, E, D, H, FMT[fmt], dt)
    X, Wr = normal(g, T, D, dtype=dt), normal(g, E, D, std=2 * D ** -0.5, dtype=dt)
    Y, idx, w = api.swiglu_mlp_moe_fwd_nograd(X, Wr, Wgu, Wd, k, norm_topk=T % 2 == 0, route_scale=1.5,
                                              gate_mul=1.25, down_mul=0.5)
    ri, rw = api.swiglu_mlp_moe_route(X, Wr, k, T % 2 == 0, 1.5)
    assert torch.equal(idx, ri) and torch.equal(w, rw)
    near(Y, experts64(X, idx, w, gu, dn, dt, 1.25, 0.5), 2 * U[dtn] + SLACK)


@pytest.mark.parametrize("fmt", [0, 2])
@pytest.mark.parametrize("T,k", [(1, 2), (6, 4), (8, 16), (40, 3), (64, 16)])
def test_experts_with_given_assignments(fmt, T, k):
    # none at all, some of no expert, one expert for everybody, an expert
    # named twice by one token
    g, E, D, H, dt = gen(T * k), 16, 200, 88, torch.bfloat16
    (Wgu, Wd), gu, dn = expert_weights(g, E, D, H, FMT[fmt], dt)
    X = normal(g, T, D, dtype=dt)
    w = torch.rand(T, k, generator=g, device="cuda")
    idx = torch.randint(-2, E + 2, (T, k), generator=g, device="cuda", dtype=torch.int32)
    cases = [torch.full_like(idx, -1), idx, torch.full_like(idx, 3), idx % 3]
    for i in cases:
        Y = api.swiglu_mlp_moe_experts(X, i, w, Wgu, Wd)
        ref = experts64(X, torch.where((i < 0) | (i >= E), torch.full_like(i, 1 << 20), i), w, gu, dn, dt)
        near(Y, ref, 2 * U["bf16"] + SLACK)
        empty = ((i < 0) | (i >= E)).all(1)
        assert torch.equal(Y[empty], torch.zeros_like(Y[empty]))


@pytest.mark.parametrize("fmt", [None, (128, False)])
def test_experts_beyond_two_gigabytes(fmt):
    # the last expert's weights lie past 2^32 bytes (4-bit: past 2^31)
    E, D, H, dt = 33, 4096, 8192, torch.bfloat16
    g = gen(9)
    if fmt is None:
        Wgu = torch.zeros(E, 2 * H, D, dtype=dt, device="cuda")
        Wd = torch.zeros(E, D, H, dtype=dt, device="cuda")
        Wgu[-1], Wd[-1] = normal(g, 2 * H, D, std=D ** -0.5, dtype=dt), normal(g, D, H, std=H ** -0.5, dtype=dt)
        gu, dn = (lambda e: Wgu[e].double()), (lambda e: Wd[e].double())
    else:
        E *= 2
        one = [codes(g, (), 2 * H, D, 128, False, dt), codes(g, (), D, H, 128, False, dt)]
        packs = []
        for (c, s, _), pair in zip(one, (True, False)):
            C = torch.full((E, *c.shape), 0x88, dtype=torch.uint8, device="cuda")
            S = torch.zeros(E, *s.shape, dtype=dt, device="cuda")
            C[-1], S[-1] = c, s
            packs.append(api.swiglu_mlp_w4_pack(C, S, None, 128, gate_up=pair))
        Wgu, Wd = packs
        gu, dn = (lambda e: weights64(*one[0], 128)), (lambda e: weights64(*one[1], 128))
    X = normal(g, 2, D, dtype=dt)
    idx = torch.tensor([[E - 1], [E - 1]], dtype=torch.int32, device="cuda")
    w = torch.ones(2, 1, device="cuda")
    near(api.swiglu_mlp_moe_experts(X, idx, w, Wgu, Wd), experts64(X, idx, w, gu, dn, dt),
         2 * U["bf16"] + SLACK)


# ---------------------------------------------------------------------------
# how they are called
# ---------------------------------------------------------------------------
def make_calls(T=6, seed=0):
    """Each operator as a function of nothing, on buffers of its own."""
    g, dt = gen(seed), torch.bfloat16
    D, H, E, k = 264, 200, 12, 3
    X, Wr = normal(g, T, D, dtype=dt), normal(g, E, D, std=2 * D ** -0.5, dtype=dt)
    dev, new = X.device, lambda *s, d=dt: torch.full(s, float("nan") if d.is_floating_point else -7, dtype=d, device="cuda")
    lin = api.swiglu_mlp_w4_pack(*codes(g, (), 333, D, 64, True, dt), 64)
    gu = api.swiglu_mlp_w4_pack(*codes(g, (), 2 * H, D, 32, False, dt), 32, gate_up=True)
    dn = api.swiglu_mlp_w4_pack(*codes(g, (), D, H, 32, False, dt), 32)
    (e16, _, _), (e4, _, _) = expert_weights(g, E, D, H, None, dt), expert_weights(g, E, D, H, (128, False), dt)
    o1 = {"Y": new(T, 333)}
    o2 = {"Y": new(T, D), "A": new(T, H)}
    outs = [{"Y": new(T, D), "idx": new(T, k, d=torch.int32), "weights": new(T, k, d=torch.float32)} for _ in range(2)]
    w1, w2 = api.w4_linear_workspace(T, 333, D, dev), api.w4_workspace(T, D, H, dev)
    w3 = [api.moe_workspace(T, D, H, E, k, dev) for _ in range(2)]
    return X, {
        "w4_linear": (lambda: api.swiglu_mlp_w4_linear(X, lin, out=o1, ws=w1), o1, w1),
        "w4_mlp": (lambda: api.swiglu_mlp_fwd_nograd_w4(X, gu, dn, out=o2, ws=w2), o2, w2),
        "moe": (lambda: api.swiglu_mlp_moe_fwd_nograd(X, Wr, *e16, k, out=outs[0], ws=w3[0]), outs[0], w3[0]),
        "moe_w4": (lambda: api.swiglu_mlp_moe_fwd_nograd(X, Wr, *e4, k, out=outs[1], ws=w3[1]), outs[1], w3[1]),
    }


OPS = ["w4_linear", "w4_mlp", "moe", "moe_w4"]


def snap(out):
    return {k: v.clone() for k, v in out.items()}


def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("T", [1, 6, 20, 41])
def test_deterministic_and_workspace_reusable(op, T):
    _, calls = make_calls(T)
    call, out, ws = calls[op]
    call()
    torch.cuda.synchronize()
    first = snap(out)
    assert all(not v.is_floating_point() or torch.isfinite(v).all() for v in first.values())
    ws[256 + 4096:].fill_(0xff)  # past the header and the counters: what an earlier call may leave
    for _ in range(20):
        call()
    assert same(snap(out), first)
    assert api.swiglu_mlp_query_error(ws) == 0


@pytest.mark.parametrize("op", OPS)
def test_back_to_back_calls_on_changing_inputs(op):
    # launches overlap: no call may read what the one before it still writes,
    # nor see inputs before the copy that precedes it
    X, calls = make_calls(5)
    call, out, _ = calls[op]
    xs = [normal(gen(50 + i), *X.shape, dtype=X.dtype) for i in range(4)]
    want = []
    for x in xs:
        X.copy_(x)
        call()
        torch.cuda.synchronize()
        want.append(snap(out))
    got = []
    for _ in range(10):
        for x in xs:
            X.copy_(x)
            call()
            got.append(snap(out))
    torch.cuda.synchronize()
    assert all(same(o, want[i % 4]) for i, o in enumerate(got))


@pytest.mark.parametrize("op", OPS)
def test_side_stream_and_graph(op):
    X, calls = make_calls(3)
    call, out, _ = calls[op]
    call()
    torch.cuda.synchronize()
    first = snap(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for v in out.values():
            v.zero_()
        call()
        got = snap(out)
    s.synchronize()
    assert same(got, first)
    if api._use_debug:
        return  # the binding waits for every call of the debug build, which a capture forbids
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    x0 = X.clone()
    X.mul_(-1)
    graph.replay()
    X.copy_(x0)
    for v in out.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert same(snap(out), first)


@pytest.mark.parametrize("op", OPS)
def test_writes_stay_in_the_outputs(op):
    _, calls = make_calls(7)
    call, out, _ = calls[op]
    guarded = {}
    for k, v in list(out.items()):
        pad = 256 // v.element_size()
        big = torch.full((v.numel() + 2 * pad,), 77, dtype=v.dtype, device="cuda")
        out[k] = big[pad:pad + v.numel()].view(v.shape)
        guarded[k] = (big, pad)
    call()
    torch.cuda.synchronize()
    for k, (big, pad) in guarded.items():
        assert bool((big[:pad] == 77).all()) and bool((big[-pad:] == 77).all()), k


def test_out_and_inputs_are_checked():
    g = gen(1)
    W = api.swiglu_mlp_w4_pack(*codes(g, (), 32, 64, 64, False, torch.bfloat16), 64)
    X = normal(g, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.swiglu_mlp_w4_linear(X, W, out={"Y": torch.empty(4, 31, dtype=X.dtype, device="cuda")})
    with pytest.raises(ValueError):
        api.swiglu_mlp_w4_linear(X, W, out={"Y": torch.empty(4, 32, device="cuda")})
    with pytest.raises(ValueError):
        api.swiglu_mlp_w4_linear(normal(g, 4, 128, dtype=X.dtype)[:, ::2], W)
    with pytest.raises(api.SwigluError) as e:
        api.swiglu_mlp_w4_linear(normal(g, 65, 64, dtype=X.dtype), W)
    assert e.value.code == 3
    with pytest.raises(api.SwigluError) as e:
        api.swiglu_mlp_w4_linear(X, W, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 4
    with pytest.raises(ValueError):
        api.swiglu_mlp_w4_pack(*codes(g, (), 32, 64, 64, False, X.dtype)[:2], group=32)


@pytest.mark.parametrize("T", [4, 41])
@pytest.mark.parametrize("op", OPS)
def test_a_wait_that_runs_out_is_reported(op, T):
    # a copy that is never made: the wait gives up at its limit, the status
    # says so, and the next call is right again
    _, calls = make_calls(T)
    call, out, ws = calls[op]
    call()
    torch.cuda.synchronize()
    first = snap(out)
    old = api.swiglu_mlp_set_wait_limit_ns(2_000_000)
    try:
        api.swiglu_mlp_inject_stall_once()
        try:
            call()
            code = api.swiglu_mlp_query_error(ws)
        except api.SwigluError as e:  # the binding checks every call of the debug build
            code = e.code
        assert code == 6
    finally:
        api.swiglu_mlp_inject_stall_once(False)
        api.swiglu_mlp_set_wait_limit_ns(old)
    call()
    assert api.swiglu_mlp_query_error(ws) == 0 and same(snap(out), first)


@pytest.mark.parametrize("T", [9, 41])
@pytest.mark.parametrize("op", OPS)
def test_debug_build(op, T):
    prev = api.use_debug_library(True)
    try:
        _, calls = make_calls(T)
        call, out, ws = calls[op]
        call()  # raises on a failed index check
        first = snap(out)
        api.lib().swiglu_mlp_debug_narrow_once(1)
        with pytest.raises(api.SwigluError) as e:
            call()
        assert e.value.code == 7
        call()
        assert same(snap(out), first)
    finally:
        api.lib().swiglu_mlp_debug_narrow_once(0)
        api.use_debug_library(prev)


def test_launch_counts_and_kernel_times():
    _, calls = make_calls(4)
    for op, n in (("w4_linear", 1), ("w4_mlp", 2), ("moe", 3), ("moe_w4", 3)):
        calls[op][0]()
        assert api.swiglu_mlp_last_launch_count() == n
    torch.cuda.synchronize()
    api.swiglu_mlp_profile_read()
    api.swiglu_mlp_profile_enable(True)
    try:
        for op in OPS:
            calls[op][0]()
    finally:
        api.swiglu_mlp_profile_enable(False)
    got = api.swiglu_mlp_profile_read()
    for name in ("w4_linear", "w4_gate_up", "w4_down", "moe_gate_up", "moe_down", "moe_w4_gate_up",
                 "moe_w4_down"):
        assert got[name][0] == 1 and got[name][1] > 0
    assert got["moe_route"][0] == 2


# ---------------------------------------------------------------------------
# modules
# ---------------------------------------------------------------------------
@torch.no_grad()
def test_w4_module():
    torch.manual_seed(0)
    mlp = SwiGLUMLP(264, 520, device="cuda", gate_multiplier=1.5)
    m = W4SwiGLUMLP(mlp, group=32, zeros=True)
    x = torch.randn(2, 3, 264, device="cuda", dtype=torch.bfloat16)
    gu, dn = (api.swiglu_mlp_w4_unpack(w) for w in (m.gate_up, m.down))
    y = m(x)
    ref, _ = api.swiglu_mlp_fwd_nograd(x.reshape(-1, 264), gu, dn, gate_mul=1.5)
    # the unpacked weights are rounded to the type, the 4-bit products' are not
    assert float((y.reshape(-1, 264) - ref).float().norm() / ref.float().norm()) <= 4 * U["bf16"]
    many = torch.randn(80, 264, device="cuda", dtype=torch.bfloat16)
    assert torch.equal(m(many), api.swiglu_mlp_fwd_nograd(many, gu, dn, gate_mul=1.5)[0])
    # 4 bits with zero points keep a uniform weight to 1 / 30 of its group's range
    full = mlp(x)
    assert float((y - full).float().norm() / full.float().norm()) <= 0.25
    same_m = W4SwiGLUMLP.from_codes(api.swiglu_mlp_w4_quantize(mlp.gate_up_weight, 32, True),
                                    api.swiglu_mlp_w4_quantize(mlp.down_weight, 32, True), 32, 1.5)
    assert torch.equal(same_m(x), y)


@torch.no_grad()
def test_moe_module():
    torch.manual_seed(1)
    m = MoESwiGLU(200, 136, 10, 3, device="cuda", dtype=torch.float16)
    x = torch.randn(70, 200, device="cuda", dtype=torch.float16)  # more than one call's tokens
    y = m(x)
    idx, w = api.swiglu_mlp_moe_route(x[:64], m.router_weight, 3)
    ref = experts64(x[:64], idx, w, lambda e: m.gate_up_weight[e].double(),
                    lambda e: m.down_weight[e].double(), torch.float16)
    near(y[:64], ref, 2 * U["f16"] + SLACK)
    assert torch.equal(y[64:], m(x[64:]))
    m.quantize(group=64)
    q = m(x)
    assert m.gate_up_weight is None and float((q - y).float().norm() / y.float().norm()) <= 0.5
    with pytest.raises(RuntimeError):
        m.quantize()
