"""Few-token serving operators of the SwiGLU MLP, as cases that can be timed
and compared: products with 4-bit weights and group scales, the whole MLP on
such weights, and a mixture-of-experts layer (router, top-k, experts, weighted
sum) with 16-bit or 4-bit experts.

``run`` computes a case either with the library's operators (``own`` true) or
in their plain form, elementary torch operations in 32 bits (``own`` false);
``exact`` computes it from the definition in 64 bits.

4-bit weights: ``codes`` uint8 [.., N, K/2] hold two codes of 0..15 per byte
(the even k in the low half), ``scales`` [.., N, ceil(K/group)] one scale per
run of ``group`` consecutive k, ``zeros`` uint8 of the scales' shape or None
(8 everywhere); the weight is scale * (code - zero).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one token through a projection of the smallest training layer of the bench: pure latency
        dict(name="w4_linear_1_small", op="w4_linear", M=1, N=2816, K=1024, group=128, zeros=False, dtype="bf16"),
        # one decoded token through a projection of the bench's main layer
        dict(name="w4_linear_1", op="w4_linear", M=1, N=11008, K=4096, group=128, zeros=False, dtype="bf16"),
        # a ragged small batch on a checkpoint with zero points and small groups; the last group is a part of one
        dict(name="w4_linear_13_ragged", op="w4_linear", M=13, N=5641, K=2056, group=32, zeros=True, dtype="f16"),
        # one decoded token through the bench's main layer
        dict(name="w4_mlp_1", op="w4_mlp", M=1, D=4096, H=11008, group=128, zeros=False, dtype="bf16"),
        # a few streams through the middle layer, zero points
        dict(name="w4_mlp_6", op="w4_mlp", M=6, D=2048, H=5632, group=64, zeros=True, dtype="f16"),
        # the few-token path's full batch
        dict(name="w4_mlp_64", op="w4_mlp", M=64, D=4096, H=11008, group=128, zeros=False, dtype="bf16"),
        # one decoded token, few large experts
        dict(name="moe_1_of_8", op="moe", T=1, D=1024, H=2816, E=8, k=2, norm=True, dtype="bf16"),
        # a small batch over many small experts
        dict(name="moe_16_of_64", op="moe", T=16, D=2048, H=1024, E=64, k=8, norm=True, dtype="bf16"),
        # the full few-token batch: nearly every expert is read
        dict(name="moe_64_of_64", op="moe", T=64, D=2048, H=1024, E=64, k=8, norm=False, dtype="f16"),
        # one decoded token, 4-bit experts
        dict(name="moe_w4_1_of_64", op="moe_w4", T=1, D=2048, H=1024, E=64, k=8, norm=True, group=128, zeros=False, dtype="bf16"),
        # ragged sizes: last groups and last tiles are parts, an odd number of experts
        dict(name="moe_w4_7_ragged", op="moe_w4", T=7, D=1032, H=2824, E=27, k=3, norm=True, group=64, zeros=True, dtype="bf16"),
        # half a batch over many experts
        dict(name="moe_w4_32_of_128", op="moe_w4", T=32, D=2048, H=512, E=128, k=8, norm=False, group=32, zeros=False, dtype="f16"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A multiple of 8, spread over the logarithm of lo..hi."""
    n = max(lo, min(hi, _logint(rng, lo, hi) // 8 * 8))
    return n + 8 if n == 3072 else n


def _draw(rng):
    op = rng.choice(["w4_linear", "w4_mlp", "moe", "moe_w4"])
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]))
    if op == "w4_linear":
        c.update(M=_logint(rng, 1, 64), N=_logint(rng, 1024, 22016), K=_size(rng, 1024, 11008))
    elif op == "w4_mlp":
        c.update(M=_logint(rng, 1, 64), D=_size(rng, 1024, 4096), H=_size(rng, 1408, 11008))
    else:
        E = _logint(rng, 8, 128)
        c.update(T=_logint(rng, 1, 64), D=_size(rng, 1024, 4096), H=_size(rng, 512, 2816), E=E,
                 k=rng.randint(1, min(8, E // 2)), norm=rng.random() < 0.5)
    if c.get("N") == 3072:
        c["N"] = 3073
    if op != "moe":
        c.update(group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5)
    return c


def draw(rng):
    big = listed()
    most_b, most_f = max(work(c)["bytes"] for c in big), max(work(c)["flops"] for c in big)
    most_w = max(c["E"] * c["D"] * c["H"] for c in big if "E" in c)  # the plain form reads every expert
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= most_b and w["flops"] <= most_f and c.get("E", 1) * c.get("D", 1) * c.get("H", 1) <= most_w:
            return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(gen, shape, std, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _quantised(gen, lead, N, K, c):
    """A Gaussian weight matrix ([lead, N, K], variance 1/K) rounded to 4 bits by its groups' largest values
    (or, with zero points, by their ranges): codes, scales, zeros."""
    g, dt = c["group"], DTYPES[c["dtype"]]
    ng = -(-K // g)
    w = torch.randn((*lead, N, ng * g), generator=gen, device="cuda", dtype=torch.float32).mul_(K ** -0.5)
    w[..., K:] = 0
    w = w.reshape(*lead, N, ng, g)
    if c["zeros"]:
        lo, hi = w.amin(-1, keepdim=True).clamp_(max=0), w.amax(-1, keepdim=True).clamp_(min=0)
        s = ((hi - lo) / 15).to(dt)
        z = (-lo / s.float()).round_().clamp_(0, 15)
    else:
        s = (w.abs().amax(-1, keepdim=True) / 7).to(dt)
        z = torch.full_like(s, 8, dtype=torch.float32)
    q = (w / s.float()).round_().add_(z).clamp_(0, 15).to(torch.uint8).reshape(*lead, N, ng * g)[..., :K]
    codes = (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous()
    return codes, s.squeeze(-1).contiguous(), z.squeeze(-1).to(torch.uint8).contiguous() if c["zeros"] else None


def _inputs(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "w4_linear":
        return dict(X=_normal(gen, (c["M"], c["K"]), 1.0, dt), W=_quantised(gen, (), c["N"], c["K"], c))
    D, H = c["D"], c["H"]
    if c["op"] == "w4_mlp":
        return dict(X=_normal(gen, (c["M"], D), 1.0, dt), Wgu=_quantised(gen, (), 2 * H, D, c), Wd=_quantised(gen, (), D, H, c))
    T, E, k = c["T"], c["E"], c["k"]
    Wr = _normal(gen, (E, D), 1.5 * D ** -0.5, dt)
    # A token whose k-th and next scores differ by less than 32-bit sums can tell apart has no one right choice of
    # experts: of four candidates for each token the first with a clear choice is taken.
    cand = _normal(gen, (4, T, D), 1.0, dt)
    top = torch.sort((cand.double() @ Wr.double().T), dim=-1, descending=True).values
    gaps = (top[..., :-1] - top[..., 1:])[..., :k].amin(-1)  # the order of the chosen ones counts too
    clear = (gaps > 1e-4).to(torch.float32) * torch.tensor([4.0, 3.0, 2.0, 1.0], device="cuda")[:, None]
    X = cand[clear.argmax(0), torch.arange(T, device="cuda")].contiguous()
    s = dict(X=X, Wr=Wr)
    if c["op"] == "moe":
        s.update(Wgu=_normal(gen, (E, 2 * H, D), D ** -0.5, dt), Wd=_normal(gen, (E, D, H), H ** -0.5, dt))
    else:
        s.update(Wgu=_quantised(gen, (E,), 2 * H, D, c), Wd=_quantised(gen, (E,), D, H, c))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        # what a serving program keeps: the weights in the library's 4-bit layout, a workspace, output buffers
        from backward_tcgen05_tma_gb300 import api

        X, dt = s["X"], s["X"].dtype
        dev, new = X.device, lambda *n, d=dt: torch.empty(*n, dtype=d, device=X.device)
        if case["op"] == "w4_linear":
            s["own_W"] = api.swiglu_mlp_w4_pack(*s["W"], group=case["group"])
            s["ws"] = api.w4_linear_workspace(case["M"], case["N"], case["K"], dev)
            s["out"] = {"Y": new(case["M"], case["N"])}
        else:
            D, H = case["D"], case["H"]
            if case["op"] == "moe":
                s["own_W"] = s["Wgu"], s["Wd"]
            else:
                s["own_W"] = (api.swiglu_mlp_w4_pack(*s["Wgu"], group=case["group"], gate_up=True),
                              api.swiglu_mlp_w4_pack(*s["Wd"], group=case["group"]))
            if case["op"] == "w4_mlp":
                s["ws"] = api.w4_workspace(case["M"], D, H, dev)
                s["out"] = {"Y": new(case["M"], D), "A": new(case["M"], H)}
            else:
                T, k = case["T"], case["k"]
                s["ws"] = api.moe_workspace(T, D, H, case["E"], k, dev)
                s["out"] = {"Y": new(T, D), "idx": new(T, k, d=torch.int32), "weights": new(T, k, d=torch.float32)}
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _dequantised(W, group):
    codes, scales, zeros = W
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).float()
    K = q.shape[-1]
    if zeros is None:
        q = q - 8
    else:
        q = q - zeros.float().repeat_interleave(group, -1)[..., :K]
    return q * scales.float().repeat_interleave(group, -1)[..., :K]


def _swiglu(gu):
    g, u = gu.chunk(2, dim=-1)
    return g / (1 + torch.exp(-g)) * u


def _plain(s):
    c, X = s["case"], s["X"]
    dt, x = X.dtype, X.float()
    if c["op"] == "w4_linear":
        return (x @ _dequantised(s["W"], c["group"]).T).to(dt)
    if c["op"] == "w4_mlp":
        a = _swiglu(x @ _dequantised(s["Wgu"], c["group"]).T)
        return (a @ _dequantised(s["Wd"], c["group"]).T).to(dt), a.to(dt)
    T, E, k = c["T"], c["E"], c["k"]
    logits = x @ s["Wr"].float().T
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    e = torch.exp(top - top[:, :1])
    w = e[:, :k] / (e[:, :k] if c["norm"] else e).sum(1, keepdim=True)
    idx = idx[:, :k]
    pick = idx.flatten() if T * k <= E else slice(None)  # gather the chosen experts, or take all of them
    if c["op"] == "moe":
        wgu, wd = s["Wgu"][pick].float(), s["Wd"][pick].float()
    else:
        wgu, wd = (_dequantised([t if t is None else t[pick] for t in s[n]], c["group"]) for n in ("Wgu", "Wd"))
    if T * k <= E:
        xs = x.repeat_interleave(k, 0)[:, :, None]
        y = wd @ _swiglu((wgu @ xs)[:, :, 0])[:, :, None]
        y = y[:, :, 0].reshape(T, k, -1)
    else:
        y = _swiglu(x @ wgu.transpose(1, 2)) @ wd.transpose(1, 2)  # [E, T, D]
        y = y[idx, torch.arange(T, device=x.device)[:, None]]
    return (w[:, :, None] * y).sum(1).to(dt), idx.to(torch.int32), w


def run(state):
    if not own:
        return _plain(state)
    from backward_tcgen05_tma_gb300 import api

    c, op = state["case"], state["case"]["op"]
    if op == "w4_linear":
        return api.swiglu_mlp_w4_linear(state["X"], state["own_W"], out=state["out"], ws=state["ws"])
    Wgu, Wd = state["own_W"]
    if op == "w4_mlp":
        return api.swiglu_mlp_fwd_nograd_w4(state["X"], Wgu, Wd, out=state["out"], ws=state["ws"])
    return api.swiglu_mlp_moe_fwd_nograd(state["X"], state["Wr"], Wgu, Wd, c["k"], norm_topk=c["norm"], out=state["out"],
                                         ws=state["ws"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _matrix_bytes(N, K, c):
    if "group" not in c:
        return 2 * N * K
    return N * K // 2 + N * -(-K // c["group"]) * (3 if c["zeros"] else 2)


def work(case):
    c = case
    if c["op"] == "w4_linear":
        return {"bytes": _matrix_bytes(c["N"], c["K"], c) + 2 * c["M"] * (c["K"] + c["N"]), "flops": 2 * c["M"] * c["N"] * c["K"]}
    D, H = c["D"], c["H"]
    layer = _matrix_bytes(2 * H, D, c) + _matrix_bytes(D, H, c)
    if c["op"] == "w4_mlp":
        return {"bytes": layer + 2 * c["M"] * (2 * D + H), "flops": 6 * c["M"] * D * H}
    T, E, k = c["T"], c["E"], c["k"]
    read = E * (1 - (1 - k / E) ** T)  # experts that some token chose, on average
    return {"bytes": int(read * layer) + 2 * E * D + 4 * T * D + 8 * T * k, "flops": 2 * T * D * E + 6 * T * k * D * H}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------
def _weights64(codes, scales, zeros, group):
    n, half = codes.shape
    w = torch.empty(n, 2 * half, dtype=torch.float64, device=codes.device)
    w[:, 0::2] = codes.bitwise_and(15).double()
    w[:, 1::2] = codes.div(16, rounding_mode="floor").double()
    for i in range(scales.shape[1]):
        part = w[:, i * group:(i + 1) * group]
        part -= 8.0 if zeros is None else zeros[:, i:i + 1].double()
        part *= scales[:, i:i + 1].double()
    return w


def _mlp64(x, wgu, wd):
    h = wd.shape[1]
    g = x @ wgu[:h].T
    a = g * torch.sigmoid(g) * (x @ wgu[h:].T)
    return a @ wd.T, a


def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    x = s["X"].double()
    if c["op"] == "w4_linear":
        return x @ _weights64(*s["W"], c["group"]).T
    if c["op"] == "w4_mlp":
        return _mlp64(x, _weights64(*s["Wgu"], c["group"]), _weights64(*s["Wd"], c["group"]))
    p = torch.softmax(x @ s["Wr"].double().T, dim=1)
    w, idx = torch.topk(p, c["k"], dim=1)
    if c["norm"]:
        w = w / w.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for e in idx.unique().tolist():
        at, slot = (idx == e).nonzero(as_tuple=True)
        if c["op"] == "moe":
            wgu, wd = s["Wgu"][e].double(), s["Wd"][e].double()
        else:
            wgu, wd = (_weights64(*(t if t is None else t[e] for t in s[n]), c["group"]) for n in ("Wgu", "Wd"))
        y[at] += w[at, slot][:, None] * _mlp64(x[at], wgu, wd)[0]
    return y, idx.to(torch.int32), w
