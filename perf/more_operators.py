"""The operators around an MLP in a transformer block, as cases that can be
timed and compared: layer norm (with the residual sum in front of it) and its
backward pass with the reduction of the weight's gradient; and a matrix
product with bias, activation and residual in its epilogue, and its backward
pass.

``run`` computes a case either with the library's operators (``own`` true) or
in their plain form, elementary torch operations in 32 bits (``own`` false);
``exact`` computes it from the definition in 64 bits.

    layer norm   S = rnd(X + R) or X,  Y = (S - mean) rstd * weight + bias over the last dimension
                 backward: dX (plus the gradient dS that comes by the residual stream), dweight, dbias
    linear       z = X W^T + bias,  Y = act(z) + R,  Z = z where it is kept for the backward pass
                 backward: dZ = dY act'(Z),  dX = dZ W,  dW = dZ^T X,  dbias = column sums of dZ;
                 with x_act, X is x_act(Xpre) and dX becomes the gradient of Xpre
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-5


def listed():
    return [
        # the norm in front of one decoded token's MLP, smallest training layer of the bench: pure latency
        dict(name="ln_fwd_1", op="ln_fwd", M=1, D=1024, residual=True, dtype="bf16"),
        # a ragged evaluation batch in fp32
        dict(name="ln_fwd_1531_f32", op="ln_fwd", M=1531, D=2056, residual=False, dtype="f32"),
        # a training step's forward norm in front of the bench's main layer, the residual sum with it
        dict(name="ln_fwd_65536", op="ln_fwd", M=65536, D=4096, residual=True, dtype="bf16"),
        # a training step's backward norm of the smallest training layer
        dict(name="ln_bwd_16384", op="ln_bwd", M=16384, D=1024, residual=False, dtype="f16"),
        # the same of the main layer, the residual stream's gradient joined in
        dict(name="ln_bwd_65536", op="ln_bwd", M=65536, D=4096, residual=True, dtype="bf16"),
        # one decoded token through the first projection of the smallest layer: latency
        dict(name="linear_1", op="linear_fwd", M=1, N=2816, K=1024, act="silu", bias=True, residual=False, keep=False, dtype="bf16"),
        # a ragged small batch through a second projection: bias and residual, no activation
        dict(name="linear_13", op="linear_fwd", M=13, N=2056, K=5640, act="none", bias=True, residual=True, keep=False, dtype="f16"),
        # a full few-token batch through the main layer's first projection
        dict(name="linear_64", op="linear_fwd", M=64, N=11008, K=4096, act="gelu_tanh", bias=True, residual=False, keep=False, dtype="bf16"),
        # a training step's first projection, smallest layer: z is kept
        dict(name="linear_16384", op="linear_fwd", M=16384, N=2816, K=1024, act="gelu", bias=True, residual=False, keep=True, dtype="bf16"),
        # a ragged batch in fp32
        dict(name="linear_1999_f32", op="linear_fwd", M=1999, N=2824, K=1032, act="relu", bias=True, residual=True, keep=False, dtype="f32"),
        # a training step's backward pass of a projection with an activation, smallest layer
        dict(name="linear_bwd_16384", op="linear_bwd", M=16384, N=2816, K=1024, act="gelu", x_act="none", bias=True, dtype="f16"),
        # the backward pass of the middle layer's second projection, whose input is the first one's activation
        dict(name="linear_bwd_32768", op="linear_bwd", M=32768, N=2048, K=5632, act="none", x_act="gelu_tanh", bias=True, dtype="bf16"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eights(rng, lo, hi):
    """A multiple of 8, spread over the logarithm of lo..hi."""
    return max(lo, min(hi, _logint(rng, lo, hi) // 8 * 8))


def _cost(c):
    """What bounds a case's time, in units that its type's products are worth (fp32 products run on the CUDA cores)."""
    w = work(c)
    return w["bytes"], w["flops"] * (24 if c["dtype"] == "f32" and "N" in c else 1)


def _draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "linear_fwd", "linear_bwd"])
    c = dict(op=op, M=_logint(rng, 1, 65536))
    c.update(dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op.startswith("ln"):
        c.update(D=_eights(rng, 256, 8192), residual=rng.random() < 0.5)
        return c
    c.update(N=_eights(rng, 1024, 11008), K=_eights(rng, 1024, 11008), act=rng.choice(ACTS), bias=rng.random() < 0.75)
    if op == "linear_fwd":
        c.update(residual=rng.random() < 0.5, keep=c["act"] != "none" and rng.random() < 0.5)
    else:
        c.update(x_act=rng.choice(ACTS))
    return c


def draw(rng):
    most = [max(v) for v in zip(*(_cost(c) for c in listed()))]
    while True:
        c = _draw(rng)
        if all(v <= m for v, m in zip(_cost(c), most)):
            return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(gen, shape, std, dtype, mean=0.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).add_(mean).to(dtype)


def _stream(gen, M, D, dtype):
    """Rows of a residual stream: channels of unlike size and offset, a few large ones."""
    scale = torch.exp(0.5 * torch.randn(D, generator=gen, device="cuda"))
    scale[torch.randint(D, (max(1, D // 512),), generator=gen, device="cuda")] *= 20
    offset = 0.3 * torch.randn(D, generator=gen, device="cuda")
    x = torch.randn((M, D), generator=gen, device="cuda")
    return x.mul_(scale).add_(offset).to(dtype)


def _inputs(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, M = DTYPES[c["dtype"]], c["M"]
    if c["op"].startswith("ln"):
        D = c["D"]
        s = dict(X=_stream(gen, M, D, dt), weight=_normal(gen, (D,), 0.1, dt, 1.0))
        if c["op"] == "ln_fwd":
            s.update(bias=_normal(gen, (D,), 0.1, dt), R=_normal(gen, (M, D), 1.0, dt) if c["residual"] else None)
        else:
            x = s["X"].float()
            mean = x.mean(1, dtype=torch.float64)
            rstd = (((x - mean[:, None].float()) ** 2).mean(1, dtype=torch.float64) + EPS).rsqrt()
            s.update(mean=mean.float(), rstd=rstd.float(), dY=_normal(gen, (M, D), 0.1, dt),
                     dS=_normal(gen, (M, D), 0.1, dt) if c["residual"] else None)
        return s
    N, K = c["N"], c["K"]
    s = dict(W=_normal(gen, (N, K), K ** -0.5, dt))
    if c["op"] == "linear_fwd":
        s.update(X=_normal(gen, (M, K), 1.0, dt), bias=_normal(gen, (N,), 0.2, dt) if c["bias"] else None,
                 R=_normal(gen, (M, N), 1.0, dt) if c["residual"] else None)
        return s
    s.update(dY=_normal(gen, (M, N), 0.1, dt), Z=None, Xpre=None)
    if c["act"] != "none":
        s.update(Z=_normal(gen, (M, N), 1.0, dt))
    x = _normal(gen, (M, K), 1.0, dt)
    if c["x_act"] != "none":
        s.update(Xpre=x)
        x = _act(c["x_act"], x.float()).to(dt)
    s.update(X=x)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        # what a program keeps: a workspace and output buffers
        from backward_tcgen05_tma_gb300 import api

        c, dt, dev = case, DTYPES[case["dtype"]], s["X"].device
        new = lambda *n, d=dt: torch.empty(*n, dtype=d, device=dev)
        M = c["M"]
        if c["op"] == "ln_fwd":
            s["out"] = {"Y": new(M, c["D"]), "mean": new(M, d=torch.float32), "rstd": new(M, d=torch.float32)}
            if c["residual"]:
                s["out"]["S"] = new(M, c["D"])
        elif c["op"] == "ln_bwd":
            s["ws"] = api.layer_norm_workspace(M, c["D"], dt, dev)
            s["out"] = {"dX": new(M, c["D"]), "dweight": new(c["D"]), "dbias": new(c["D"])}
        elif c["op"] == "linear_fwd":
            s["ws"] = api.linear_workspace(M, c["N"], c["K"], dt, api.SWIGLU_OP_FWD, dev)
            s["out"] = {"Y": new(M, c["N"])}
            if c["keep"]:
                s["out"]["Z"] = new(M, c["N"])
        else:
            s["ws"] = api.linear_workspace(M, c["N"], c["K"], dt, api.SWIGLU_OP_BWD, dev)
            s["out"] = {"dX": new(M, c["K"]), "dW": new(c["N"], c["K"])}
            if c["bias"]:
                s["out"]["dbias"] = new(c["N"])
            if c["act"] != "none":
                s["out"]["dZ"] = new(M, c["N"])
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z))


def _dact(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if name == "gelu_tanh":
        k = (2 / math.pi) ** 0.5
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def _plain(s):
    c = s["case"]
    op, dt = c["op"], s["X"].dtype
    if op == "ln_fwd":
        x = s["X"].float()
        if c["residual"]:
            x = (x + s["R"].float()).to(dt).float()
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = ((d * d).mean(1) + EPS).rsqrt()
        y = (d * rstd[:, None] * s["weight"].float() + s["bias"].float()).to(dt)
        return (y, x.to(dt), mean, rstd) if c["residual"] else (y, mean, rstd)
    if op == "ln_bwd":
        dy, rstd = s["dY"].float(), s["rstd"][:, None]
        xh = (s["X"].float() - s["mean"][:, None]) * rstd
        t = dy * s["weight"].float()
        dx = rstd * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["dS"].float()
        return dx.to(dt), (dy * xh).sum(0).to(dt), dy.sum(0).to(dt)
    if op == "linear_fwd":
        z = s["X"].float() @ s["W"].float().T
        if c["bias"]:
            z = z + s["bias"].float()
        y = _act(c["act"], z)
        if c["residual"]:
            y = y + s["R"].float()
        return (y.to(dt), z.to(dt)) if c["keep"] else y.to(dt)
    dz = s["dY"].float()
    if c["act"] != "none":
        dz = dz * _dact(c["act"], s["Z"].float())
    dx = dz @ s["W"].float()
    if c["x_act"] != "none":
        dx = dx * _dact(c["x_act"], s["Xpre"].float())
    dw = dz.T @ s["X"].float()
    return (dx.to(dt), dw.to(dt), dz.sum(0).to(dt)) if c["bias"] else (dx.to(dt), dw.to(dt))


def run(state):
    if not own:
        return _plain(state)
    from backward_tcgen05_tma_gb300 import api

    c, s, out = state["case"], state, state["out"]
    if c["op"] == "ln_fwd":
        y, stream, mean, rstd = api.swiglu_mlp_layer_norm_fwd(s["X"], s["weight"], s["bias"], EPS, residual=s["R"], out=out)
        return (y, stream, mean, rstd) if c["residual"] else (y, mean, rstd)
    if c["op"] == "ln_bwd":
        return api.swiglu_mlp_layer_norm_bwd(s["dY"], s["X"], s["weight"], s["mean"], s["rstd"], dS=s["dS"], out=out, ws=s["ws"])
    if c["op"] == "linear_fwd":
        y, z = api.swiglu_mlp_linear_fwd(s["X"], s["W"], s["bias"], activation=c["act"], residual=s["R"], keep=c["keep"], out=out,
                                         ws=s["ws"])
        return (y, z) if c["keep"] else y
    dx, dw, db = api.swiglu_mlp_linear_bwd(s["dY"], s["X"], s["W"], s["Z"], activation=c["act"], X_pre=s["Xpre"],
                                           x_activation=c["x_act"], need_dbias=c["bias"], out=out, ws=s["ws"])
    return (dx, dw, db) if c["bias"] else (dx, dw)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c, M = case, case["M"]
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"].startswith("ln"):
        D, r = c["D"], c["residual"]
        if c["op"] == "ln_fwd":
            return {"bytes": e * (M * D * (4 if r else 2) + 2 * D) + 8 * M, "flops": (9 if r else 8) * M * D}
        return {"bytes": e * (M * D * (4 if r else 3) + 3 * D) + 8 * M, "flops": (14 if r else 13) * M * D}
    N, K = c["N"], c["K"]
    if c["op"] == "linear_fwd":
        mn = 1 + c["residual"] + c["keep"]
        return {"bytes": e * (M * K + N * K + M * N * mn + N * c["bias"]), "flops": 2 * M * N * K}
    mn, mk = 1 + (c["act"] != "none"), 2 + (c["x_act"] != "none")
    return {"bytes": e * (M * N * mn + M * K * mk + 2 * N * K + N * c["bias"]), "flops": 4 * M * N * K}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------
def _phi(z):
    """The normal distribution function, by its complement where that is the smaller one."""
    return 0.5 * torch.erfc(-z / math.sqrt(2))


def _act64(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * _phi(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if name == "silu" else z


def _slope64(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if name == "gelu":
        return _phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    inner, slope = z, torch.ones_like(z)
    if name == "gelu_tanh":
        k = math.sqrt(8 / math.pi)
        inner, slope = k * (z + 0.044715 * z ** 3), k * (1 + 0.134145 * z ** 2)
    p = torch.sigmoid(inner)
    return p + z * p * torch.sigmoid(-inner) * slope


def exact(case, seed):
    c = case
    s = {k: v if v is None else v.double() for k, v in _inputs(c, seed).items()}
    x = s["X"]
    if c["op"] == "ln_fwd":
        total = x + s["R"] if c["residual"] else x
        x = total.to(DTYPES[c["dtype"]]).double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(s["bias"], (x - mean[:, None]) * rstd[:, None], s["weight"])
        return (y, total, mean, rstd) if c["residual"] else (y, mean, rstd)
    if c["op"] == "ln_bwd":
        xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
        g = s["dY"] * s["weight"]
        D = x.shape[1]
        # the gradient without its parts along the row of ones and along xh
        dx = g - g.sum(1, keepdim=True) / D - xh * torch.einsum("md,md->m", g, xh)[:, None] / D
        dx = dx * s["rstd"][:, None]
        dx = dx + s["dS"] if c["residual"] else dx
        return dx, torch.einsum("md,md->d", s["dY"], xh), s["dY"].sum(0)
    if c["op"] == "linear_fwd":
        z = torch.nn.functional.linear(x, s["W"], s["bias"])
        y = _act64(c["act"], z)
        y = y + s["R"] if c["residual"] else y
        return (y, z) if c["keep"] else y
    dz = s["dY"] if c["act"] == "none" else s["dY"] * _slope64(c["act"], s["Z"])
    dx = torch.einsum("mn,nk->mk", dz, s["W"])
    if c["x_act"] != "none":
        dx = dx * _slope64(c["x_act"], s["Xpre"])
    dw = torch.einsum("mn,mk->nk", dz, x)
    return (dx, dw, dz.sum(0)) if c["bias"] else (dx, dw)
