"""What stands around an MLP in a transformer block, as autograd functions and
modules: layer norm (with the residual sum in front of it), linear layers with
bias, activation and residual, the MLP without a gate that two of them make,
and the pre-norm sublayer x + mlp(norm(x)) of any of this package's MLPs.

The tensors are CUDA tensors of one dtype (bf16, fp16, or fp32 for the IEEE
mode).  Norms, products, activations and their gradients run in the library's
kernels, and so do the sums of a residual stream in a norm or in an ``MLP``; the
one behind another kind of MLP in ``MLPBlock`` is a sum of tensors, unless it is
left to the next norm (``join=False``).  Nothing that a
backward pass needs is overwritten, so a graph may be kept and run again;
double differentiation and forward-mode derivatives are refused.  A captured training step takes its
gradients with ``torch.autograd.grad``, or through leaves that no graph from
outside the capture holds.
"""
from __future__ import annotations

import math

import torch

from . import api
from .module import refuse_tangents, rows_of as _rows


def _output(x, X, N):
    """An output [..., N] for x's batch and its rows [M, N].  The output is no view:
    autograd refuses changes in place of a custom function's views."""
    Y = x.new_empty(*x.shape[:-1], N)
    return Y, Y.view(X.shape[0], N)


def _grad_rows(g, D, dtype):
    """A gradient as rows of the forward's type (it may come expanded)."""
    return _rows(g.to(dtype), D)


def _last(x, D, what):
    if x.dim() == 0 or x.shape[-1] != D:
        raise ValueError("%s: expected [..., %d], got %s" % (what, D, tuple(x.shape)))


def _alike(x, other, shape, what):
    if other is not None and other.shape != shape:
        raise ValueError("%s must have the shape %s, got %s" % (what, tuple(shape), tuple(other.shape)))


def _recording(*tensors):
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


class LayerNormFunction(torch.autograd.Function):
    """(Y, S) = (norm(x + residual), x + residual); without a residual Y alone."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, residual):
        D = x.shape[-1]
        X, out = _rows(x, D), {}
        r = None if residual is None else _rows(residual, D)
        Y, out["Y"] = _output(x, X, D)
        S = X
        if residual is not None:
            S, out["S"] = _output(x, X, D)
        _, _, mean, rstd = api.swiglu_mlp_layer_norm_fwd(X, weight, bias, eps, residual=r, out=out)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(S, weight, mean, rstd)
        ctx.shape = x.shape
        ctx.has_residual = residual is not None
        return Y if residual is None else (Y, S)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY, dS=None):
        S, weight, mean, rstd = ctx.saved_tensors
        _, need_w, need_b, _, need_r = ctx.needs_input_grad
        if dY is None:  # the sum alone was used
            return dS, None, None, None, dS if ctx.has_residual else None
        D = S.shape[-1]
        dX, dw, db = api.swiglu_mlp_layer_norm_bwd(
            _grad_rows(dY, D, S.dtype), S.reshape(-1, D), weight, mean, rstd,
            dS=None if dS is None else _grad_rows(dS, D, S.dtype), need_dweight=need_w, need_dbias=need_b)
        dX = dX.reshape(ctx.shape)
        return dX, dw, db, None, dX if need_r else None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, residual=None):
    """Layer norm over the last dimension.  With ``residual`` (x's shape) the
    norm is that of the rounded sum x + residual, and (norm, sum) is returned:
    the sum is the residual stream behind."""
    D = x.shape[-1] if x.dim() else 0
    _last(x, D, "layer_norm")
    _alike(x, residual, x.shape, "residual")
    refuse_tangents("layer_norm", x, weight, bias, residual)
    if _recording(x, weight, bias, residual):
        return LayerNormFunction.apply(x, weight, bias, float(eps), residual)
    r = None if residual is None else _rows(residual, D)
    Y, S, _, _ = api.swiglu_mlp_layer_norm_fwd(_rows(x, D), weight, bias, float(eps), residual=r,
                                               stats=False)
    return Y.reshape(x.shape) if residual is None else (Y.reshape(x.shape), S.reshape(x.shape))


class LinearFunction(torch.autograd.Function):
    """Y = act(x W^T + b) + residual."""

    @staticmethod
    def forward(ctx, x, weight, bias, activation, residual):
        N, K = weight.shape
        X = _rows(x, K)
        R = None if residual is None else _rows(residual, N)
        Y, rows = _output(x, X, N)
        _, Z = api.swiglu_mlp_linear_fwd(X, weight, bias, activation, R, keep=activation != "none", out={"Y": rows})
        ctx.save_for_backward(X, weight, Z)
        ctx.activation = activation
        ctx.shape = x.shape
        return Y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        X, weight, Z = ctx.saved_tensors
        need_x, need_w, need_b, _, need_r = ctx.needs_input_grad
        dX = dW = db = None
        if need_x or need_w or need_b:
            g = _grad_rows(dY, weight.shape[0], X.dtype)
            dX, dW, db = api.swiglu_mlp_linear_bwd(g, X, weight, Z, ctx.activation, need_dX=need_x,
                                                   need_dW=need_w, need_dbias=need_b)
        return (None if dX is None else dX.reshape(ctx.shape), dW, db, None, dY if need_r else None)


def linear(x, weight, bias=None, activation: str = "none", residual=None):
    """act(x W^T + bias) + residual, W [N, K] as nn.Linear keeps it; activation:
    "none", "relu", "gelu", "gelu_tanh" or "silu"."""
    N, K = weight.shape
    api.activation_code(activation)
    _last(x, K, "linear")
    _alike(x, residual, (*x.shape[:-1], N), "residual")
    refuse_tangents("linear", x, weight, bias, residual)
    if _recording(x, weight, bias, residual):
        return LinearFunction.apply(x, weight, bias, activation, residual)
    R = None if residual is None else _rows(residual, N)
    Y, _ = api.swiglu_mlp_linear_fwd(_rows(x, K), weight, bias, activation, R)
    return Y.reshape(*x.shape[:-1], N)


class MLPFunction(torch.autograd.Function):
    """Y = act(x W1^T + b1) W2^T + b2 + residual; backward multiplies by the
    activation's derivative where it takes the second layer's input gradient."""

    @staticmethod
    def forward(ctx, x, w1, b1, w2, b2, activation, residual):
        X = _rows(x, w1.shape[1])
        R = None if residual is None else _rows(residual, w2.shape[0])
        A, Z = api.swiglu_mlp_linear_fwd(X, w1, b1, activation, keep=activation != "none")
        Y, rows = _output(x, X, w2.shape[0])
        api.swiglu_mlp_linear_fwd(A, w2, b2, "none", R, out={"Y": rows})
        ctx.save_for_backward(X, w1, Z, A, w2)
        ctx.activation = activation
        ctx.shape = x.shape
        return Y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        X, w1, Z, A, w2 = ctx.saved_tensors
        need_x, need_w1, need_b1, need_w2, need_b2, _, need_r = ctx.needs_input_grad
        first = need_x or need_w1 or need_b1
        dX = dW1 = db1 = dW2 = db2 = None
        if first or need_w2 or need_b2:
            g = _grad_rows(dY, w2.shape[0], X.dtype)
            dZ, dW2, db2 = api.swiglu_mlp_linear_bwd(g, A, w2, X_pre=Z, x_activation=ctx.activation,
                                                     need_dX=first, need_dW=need_w2,
                                                     need_dbias=need_b2)
        if first:
            dX, dW1, db1 = api.swiglu_mlp_linear_bwd(dZ, X, w1, need_dX=need_x, need_dW=need_w1,
                                                     need_dbias=need_b1)
        return (None if dX is None else dX.reshape(ctx.shape), dW1, db1, dW2, db2, None,
                dY if need_r else None)


def mlp(x, w1, b1, w2, b2, activation: str = "gelu", residual=None):
    """act(x W1^T + b1) W2^T + b2 + residual."""
    api.activation_code(activation)
    _last(x, w1.shape[1], "mlp")
    _alike(x, residual, (*x.shape[:-1], w2.shape[0]), "residual")
    refuse_tangents("mlp", x, w1, b1, w2, b2, residual)
    if _recording(x, w1, b1, w2, b2, residual):
        return MLPFunction.apply(x, w1, b1, w2, b2, activation, residual)
    return linear(linear(x, w1, b1, activation), w2, b2, "none", residual)


class LayerNorm(torch.nn.Module):
    """Layer norm over the last dimension; parameters and state as
    nn.LayerNorm's.  ``forward(x, residual)`` returns (norm, x + residual)."""

    def __init__(self, hidden_size: int, eps: float = 1e-5, elementwise_affine: bool = True,
                 bias: bool = True, dtype=torch.bfloat16, device=None):
        super().__init__()
        self.hidden_size, self.eps = int(hidden_size), float(eps)
        new = lambda f: torch.nn.Parameter(f(self.hidden_size, dtype=dtype, device=device))
        self.register_parameter("weight", new(torch.ones) if elementwise_affine else None)
        self.register_parameter("bias", new(torch.zeros) if elementwise_affine and bias else None)

    def forward(self, x, residual=None):
        _last(x, self.hidden_size, "LayerNorm")
        return layer_norm(x, self.weight, self.bias, self.eps, residual)

    def extra_repr(self):
        return "hidden_size=%d, eps=%g" % (self.hidden_size, self.eps)


# names that configurations give these activations
HIDDEN_ACTS = {"relu": "relu", "gelu": "gelu", "gelu_new": "gelu_tanh", "gelu_fast": "gelu_tanh",
               "gelu_pytorch_tanh": "gelu_tanh", "gelu_tanh": "gelu_tanh", "silu": "silu",
               "swish": "silu"}


class MLP(torch.nn.Module):
    """down(act(up(x))), the MLP without a gate, with biases unless ``bias`` is
    False.  Loads ``fc1``/``fc2`` or ``up_proj``/``down_proj`` state as well as
    its own (``up_weight``, ``up_bias``, ``down_weight``, ``down_bias``)."""

    def __init__(self, config=None, intermediate_size: int | None = None, *,
                 hidden_size: int | None = None, activation: str | None = None, bias: bool = True,
                 dtype=torch.bfloat16, device=None):
        super().__init__()
        if config is not None and not isinstance(config, int):
            D, H = int(config.hidden_size), int(config.intermediate_size)
            activation = getattr(config, "hidden_act", "gelu") if activation is None else activation
        else:
            D = int(hidden_size if config is None else config)
            H = int(intermediate_size)
        act = "gelu" if activation is None else activation
        if act not in HIDDEN_ACTS:
            raise ValueError("MLP computes %s, not %r" % (", ".join(HIDDEN_ACTS), act))
        self.activation = HIDDEN_ACTS[act]
        self.hidden_size, self.intermediate_size = D, H
        new = lambda *s: torch.nn.Parameter(torch.empty(*s, dtype=dtype, device=device))
        self.up_weight, self.down_weight = new(H, D), new(D, H)
        self.register_parameter("up_bias", new(H) if bias else None)
        self.register_parameter("down_bias", new(D) if bias else None)
        self.reset_parameters()
        self._register_load_state_dict_pre_hook(_mlp_keys)

    def reset_parameters(self):
        # nn.Linear's default: U(-1/sqrt(fan_in), 1/sqrt(fan_in))
        with torch.no_grad():
            for p, fan_in in ((self.up_weight, self.hidden_size), (self.up_bias, self.hidden_size),
                              (self.down_weight, self.intermediate_size),
                              (self.down_bias, self.intermediate_size)):
                if p is not None:
                    p.uniform_(-1 / math.sqrt(fan_in), 1 / math.sqrt(fan_in))

    def forward(self, x, residual=None):
        return mlp(x, self.up_weight, self.up_bias, self.down_weight, self.down_bias,
                   self.activation, residual)

    def extra_repr(self):
        return "hidden_size=%d, intermediate_size=%d, activation=%s, bias=%s" % (
            self.hidden_size, self.intermediate_size, self.activation, self.up_bias is not None)


def _mlp_keys(state_dict, prefix, *args, **kwargs):
    for ours, names in (("up", ("fc1", "up_proj")), ("down", ("fc2", "down_proj"))):
        for name in names:
            for part in ("weight", "bias"):
                if "%s%s.%s" % (prefix, name, part) in state_dict:
                    state_dict["%s%s_%s" % (prefix, ours, part)] = state_dict.pop(
                        "%s%s.%s" % (prefix, name, part))


class MLPBlock(torch.nn.Module):
    """The pre-norm sublayer of a transformer block: with s = x (+ delta),
    s + mlp(norm(s)).

    ``mlp`` is an ``MLP`` (the sum is in its second product's epilogue), a
    ``module.SwiGLUMLP``, or for inference a ``serving.W4SwiGLUMLP`` or
    ``serving.MoESwiGLU``.  ``delta`` is what the sublayer before (an attention,
    or another of these) adds to the stream: it is added in the norm's kernel.
    With ``join=False`` the sum behind is left to the next one in the same way:
    (s, mlp(norm(s))) is returned."""

    def __init__(self, mlp, hidden_size: int | None = None, eps: float = 1e-5, bias: bool = True,
                 dtype=None, device=None):
        super().__init__()
        D = int(mlp.hidden_size if hidden_size is None else hidden_size)
        # the norm's type and place, unless given: 4-bit weights are no parameters, their module says
        like = next(mlp.parameters(), mlp)
        dtype = getattr(like, "dtype", None) if dtype is None else dtype
        device = getattr(like, "device", None) if device is None else device
        dtype = torch.bfloat16 if dtype is None else dtype
        self.norm = LayerNorm(D, eps, bias=bias, dtype=dtype, device=device)
        self.mlp = mlp

    def forward(self, x, delta=None, join: bool = True):
        if delta is None:
            y, s = self.norm(x), x
        else:
            y, s = self.norm(delta, x)
        if not join:
            return s, self.mlp(y)
        if isinstance(self.mlp, MLP):
            return self.mlp(y, s)
        return s + self.mlp(y)
