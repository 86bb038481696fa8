"""Inference modules over the few-token serving operators: a SwiGLU MLP on
4-bit weights, and a mixture-of-experts layer with 16-bit or 4-bit experts.

Both compute without gradients and refuse inputs that require them.  The
kernels take up to 64 tokens a call: the MLP expands its weights and takes the
dense no-grad path for more, the mixture of experts goes through a larger
batch 64 tokens at a time.  Tensors must be contiguous CUDA tensors, bf16 or
fp16.
"""
from __future__ import annotations

import torch

from . import api

MAX_TOKENS = 64  # of one call of the few-token operators


def _no_grad_only(x, what):
    if torch.is_grad_enabled() and x.requires_grad:
        raise RuntimeError("%s has no backward pass: call it under torch.no_grad()" % what)


class PackedW4(torch.nn.Module):
    """An ``api.W4Weights`` as state of a module: the packed bytes are a buffer
    (``packed``), sizes and format go with them as extra state, so that saving,
    loading and moving the module takes the weights along.  Loading replaces
    sizes and format; the bytes stay on the device where they were."""

    FIELDS = ("N", "K", "group", "zeros", "gate_up", "experts")

    def __init__(self, W=None, device=None):
        super().__init__()
        self._weights = W
        self._format = None if W is None else {f: getattr(W, f) for f in self.FIELDS} | {
            "dtype": str(W.dtype).removeprefix("torch.")}
        self.register_buffer("packed", torch.empty(0, dtype=torch.uint8, device=device)
                             if W is None else W.packed)

    @property
    def weights(self) -> api.W4Weights:
        packed = self.packed
        if self._weights is None or self._weights.packed is not packed:  # loaded or moved
            if self._format is None:
                raise RuntimeError("no 4-bit weights have been set or loaded")
            f = dict(self._format)
            self._weights = api.W4Weights(packed, dtype=getattr(torch, f.pop("dtype")), **f)
        return self._weights

    def get_extra_state(self):
        return self._format

    def set_extra_state(self, state):
        self._format, self._weights = state, None

    def _load_from_state_dict(self, state_dict, prefix, *args):
        new = state_dict.get(prefix + "packed")
        if new is not None and new.shape != self.packed.shape:
            self.packed = torch.empty_like(new, device=self.packed.device)
        super()._load_from_state_dict(state_dict, prefix, *args)


class W4SwiGLUMLP(torch.nn.Module):
    """down(SiLU(gate(x)) * up(x)) on 4-bit weights with group scales.

    ``W4SwiGLUMLP(mlp)`` rounds the weights of a ``module.SwiGLUMLP``;
    ``from_codes`` takes a checkpoint's codes, scales and zero points;
    ``W4SwiGLUMLP(device=...)`` is empty until ``load_state_dict`` fills it.
    The multipliers are part of the state."""

    def __init__(self, mlp=None, group: int = 128, zeros: bool = False, device=None):
        super().__init__()
        self.gate_multiplier = self.down_multiplier = 1.0
        self.gate_up_w4, self.down_w4 = PackedW4(device=device), PackedW4(device=device)
        if mlp is not None:
            self.gate_multiplier, self.down_multiplier = mlp.gate_multiplier, mlp.down_multiplier
            gu = api.swiglu_mlp_w4_quantize(mlp.gate_up_weight.detach(), group, zeros)
            down = api.swiglu_mlp_w4_quantize(mlp.down_weight.detach(), group, zeros)
            self._set(gu, down, group)

    def _set(self, gate_up, down, group):
        self.gate_up_w4 = PackedW4(api.swiglu_mlp_w4_pack(*gate_up, group=group, gate_up=True))
        self.down_w4 = PackedW4(api.swiglu_mlp_w4_pack(*down, group=group))

    @property
    def gate_up(self) -> api.W4Weights:
        return self.gate_up_w4.weights

    @property
    def down(self) -> api.W4Weights:
        return self.down_w4.weights

    def get_extra_state(self):
        return {"gate_multiplier": self.gate_multiplier, "down_multiplier": self.down_multiplier}

    def set_extra_state(self, state):
        self.gate_multiplier = float(state["gate_multiplier"])
        self.down_multiplier = float(state["down_multiplier"])

    @classmethod
    def from_codes(cls, gate_up, down, group: int = 128, gate_multiplier: float = 1.0,
                   down_multiplier: float = 1.0):
        """``gate_up`` and ``down``: (codes, scales, zeros or None), as
        ``api.swiglu_mlp_w4_quantize`` returns them; gate rows before up rows."""
        m = cls()
        m.gate_multiplier, m.down_multiplier = float(gate_multiplier), float(down_multiplier)
        m._set(gate_up, down, group)
        return m

    def forward(self, x):
        _no_grad_only(x, "W4SwiGLUMLP")
        X = x.reshape(-1, x.shape[-1]).contiguous()
        muls = dict(gate_mul=self.gate_multiplier, down_mul=self.down_multiplier)
        if X.shape[0] <= MAX_TOKENS:
            Y, _ = api.swiglu_mlp_fwd_nograd_w4(X, self.gate_up, self.down, **muls)
        else:
            Y, _ = api.swiglu_mlp_fwd_nograd(X, api.swiglu_mlp_w4_unpack(self.gate_up),
                                             api.swiglu_mlp_w4_unpack(self.down), **muls)
        return Y.reshape(x.shape)


class MoESwiGLU(torch.nn.Module):
    """A router and ``num_experts`` SwiGLU MLPs, ``top_k`` of them per token.

    Weights: ``router_weight`` [E, D], ``gate_up_weight`` [E, 2H, D] (gate rows
    before up rows), ``down_weight`` [E, D, H].  ``quantize`` replaces the
    experts' weights by 4-bit copies (``gate_up_w4``, ``down_w4``), and so does
    loading the state of a quantised layer."""

    def __init__(self, hidden_size: int, intermediate_size: int, num_experts: int, top_k: int, *,
                 norm_topk: bool = True, route_scale: float = 1.0, dtype=torch.bfloat16,
                 device=None):
        super().__init__()
        D, H, E = int(hidden_size), int(intermediate_size), int(num_experts)
        self.top_k, self.norm_topk, self.route_scale = int(top_k), bool(norm_topk), float(route_scale)
        new = lambda *s: torch.nn.Parameter(torch.empty(*s, dtype=dtype, device=device),
                                            requires_grad=False)
        self.router_weight = new(E, D)
        self.gate_up_weight = new(E, 2 * H, D)
        self.down_weight = new(E, D, H)
        self.gate_up_w4 = self.down_w4 = None
        with torch.no_grad():  # nn.Linear's default: U(-1/sqrt(fan_in), 1/sqrt(fan_in))
            for w, fan_in in ((self.router_weight, D), (self.gate_up_weight, D),
                              (self.down_weight, H)):
                w.uniform_(-fan_in ** -0.5, fan_in ** -0.5)

    def quantize(self, group: int = 128, zeros: bool = False):
        """Rounds the experts to 4 bits and frees their 16-bit weights."""
        if self.gate_up_w4 is not None:
            raise RuntimeError("the experts are in 4 bits already")
        gu = api.swiglu_mlp_w4_quantize(self.gate_up_weight.detach(), group, zeros)
        down = api.swiglu_mlp_w4_quantize(self.down_weight.detach(), group, zeros)
        self._experts_w4(PackedW4(api.swiglu_mlp_w4_pack(*gu, group=group, gate_up=True)),
                         PackedW4(api.swiglu_mlp_w4_pack(*down, group=group)))
        return self

    def _experts_w4(self, gate_up, down):
        self.gate_up_w4, self.down_w4 = gate_up, down
        self.gate_up_weight = self.down_weight = None

    def _load_from_state_dict(self, state_dict, prefix, *args):
        if self.gate_up_w4 is None and prefix + "gate_up_w4.packed" in state_dict:
            device = self.router_weight.device
            self._experts_w4(PackedW4(device=device), PackedW4(device=device))
        super()._load_from_state_dict(state_dict, prefix, *args)

    def forward(self, x):
        _no_grad_only(x, "MoESwiGLU")
        D = x.shape[-1]
        X = x.reshape(-1, D).contiguous()
        if self.gate_up_w4 is not None:
            gu, down = self.gate_up_w4.weights, self.down_w4.weights
        else:
            gu, down = self.gate_up_weight.detach(), self.down_weight.detach()
        Y = torch.empty_like(X)
        for t in range(0, X.shape[0], MAX_TOKENS):
            part = slice(t, t + MAX_TOKENS)
            api.swiglu_mlp_moe_fwd_nograd(X[part], self.router_weight.detach(), gu, down,
                                          self.top_k, self.norm_topk, self.route_scale,
                                          out={"Y": Y[part]})
        return Y.reshape(x.shape)
