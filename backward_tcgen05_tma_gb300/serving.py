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


class W4SwiGLUMLP(torch.nn.Module):
    """down(SiLU(gate(x)) * up(x)) on 4-bit weights with group scales.

    ``W4SwiGLUMLP(mlp)`` rounds the weights of a ``module.SwiGLUMLP``;
    ``from_codes`` takes a checkpoint's codes, scales and zero points."""

    def __init__(self, mlp=None, group: int = 128, zeros: bool = False):
        super().__init__()
        self.gate_multiplier = self.down_multiplier = 1.0
        if mlp is not None:
            self.gate_multiplier, self.down_multiplier = mlp.gate_multiplier, mlp.down_multiplier
            gu = api.swiglu_mlp_w4_quantize(mlp.gate_up_weight.detach(), group, zeros)
            down = api.swiglu_mlp_w4_quantize(mlp.down_weight.detach(), group, zeros)
            self._set(gu, down, group)

    def _set(self, gate_up, down, group):
        self.gate_up = api.swiglu_mlp_w4_pack(*gate_up, group=group, gate_up=True)
        self.down = api.swiglu_mlp_w4_pack(*down, group=group)

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
    experts' weights by 4-bit copies."""

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
        self._w4 = None
        with torch.no_grad():  # nn.Linear's default: U(-1/sqrt(fan_in), 1/sqrt(fan_in))
            for w, fan_in in ((self.router_weight, D), (self.gate_up_weight, D),
                              (self.down_weight, H)):
                w.uniform_(-fan_in ** -0.5, fan_in ** -0.5)

    def quantize(self, group: int = 128, zeros: bool = False):
        """Rounds the experts to 4 bits and frees their 16-bit weights."""
        if self._w4 is not None:
            raise RuntimeError("the experts are in 4 bits already")
        gu = api.swiglu_mlp_w4_quantize(self.gate_up_weight.detach(), group, zeros)
        down = api.swiglu_mlp_w4_quantize(self.down_weight.detach(), group, zeros)
        self._w4 = (api.swiglu_mlp_w4_pack(*gu, group=group, gate_up=True),
                    api.swiglu_mlp_w4_pack(*down, group=group))
        self.gate_up_weight = self.down_weight = None
        return self

    def forward(self, x):
        _no_grad_only(x, "MoESwiGLU")
        D = x.shape[-1]
        X = x.reshape(-1, D).contiguous()
        gu, down = self._w4 or (self.gate_up_weight.detach(), self.down_weight.detach())
        Y = torch.empty_like(X)
        for t in range(0, X.shape[0], MAX_TOKENS):
            part = slice(t, t + MAX_TOKENS)
            api.swiglu_mlp_moe_fwd_nograd(X[part], self.router_weight.detach(), gu, down,
                                          self.top_k, self.norm_topk, self.route_scale,
                                          out={"Y": Y[part]})
        return Y.reshape(x.shape)
