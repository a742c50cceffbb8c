"""MoEBlock: the MoE half of a decoder block at serving time.

    n   = N_pre(r)                      (once, at the start of the stack)
    y   = layer(n)                      (where it is the faster: one moe_forward_few call)
    r'  = res_scale * r + branch_scale * gate * N_post(y)
    n'  = N_next(r')                    (fused with the line above)

The residual stream r keeps its own type (fp32 or bf16); n is the layer's
input type.
"""
from __future__ import annotations

import torch

from . import norm
from .layer import MoELayer


class MoEBlock:
    """gate: what every call uses; a gate by token or in full belongs to a call's rows and is given to forward."""

    def __init__(self, layer: MoELayer, *, kind: str = "rms", eps: float = 1e-6, w_offset: float = 0.0, pre_w=None,
                 post_w=None, post_kind: str = None, gate=None, gate_by: str = "channel", gate_sigmoid: bool = False,
                 res_scale: float = 1.0, branch_scale: float = 1.0, next_w=None, next_kind: str = None, pre_b=None,
                 post_b=None, next_b=None):
        self.layer = layer
        self.gate = gate
        self.pre_args = dict(w=pre_w, b=pre_b, kind=kind, eps=eps, w_offset=w_offset)
        # post_kind "none": no norm after the layer
        self.post_args = dict(w=post_w, b=post_b, kind=post_kind or kind, eps=eps, w_offset=w_offset, gate_by=gate_by,
                              gate_sigmoid=gate_sigmoid, res_scale=res_scale, branch_scale=branch_scale, next_w=next_w,
                              next_b=next_b, next_kind=next_kind)
        self.in_dtype = torch.float32 if layer.dtype == "f32" else torch.bfloat16

    def forward(self, r: torch.Tensor, n: torch.Tensor = None, next_norm: bool = True, gate: torch.Tensor = None):
        """(r', n') of residual stream r [T, D]; n is N_pre(r) where the block before has it already, gate this
        call's ([T] or [T, D] by the block's gate_by; None: the block's own)."""
        T = r.shape[0]
        if n is None:
            n = norm.pre(r, out=torch.empty(r.shape, dtype=self.in_dtype, device=r.device), **self.pre_args)
        y = self.layer.forward_few(n) if self.layer.few_pays(T) else self.layer.forward(n)
        nxt = torch.empty(r.shape, dtype=self.in_dtype, device=r.device) if next_norm else None
        return norm.post(y, r, next_norm=next_norm, next_out=nxt, gate=self.gate if gate is None else gate, **self.post_args)
