"""Norms before and after a block (moe_norm_pre, moe_norm_post).

    N(v)  = (v - mu) / sqrt(mean((v - mu)^2) + eps) * (w + w_offset) + b
    pre:    N(x)
    post:   r' = res_scale * r + branch_scale * gate * N(y);  N_next(r')

Tensors are [T, D] in fp32 or bf16; rows may be strided views.
"""
from __future__ import annotations

import torch

from . import _lib as L

KINDS = {"none": L.MOE_NORM_NONE, "rms": L.MOE_NORM_RMS, "layer": L.MOE_NORM_LAYER}
GATES = {"none": L.MOE_GATE_NONE, "channel": L.MOE_GATE_CHANNEL, "token": L.MOE_GATE_TOKEN, "full": L.MOE_GATE_FULL}


def _kind(kind: str) -> int:
    k = KINDS.get(kind)
    if k is None:
        raise ValueError(f"kind: one of {sorted(KINDS)}, not {kind!r}")
    return k


def pre(x, w=None, b=None, *, kind: str = "rms", eps: float = 1e-6, w_offset: float = 0.0, out=None) -> torch.Tensor:
    """N(x), in out's type (x's if out is None)."""
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    L.moe_norm_pre(x, w, b, _kind(kind), eps, w_offset, out)
    return out


def post(y, res, w=None, b=None, *, kind: str = "rms", eps: float = 1e-6, w_offset: float = 0.0, gate=None,
         gate_by: str = "channel", gate_sigmoid: bool = False, res_scale: float = 1.0, branch_scale: float = 1.0,
         next_w=None, next_b=None, next_norm: bool = None, next_kind: str = None, out=None, next_out=None):
    """(r', N_next(r') or None).

    gate [D] ("channel"), [T] ("token") or [T, D] ("full"); None: 1.  The next
    norm is taken where next_w, next_out or next_norm asks for it, of
    next_kind (None: kind, or "rms" after kind "none"; "none": no next norm),
    with the same eps and w_offset.  out may be res itself.
    """
    if out is None:
        out = torch.empty(res.shape, dtype=res.dtype, device=res.device)
    by = L.MOE_GATE_NONE
    if gate is not None:
        by = GATES.get(gate_by)
        if by is None:
            raise ValueError(f"gate_by: one of {sorted(GATES)}, not {gate_by!r}")
    if next_norm is None:
        next_norm = next_w is not None or next_out is not None
    nk = _kind(next_kind or (kind if kind != "none" else "rms")) if next_norm else L.MOE_NORM_NONE
    if nk == L.MOE_NORM_NONE:
        next_out = None
    elif next_out is None:
        next_out = torch.empty(res.shape, dtype=y.dtype, device=res.device)
    L.moe_norm_post(y, res, out, next_out, _kind(kind), eps, w_offset, w, b, nk, next_w, next_b, res_scale, branch_scale, by, gate, gate_sigmoid)
    return out, next_out
