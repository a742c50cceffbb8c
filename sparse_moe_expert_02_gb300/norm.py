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


def _fields(kind: str, eps: float, w_offset: float, w, b, D: int):
    """A moe_norm's fields."""
    k = KINDS.get(kind)
    if k is None:
        raise ValueError(f"kind: one of {sorted(KINDS)}, not {kind!r}")
    wp = bp = dt = 0
    if w is not None:
        wp, dt = _vector(w, D, "norm parameters")
    if b is not None:
        bp, bd = _vector(b, D, "norm parameters")
        if w is not None and bd != dt:
            raise ValueError("norm parameters: w and b of one type")
        dt = bd
    return k, eps, w_offset, dt, wp, bp


def _vector(t, n: int, what: str):
    """(address, moe_dtype) of a contiguous device vector of n fp32 or bf16."""
    dt = L._DTYPE_OF.get(t.dtype)
    if dt is None or not t.is_cuda or t.dim() != 1 or t.size(0) != n or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous device tensor [{n}] of fp32 or bf16")
    return t.data_ptr(), dt


def _same(t, shape, what: str):
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(shape)}, not {tuple(t.shape)}")


def pre(x, w=None, b=None, *, kind: str = "rms", eps: float = 1e-6, w_offset: float = 0.0, out=None) -> torch.Tensor:
    """N(x), in out's type (x's if out is None)."""
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _same(out, x.shape, "out")
    L.moe_norm_pre(L.NORM_STRUCT.pack(*_fields(kind, eps, w_offset, w, b, x.shape[-1])), x, out)
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
    shape = y.shape
    T, D = shape
    _same(res, shape, "res")
    if out is None:
        out = torch.empty(res.shape, dtype=res.dtype, device=res.device)
    else:
        _same(out, shape, "out")
    g = gd = gl = 0
    by = L.MOE_GATE_NONE
    if gate is not None and gate_by != "none":
        if gate_by not in GATES:
            raise ValueError(f"gate_by: one of {sorted(GATES)}, not {gate_by!r}")
        by = GATES[gate_by]
        if by == L.MOE_GATE_FULL:
            _same(gate, shape, "gate")
            g, gd, gl = L._rows(gate, "gate")
        else:
            g, gd = _vector(gate, D if by == L.MOE_GATE_CHANNEL else T, "gate")
    if next_norm is None:
        next_norm = next_w is not None or next_out is not None
    next_kind = next_kind or (kind if kind != "none" else "rms")
    next_norm = next_norm and next_kind != "none"
    nf = _fields(next_kind, eps, w_offset, next_w, next_b, D) if next_norm else (0, 0.0, 0.0, 0, 0, 0)
    if not next_norm:
        next_out = None
    elif next_out is None:
        next_out = torch.empty(res.shape, dtype=y.dtype, device=res.device)
    else:
        _same(next_out, shape, "next_out")
    L.moe_norm_post(L.POST_STRUCT.pack(*_fields(kind, eps, w_offset, w, b, D), *nf, res_scale, branch_scale, by, gd,
                                       gate_sigmoid, g, gl), y, res, out, next_out)
    return out, next_out
