"""Weights in 4-bit integers with a scale per group of columns, beside 16- or
32-bit activations: quantise, read back, multiply.

An ``I4Tensor`` holds a [..., rows, cols] tensor as unsigned codes, two a byte,
and a scale (and, if asked for, a zero point) per 32, 64 or 128 columns:
value = scale * (code - zero), zero 8 where none is stored (moe_int4_quantize
in the C header says how they are chosen).
"""
from __future__ import annotations

import torch

from . import _lib as L


class I4Tensor:
    """codes uint8 [..., rows, cols/2], scales fp32 or bf16 [..., rows, ceil(cols/group)], zeros uint8 like scales or None."""
    __slots__ = ("codes", "scales", "zeros", "cols", "group")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, cols: int, group: int):
        if group not in (32, 64, 128) or cols < 32 or cols % 32:
            raise ValueError("I4Tensor: a multiple of 32 columns, in groups of 32, 64 or 128")
        nb = -(-cols // group)
        if codes.dtype != torch.uint8 or scales.dtype not in (torch.float32, torch.bfloat16) or (zeros is not None and
                                                                                                 zeros.dtype != torch.uint8):
            raise ValueError("I4Tensor: uint8 codes, fp32 or bf16 scales, uint8 zeros or None")
        lead = tuple(codes.shape[:-1])
        if codes.dim() < 2 or codes.shape[-1] != cols // 2 or tuple(scales.shape) != lead + (nb,) or (
                zeros is not None and tuple(zeros.shape) != lead + (nb,)):
            raise ValueError(f"I4Tensor: codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not hold {cols} columns "
                             f"in groups of {group}")
        self.codes, self.scales, self.zeros, self.cols, self.group = codes, scales, zeros, cols, group

    @property
    def shape(self):
        return tuple(self.codes.shape[:-1]) + (self.cols,)


def empty(rows, cols: int, group: int = 128, zeros: bool = False, scale_dtype: torch.dtype = torch.bfloat16, device="cuda") -> I4Tensor:
    """Uninitialised codes, scales and, if asked for, zero points; rows is a number or the leading shape."""
    lead = (rows,) if isinstance(rows, int) else tuple(rows)
    nb = -(-cols // group)
    return I4Tensor(torch.empty(lead + (cols // 2,), dtype=torch.uint8, device=device),
                    torch.empty(lead + (nb,), dtype=scale_dtype, device=device),
                    torch.empty(lead + (nb,), dtype=torch.uint8, device=device) if zeros else None, cols, group)


def quantize(x: torch.Tensor, group: int = 128, zeros: bool = False, scale_dtype: torch.dtype = torch.bfloat16,
             out: I4Tensor = None) -> I4Tensor:
    """fp32 or bf16 x [..., rows, cols] (strided rows if 2-D) to 4 bits; out decides the form where it is given."""
    if out is None:
        out = empty(x.shape[:-1], x.shape[-1], group, zeros, scale_dtype, x.device)
    if x.dim() != 2 or out.codes.dim() != 2:
        if out.shape != tuple(x.shape):
            raise ValueError(f"out holds {out.shape}, not {tuple(x.shape)}")
        x = x.reshape(-1, x.shape[-1])
    L.moe_int4_quantize(x, out.codes, out.scales, out.zeros, out.cols, out.group)
    return out


def dequantize(q: I4Tensor, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor = None) -> torch.Tensor:
    """The values of q, in out's type (dtype if out is None), rounded once."""
    if out is None:
        out = torch.empty(q.shape, dtype=dtype, device=q.codes.device)
    flat = out
    if out.dim() != 2 or q.codes.dim() != 2:
        if tuple(out.shape) != q.shape:
            raise ValueError(f"out: shape {q.shape}, not {tuple(out.shape)}")
        flat = out.view(-1, out.shape[-1])
    L.moe_int4_dequantize(q.codes, q.scales, q.zeros, q.cols, q.group, flat)
    return out


def matmul(x: torch.Tensor, w: I4Tensor, offsets: torch.Tensor = None, out: torch.Tensor = None, out_dtype: torch.dtype = None,
           err: torch.Tensor = None) -> torch.Tensor:
    """x [rows, K] times w [N, K] (or its group's of w [G, N, K]) transposed, in out_dtype (x's if None).

    Groups, rows of no group and err as in ``grouped``.  For bf16 x of more than max(8 G, 32) rows (those of no group
    counted) the weights' values are rounded to bf16 once; else, and for fp32 x, they are multiplied as they are.
    """
    if out is None:
        out = torch.empty((x.shape[0], w.codes.shape[-2]), dtype=out_dtype or x.dtype, device=x.device)
    L.moe_int4_gemm(x, w.codes, w.scales, w.zeros, w.cols, w.group, offsets, out, err)
    return out
