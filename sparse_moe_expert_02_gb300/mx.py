"""Microscaled 4-bit floating point (MXFP4): quantise, read back, multiply.

An ``MXTensor`` holds a [..., rows, cols] tensor as E2M1 codes, two a byte, and
one power-of-two scale byte per 32 columns (moe_mx_quantize in the C header
says how they are chosen).
"""
from __future__ import annotations

import torch

from . import _lib as L


class MXTensor:
    """codes uint8 [..., rows, 16*nb] and scales uint8 [..., rows, nb], nb = ceil(cols/32)."""
    __slots__ = ("codes", "scales", "cols")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, cols: int):
        nb = -(-cols // 32)
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise ValueError("MXTensor: uint8 codes and scales")
        if codes.shape[-1] != 16 * nb or scales.shape != codes.shape[:-1] + (nb,):
            raise ValueError(f"MXTensor: codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not hold {cols} columns")
        self.codes, self.scales, self.cols = codes, scales, cols

    @property
    def shape(self):
        return tuple(self.codes.shape[:-1]) + (self.cols,)


def empty(rows, cols: int, device="cuda") -> MXTensor:
    """Uninitialised codes and scales; rows is a number or the leading shape."""
    lead = (rows,) if isinstance(rows, int) else tuple(rows)
    nb = -(-cols // 32)
    return MXTensor(torch.empty(lead + (16 * nb,), dtype=torch.uint8, device=device),
                    torch.empty(lead + (nb,), dtype=torch.uint8, device=device), cols)


def quantize(x: torch.Tensor, out: MXTensor = None) -> MXTensor:
    """fp32 or bf16 x [..., rows, cols] (strided rows if 2-D) to 4 bits."""
    if out is None:
        out = empty(x.shape[:-1], x.shape[-1], x.device)
    if x.dim() != 2 or out.codes.dim() != 2:
        if out.shape != tuple(x.shape):
            raise ValueError(f"out holds {out.shape}, not {tuple(x.shape)}")
        x = x.reshape(-1, x.shape[-1])
    L.moe_mx_quantize(x, out.codes, out.scales, out.cols)
    return out


def dequantize(q: MXTensor, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor = None) -> torch.Tensor:
    """The values of q, in out's type (dtype if out is None); exact in both."""
    if out is None:
        out = torch.empty(q.shape, dtype=dtype, device=q.codes.device)
    flat = out
    if out.dim() != 2 or q.codes.dim() != 2:
        if tuple(out.shape) != q.shape:
            raise ValueError(f"out: shape {q.shape}, not {tuple(out.shape)}")
        flat = out.view(-1, out.shape[-1])
    L.moe_mx_dequantize(q.codes, q.scales, q.cols, flat)
    return out


def matmul(a: MXTensor, b: MXTensor, offsets: torch.Tensor = None, out: torch.Tensor = None,
           out_dtype: torch.dtype = torch.bfloat16, err: torch.Tensor = None) -> torch.Tensor:
    """a [rows, K] times b [N, K] (or one of b [G, N, K] for each row) transposed.

    offsets: int32 [G+1] on the device, group g's rows are offsets[g] ..
    offsets[g+1]-1; rows of no group are left as they are in out.  err: int32
    [4], zeroed, receives a device error (see moe_mx_gemm); without it, an
    output left incomplete by a wait that ran out goes unreported.
    """
    if out is None:
        out = torch.empty((a.codes.shape[0], b.codes.shape[-2]), dtype=out_dtype, device=a.codes.device)
    L.moe_mx_gemm(a.codes, a.scales, a.cols, b.codes, b.scales, b.cols, offsets, out, err)
    return out
