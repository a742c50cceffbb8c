"""The experts' products and what lies between them, for training and for
weights that a layer call does not run (moe_grouped_gemm and its gradients,
moe_swiglu, moe_swiglu_grad).

    out_r = W_g x_r             matmul
    dx_r  = W_g^T dy_r          matmul_dx
    dW_g  = sum_r dy_r x_r^T    matmul_dw
    h_r   = weight_r silu(gate_r) up_r     swiglu, swiglu_grad

for the rows r of group g: offsets[g] .. offsets[g+1]-1, int32 [G+1] on the
device (as the layer's permutation writes them); None: one group of all rows.
Rows of no group are not read, and are left as they are in out.  Rows are
[rows, columns] tensors in fp32 or bf16 and may be strided views; weights are
contiguous [G, N, K] or [N, K].  Tensors are on the current device and used on
its current stream.

err: int32 [4], zeroed, receives a device error (see the C header); without
it, an output left incomplete by a wait that ran out goes unreported.
"""
from __future__ import annotations

import torch

from . import _lib as L


def matmul(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor = None, out: torch.Tensor = None,
           out_dtype: torch.dtype = None, err: torch.Tensor = None) -> torch.Tensor:
    """x [rows, K] times its group's w [N, K] transposed, in out_dtype (x's if None)."""
    if out is None:
        out = torch.empty((x.shape[0], w.shape[-2]), dtype=out_dtype or x.dtype, device=x.device)
    L.moe_grouped_gemm(x, w, offsets, out, err)
    return out


def matmul_dx(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor = None, out: torch.Tensor = None,
              out_dtype: torch.dtype = None, err: torch.Tensor = None) -> torch.Tensor:
    """The gradient of matmul by its rows: dy [rows, N] times its group's w [N, K]."""
    if out is None:
        out = torch.empty((dy.shape[0], w.shape[-1]), dtype=out_dtype or dy.dtype, device=dy.device)
    L.moe_grouped_gemm_dx(dy, w, offsets, out, err)
    return out


def matmul_dw(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor = None, out: torch.Tensor = None,
              out_dtype: torch.dtype = None, accumulate: bool = False, err: torch.Tensor = None) -> torch.Tensor:
    """The gradient of matmul by its weights, [G, N, K] (no offsets: [N, K]): for each group, dy [rows, N] transposed
    times x [rows, K].  A group without rows gets zeros; accumulate adds to what out holds."""
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an out to add to")
        lead = () if offsets is None else (offsets.shape[0] - 1,)
        out = torch.empty(lead + (dy.shape[1], x.shape[1]), dtype=out_dtype or x.dtype, device=x.device)
    L.moe_grouped_gemm_dw(dy, x, offsets, out, accumulate, err)
    return out


def swiglu(gate: torch.Tensor, up: torch.Tensor, weight: torch.Tensor = None, out: torch.Tensor = None,
           out_dtype: torch.dtype = None) -> torch.Tensor:
    """weight * silu(gate) * up; gate, up [rows, I] (they may be halves of one buffer), weight fp32 [rows] or None (1).
    out may be gate or up itself."""
    if out is None:
        out = torch.empty(gate.shape, dtype=out_dtype or gate.dtype, device=gate.device)
    L.moe_swiglu(gate, up, weight, out)
    return out


def swiglu_grad(dh: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, weight: torch.Tensor = None, dgate: torch.Tensor = None,
                dup: torch.Tensor = None, dweight: torch.Tensor = None):
    """(dgate, dup, dweight) of swiglu; dweight fp32 [rows], where weight or dweight is given (else None).
    dgate and dup may be any of the inputs."""
    if dgate is None:
        dgate = torch.empty(gate.shape, dtype=gate.dtype, device=gate.device)
    if dup is None:
        dup = torch.empty(up.shape, dtype=up.dtype, device=up.device)
    if dweight is None and weight is not None:
        dweight = torch.empty(weight.shape, dtype=torch.float32, device=gate.device)
    L.moe_swiglu_grad(dh, gate, up, weight, dgate, dup, dweight)
    return dgate, dup, dweight
