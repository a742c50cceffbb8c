"""64-bit numpy definitions of the block operators, for their tests (no code
shared with the package)."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], np.float64)


def norm(v, kind, eps, w=None, b=None, w_offset=0.0):
    v = np.asarray(v, np.float64)
    if kind == "none":
        return v
    mu = v.mean(-1, keepdims=True) if kind == "layer" else 0.0
    d = v - mu
    y = d / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * (w + w_offset)
    return y if b is None else y + b


def mx_quantize(x):
    """(codes [R, 16*nb] uint8, scales [R, nb] uint8) of float32 x [R, C], block by block."""
    R, C = x.shape
    nb = -(-C // 32)
    v = np.zeros((R, nb * 32), np.float64)
    v[:, :C] = x
    v = v.reshape(R, nb, 32)
    codes = np.zeros((R, nb, 32), np.uint8)
    scales = np.full((R, nb), 127, np.uint8)
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    for r in range(R):
        for k in range(nb):
            a = np.abs(v[r, k])
            m = a.max()
            if not np.isfinite(a).all():
                scales[r, k] = 255
                continue
            e = 0
            if m > 0:
                e = max(int(np.frexp(m)[1]) - 1 - 2, -127)
            scales[r, k] = e + 127
            q = np.ldexp(a, -e)
            lo = np.searchsorted(mid, q, side="left")   # ties stay below ...
            hi = np.searchsorted(mid, q, side="right")  # ... or go above
            i = np.where((lo != hi) & (lo % 2 == 1), hi, lo)  # the even code of a tie
            codes[r, k] = i + 8 * np.signbit(v[r, k])
    c = codes.reshape(R, nb * 32)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8), scales


def mx_values(codes, scales):
    """float64 values [..., 32*nb]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    f = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(f, 32, -1)


def mx_round(v):
    """v [R, C] as microscaled 4 bits hold it (v is rounded to float32 first, as a kernel holds it)."""
    q, s = mx_quantize(np.asarray(v, np.float32))
    return mx_values(q, s)[:, :v.shape[1]]


def topk(z, k):
    """(indices, weights) of one row of logits: largest first, the lower index on a tie."""
    idx = np.lexsort((np.arange(len(z)), -z))[:k]
    p = np.exp(z[idx] - z[idx[0]])
    return idx, p / p.sum()


def mx_layer(x, idx, w, gate, up, down):
    """The layer over microscaled weights given as float64 values [E+1, ...]; x float64 [T, D]."""
    E = gate.shape[0] - 1
    out = np.zeros((x.shape[0], down.shape[1]))
    for t in range(x.shape[0]):
        v = mx_round(x[t:t + 1])[0]
        for e, p in [(E, 1.0)] + list(zip(idx[t], w[t])):
            a, u = gate[e] @ v, up[e] @ v
            h = mx_round((a / (1 + np.exp(-a)) * u)[None])[0]
            out[t] += p * (down[e] @ h)
    return out
