"""64-bit definitions of the experts' products for their tests, with bounds of
what fp32 sums and one rounding at the end may be off (no code shared with the
package).

A sum of n products in 32 bits, in any order and truncated at each step, is off
by at most n 2^-23 of the sum of their magnitudes (products of two bf16 are
exact; a product of two fp32 adds half a step, 2^-24, which n + 2 covers).  A
rounding to the output's type adds at most finfo.eps / 2 of the value.
"""
import torch


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, ref, bound):
    """Every element within its bound; where the definition gives an infinity or a NaN, so does got.  What lies half a
    step or more beyond the largest value of got's type is an infinity of it."""
    top = (2 - half_step(got.dtype)) * 2.0 ** 127
    got, ref = got.double().cpu(), ref.cpu()
    bound = bound.cpu()
    ref = torch.where(ref.abs() >= top, ref.sign() * float("inf"), ref)
    finite = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), "NaNs differ"
    assert torch.equal(got[~finite & ~torch.isnan(ref)], ref[~finite & ~torch.isnan(ref)]), "infinities differ"
    over = ((got - ref).abs() - bound)[finite]
    assert over.numel() == 0 or over.max() <= 0, f"off by {over.max().item():.3e} more than the bound, at {int((over > 0).sum())} of {over.numel()}"


def ranges(offsets, rows):
    """[lo, hi) of each group: entries cut to [0, rows]."""
    if offsets is None:
        return [(0, rows)]
    cut = [min(max(int(v), 0), rows) for v in offsets]
    return [(a, max(a, b)) for a, b in zip(cut, cut[1:])]


def product(op, a, b, groups, out, out_dtype, accumulate=False):
    """(values, bounds) of op on a and b; out: what the output held."""
    a, b = a.double(), b.double()
    ref = out.double().clone()
    bound = torch.zeros_like(ref)
    for g, (lo, hi) in enumerate(groups):
        if op == "dw":
            x, w, at = a[lo:hi].mT, b[lo:hi], g
        else:
            x, w, at = a[lo:hi], (b[g].mT if op == "fwd" else b[g]), slice(lo, hi)
        n = x.shape[1]
        v = x @ w
        m = x.abs() @ w.abs()
        if accumulate:
            v, m = ref[at] + v, ref[at].abs() + m
        ref[at] = v
        bound[at] = (n + 2) * 2.0 ** -23 * m + half_step(out_dtype) * (v.abs() + (n + 2) * 2.0 ** -23 * m) + 1e-45
    return ref, bound


def swiglu(gate, up, weight, out_dtype):
    g, u = gate.double(), up.double()
    w = 1.0 if weight is None else weight.double()[:, None]
    h = w * g * torch.sigmoid(g) * u
    # four products and a sigmoid: 2^-20 of the value; its exponential's argument is off by |g| 2^-22
    return h, (2.0 ** -20 + g.abs() * 2.0 ** -22 + half_step(out_dtype)) * h.abs() + 1e-38


def swiglu_grad(dh, gate, up, weight):
    g, u, d = gate.double(), up.double(), dh.double()
    w = torch.ones_like(g[:, :1]) if weight is None else weight.double()[:, None]
    s = torch.sigmoid(g)
    rel = 2.0 ** -20 + g.abs() * 2.0 ** -22
    dg, du, terms = w * d * u * s * (1 + g * (1 - s)), w * d * g * s, d * g * s * u
    # dgate is the sum of s and silu (1 - s), which may cancel, and 1 - s is off by 2^-24 times what multiplies it
    parts = (w * d * u).abs() * (s + (g * s).abs() * (1 - s + 2.0 ** -3))
    e = half_step(gate.dtype)
    return ((dg, rel * parts + e * (dg.abs() + rel * parts) + 1e-38), (du, (rel + e) * du.abs() * (1 + rel) + 1e-38),
            (terms.sum(1), (rel * terms.abs()).sum(1) + (g.shape[1] + 2) * 2.0 ** -23 * terms.abs().sum(1) + 1e-38))


def int4_values(codes, scales, zeros, group):
    """64-bit values of codes [R, C/2]."""
    R, half = codes.shape
    c = torch.empty((R, 2 * half), dtype=torch.float64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = (codes % 16).double(), (codes // 16).double()
    at = torch.arange(2 * half, device=codes.device) // group
    return (c - (8.0 if zeros is None else zeros.double()[:, at])) * scales.double()[:, at]


def int4_quantize(x, group, zeros, scale_dtype):
    """(codes, scales, zeros) of fp32 or bf16 x [R, C], group by group; the scale's quotient is a 32-bit one."""
    R, C = x.shape
    nb = -(-C // group)
    codes = torch.zeros((R, C), dtype=torch.int64)
    scales, zs = torch.zeros((R, nb), dtype=scale_dtype), torch.full((R, nb), 8, dtype=torch.uint8)
    x = x.float().cpu()
    for b in range(nb):
        v = x[:, b * group:(b + 1) * group]
        lo, hi = v.amin(1).clamp(max=0), v.amax(1).clamp(min=0)
        if zeros:
            s = (hi / torch.full_like(hi, 15.0) - lo / torch.full_like(lo, 15.0)).to(scale_dtype)
        else:
            s = (torch.maximum(hi, -lo) / torch.full_like(hi, 7.0)).to(scale_dtype)
        s = torch.where(s == 0, torch.ones_like(s), s)
        bad = ~torch.isfinite(v).all(1)
        q = v.double() / s.double()[:, None]
        z = torch.round(-lo.double() / s.double()).clamp(0, 15) if zeros else torch.full((R,), 8.0, dtype=torch.float64)
        c = (torch.round(q) + z[:, None]).clamp(0, 15)
        codes[:, b * group:(b + 1) * group] = torch.where(bad[:, None], torch.zeros_like(c), c).long()
        scales[:, b] = torch.where(bad, torch.full_like(s, float("nan")), s)
        if zeros:
            zs[:, b] = torch.where(bad, torch.zeros_like(z), z).to(torch.uint8)
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).to(torch.uint8)
    return packed, scales, zs if zeros else None
