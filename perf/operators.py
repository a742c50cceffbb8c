"""Cases and plain forms of the block operators around the routed-MoE layer.

Four operators, as one decoder block uses them at serving time:

  norm      the norm before the layer (``norm.pre``), and the norm after it
            fused with the gate, the residual scale, the residual add and the
            next norm (``norm.post``)
  quant     microscaled 4-bit floating point (E2M1 elements, one power-of-two
            scale per 32 columns): quantise and read back
  product   the product of two microscaled 4-bit matrices, dense or grouped by
            expert over ragged row ranges
  few       the whole mixture-of-experts layer for a few tokens, with fp32,
            bf16, FP8 or microscaled 4-bit expert weights

``own`` False: ``run`` computes an operator in elementary torch operations in
32 bits; True: it calls this package.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token: norm after the layer, per-channel gate, residual, next block's norm
        dict(name="post_decode_T1", op="norm", form="post", T=1, D=4096, dtype="bf16", kind="rms", gate="channel",
             sigmoid=False, bias=False, next=True),
        # an odd-sized fp32 block with LayerNorm and a full sigmoid gate (rows unaligned to 16 bytes)
        dict(name="post_odd_f32_T301", op="norm", form="post", T=301, D=1023, dtype="f32", kind="layer", gate="full",
             sigmoid=True, bias=True, next=False),
        # prefill: the same fusion over 8192 tokens (HBM-bound)
        dict(name="post_prefill_T8192", op="norm", form="post", T=8192, D=4096, dtype="bf16", kind="rms",
             gate="channel", sigmoid=False, bias=False, next=True),
        # decode activations: x quantised before the expert products
        dict(name="quant_decode_T128", op="quant", rows=128, cols=4096, dtype="bf16"),
        # prefill activations, and a slab of fp32 expert weights of the same size when they are loaded
        dict(name="quant_prefill_T16384", op="quant", rows=16384, cols=4096, dtype="bf16"),
        # a few rows against one projection: bound by the weights' bytes and by latency
        dict(name="product_rows7", op="product", rows=7, N=4096, K=4096, G=1, zipf=0.0),
        # ragged expert groups (some empty, one of hundreds of rows), as the permutation leaves them
        dict(name="product_grouped_G64", op="product", rows=4001, N=1024, K=4096, G=64, zipf=1.2),
        # a prefill-sized dense product: bound by the tensor cores
        dict(name="product_dense_8192", op="product", rows=8192, N=4096, K=4096, G=1, zipf=0.0),
        # one token through the full-size layer, bf16 weights: 277 MB of the chosen experts
        dict(name="few_bf16_T1", op="few", dtype="bf16", T=1, D=4096, E=512, I=1024, k=10, zipf=0.0),
        # one token, 4-bit weights: the same layer at a quarter of the bytes
        dict(name="few_mxfp4_T1", op="few", dtype="mxfp4", T=1, D=4096, E=512, I=1024, k=10, zipf=0.0),
        # a small batch of sequences, FP8 weights, popular experts shared between tokens
        dict(name="few_fp8_T8", op="few", dtype="fp8", T=8, D=4096, E=256, I=1024, k=10, zipf=1.0),
        # a reduced fp32 layer with an odd token count: bound by latency
        dict(name="few_f32_T5", op="few", dtype="f32", T=5, D=512, E=32, I=256, k=4, zipf=1.2),
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]: half of them odd, half round."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = n | 1 if rng.random() < 0.5 else max(lo, n // 10 * 10)
    return min(hi, max(lo, n))


def draw(rng):
    op = rng.choice(["norm", "quant", "product", "few"])
    if op == "norm":
        form = rng.choice(["pre", "post", "post"])
        T = _size(rng, 1, 8192)
        D = _size(rng, 64, 8192) if rng.random() < 0.5 else rng.choice([128, 256, 512, 1024, 2048, 4096])
        dtype = rng.choice(["bf16", "f32"])
        T = max(1, min(T, 8192 * 4096 * 2 // (D * (2 if dtype == "bf16" else 4)) // 2))
        return dict(op="norm", form=form, T=T, D=D, dtype=dtype, kind=rng.choice(["rms", "layer"]),
                    gate=rng.choice(["none", "channel", "token", "full"]) if form == "post" else "none",
                    sigmoid=form == "post" and rng.random() < 0.5, bias=rng.random() < 0.5,
                    next=form == "post" and rng.random() < 0.5)
    if op == "quant":
        cols = _size(rng, 32, 8192)
        return dict(op="quant", rows=max(1, min(_size(rng, 1, 16384), 16384 * 4096 // (2 * cols))), cols=cols,
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "product":
        G = rng.choice([1, 1, 3, 8, 17, 64])
        K = 32 * _size(rng, 2, 128)
        N = _size(rng, 64, 4096)
        rows = min(_size(rng, 1, 8192), 8192 * 4096 // N)
        if G > 1:
            rows = min(rows, 4001)
        return dict(op="product", rows=rows, N=N, K=K, G=G, zipf=rng.choice([0.0, 1.2]))
    D, I = rng.choice([512, 1024, 2048, 4096]), rng.choice([256, 512, 1024])
    E = rng.choice([16, 33, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp8", "mxfp4", "f32"])
    if dtype == "f32":
        D, I = min(D, 1024), min(I, 512)
    return dict(op="few", dtype=dtype, T=rng.randint(1, 16), D=D, E=E, I=I, k=rng.choice([1, 2, 4, 8, 10]),
                zipf=rng.choice([0.0, 1.0]))


# ------------------------------------------------------- inputs (seeded)

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _mx_pack(v):
    """E2M1 codes (two per byte, even column in the low half) and E8M0 scales of fp32 v [..., K], K a multiple of 32."""
    b = v.reshape(v.shape[:-1] + (v.shape[-1] // 32, 32))
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax)[1] - 3).clamp(-127, 125)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    a = torch.ldexp(b, -e[..., None])
    c = a < 0
    a = a.abs()
    n = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    n = (n + 8 * c.to(torch.uint8)).reshape(v.shape)
    return n[..., 0::2] | (n[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _mx_weights(shape, g, std):
    """Normal weights as microscaled codes and scales, made in slabs of groups."""
    G, R, K = shape
    q = torch.empty((G, R, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((G, R, K // 32), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (R * K))
    for i in range(0, G, step):
        n = min(step, G - i)
        q[i:i + n], s[i:i + n] = _mx_pack(_randn((n, R, K), g, std))
    return q, s


def _fp8_weights(shape, g, std):
    """Normal weights as E4M3 codes and fp32 scales of 128 x 128 blocks, made in slabs of groups."""
    G, R, K = shape
    q = torch.empty((G, R, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((G, R // 128, K // 128), device="cuda")
    step = max(1, (1 << 26) // (R * K))
    for i in range(0, G, step):
        n = min(step, G - i)
        b = _randn((n, R // 128, 128, K // 128, 128), g, std)
        amax = b.abs().amax((2, 4), keepdim=True)
        q[i:i + n] = (b * (448 / amax)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(n, R, K)
        s[i:i + n] = (amax / 448).reshape(n, R // 128, K // 128)
    return q, s


def _bf16_weights(shape, g, std, dtype):
    w = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 26) // (shape[1] * shape[2]))
    for i in range(0, shape[0], step):
        n = min(step, shape[0] - i)
        w[i:i + n] = _randn((n,) + tuple(shape[1:]), g, std)
    return w


def _group_sizes(case, seed):
    """Rows of each group: drawn with the popularities of a random ranking, so some groups are empty."""
    g = torch.Generator().manual_seed(seed)
    G, rows = case["G"], case["rows"]
    p = (torch.randperm(G, generator=g) + 1.0) ** -case["zipf"]
    n = torch.bincount(torch.multinomial(p, rows, replacement=True, generator=g), minlength=G)
    return n


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "norm":
        T, D, dt = case["T"], case["D"], _DT[case["dtype"]]
        s = dict(case=case, x=_randn((T, D), g, 1.5, dt))
        s["w"] = (1 + 0.1 * _randn((D,), g)).to(dt)
        s["b"] = _randn((D,), g, 0.1, dt) if case["bias"] else None
        s["out"] = torch.empty((T, D), dtype=dt, device="cuda")
        if case["form"] == "post":
            s["res"] = _randn((T, D), g, 2.0, dt)
            shape = {"none": None, "channel": (D,), "token": (T,), "full": (T, D)}[case["gate"]]
            s["gate"] = None if shape is None else _randn(shape, g, 1.0, dt)
            s["next_w"] = (1 + 0.1 * _randn((D,), g)).to(dt) if case["next"] else None
            s["next_out"] = torch.empty((T, D), dtype=dt, device="cuda") if case["next"] else None
        return s
    if case["op"] == "quant":
        x = _randn((case["rows"], case["cols"]), g)
        # activations: a few channels are far larger than the rest
        x *= torch.exp(1.5 * torch.randn((case["cols"],), generator=g, device="cuda"))
        s = dict(case=case, x=x.to(_DT[case["dtype"]]))
        s["back"] = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
        if own:
            from sparse_moe_expert_02_gb300 import mx
            s["q"] = mx.empty(case["rows"], case["cols"])
        return s
    if case["op"] == "product":
        rows, N, K, G = case["rows"], case["N"], case["K"], case["G"]
        s = dict(case=case)
        s["aq"], s["as"] = _mx_pack(_randn((rows, K), g))
        s["bq"], s["bs"] = _mx_weights((G, N, K), g, K ** -0.5)
        n = _group_sizes(case, seed)
        s["most"] = int(n.max())
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).to(torch.int32).cuda()
        s["out"] = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
        if own:
            from sparse_moe_expert_02_gb300 import mx
            s["a"] = mx.MXTensor(s["aq"], s["as"], K)
            s["b"] = mx.MXTensor(s["bq"], s["bs"], K)
        return s
    D, E, I, k, dtype = case["D"], case["E"], case["I"], case["k"], case["dtype"]
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    w = dict(w_router=_randn((E, D), g, D ** -0.5, dt))
    rank = torch.randperm(E, generator=g, device="cuda") + 1.0
    w["b_router"] = -case["zipf"] * torch.log(rank)
    for name, shape, std in (("gate", (E + 1, I, D), D ** -0.5), ("up", (E + 1, I, D), D ** -0.5),
                             ("down", (E + 1, D, I), I ** -0.5)):
        if dtype == "mxfp4":
            w["w_" + name], w["s_" + name] = _mx_weights(shape, g, std)
        elif dtype == "fp8":
            w["w_" + name], w["s_" + name] = _fp8_weights(shape, g, std)
        else:
            w["w_" + name] = _bf16_weights(shape, g, std, dt)
    s = dict(case=case, w=w, x=_randn((case["T"], D), g, 1.0, dt))
    s["out"] = torch.empty((case["T"], D), dtype=dt, device="cuda")
    if own:
        from sparse_moe_expert_02_gb300 import MoELayer
        s["layer"] = MoELayer(D, E, I, k, dtype, w, T_max=case["T"], has_router_bias=True,
                              out_dtype="f32" if dtype == "f32" else "bf16")
    return s


# ------------------------------------------------------------ plain forms

def _norm_plain(x, w, b, kind):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    x = x * w.float()
    return x if b is None else x + b.float()


def _plain_norm(s):
    case = s["case"]
    n = _norm_plain(s["x"].float(), s["w"], s["b"], case["kind"])
    if case["form"] == "pre":
        return n.to(s["x"].dtype)
    if s["gate"] is not None:
        a = s["gate"].float()
        a = 1 / (1 + torch.exp(-a)) if case["sigmoid"] else a
        n = n * (a[:, None] if case["gate"] == "token" else a)
    r = 0.75 * s["res"].float() + 1.25 * n
    out = r.to(s["x"].dtype)
    # the next norm sees the residual stream as it is stored
    return [out] if s["next_w"] is None else [out, _norm_plain(out.float(), s["next_w"], None, case["kind"]).to(out.dtype)]


def _mx_values(q, s):
    """fp32 values of codes and scales."""
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=q.device)
    v = torch.stack([lut[(q & 15).int()], lut[(q >> 4).int()]], -1).reshape(q.shape[:-1] + (q.shape[-1] // 16, 32))
    return torch.ldexp(v, (s.int() - 127)[..., None]).reshape(q.shape[:-1] + (2 * q.shape[-1],))


def _plain_quant(s):
    x = s["x"].float()
    cols = x.shape[1]
    x = torch.nn.functional.pad(x, (0, -cols % 32))
    return _mx_values(*_mx_pack(x))[:, :cols].to(torch.bfloat16)


def _plain_product(s):
    a, b = _mx_values(s["aq"], s["as"]), _mx_values(s["bq"], s["bs"])
    if s["case"]["G"] == 1:
        return (a @ b[0].T).to(torch.bfloat16)
    row = torch.arange(a.shape[0], device=a.device)
    group = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    place = row - s["offsets"].long()[group]
    padded = torch.zeros((s["case"]["G"], s["most"], a.shape[1]), device=a.device)
    padded[group, place] = a
    return (padded @ b.transpose(1, 2))[group, place].to(torch.bfloat16)


def _fp8_values(q, s):
    v = q.view(torch.float8_e4m3fn).float()
    b = v.reshape(v.shape[:-2] + (s.shape[-2], 128, s.shape[-1], 128))
    return (b * s[..., :, None, :, None]).reshape(v.shape)


def _as_read(v, dtype):
    """Activations as the expert products of a layer type read them."""
    if dtype == "mxfp4":
        return _mx_values(*_mx_pack(v))
    if dtype == "fp8":
        b = v.reshape(v.shape[:-1] + (v.shape[-1] // 128, 128))
        amax = b.abs().amax(-1, keepdim=True)
        amax = torch.where(amax > 0, amax, torch.full_like(amax, 448.0))
        most = torch.full_like(amax, 448.0)  # a tensor: a division, not a product with a reciprocal
        c = (b * (most / amax)).clamp(-448, 448).to(torch.float8_e4m3fn).float()
        return (c * (amax / most)).reshape(v.shape)
    return v


def _plain_few(s):
    case, w, x = s["case"], s["w"], s["x"].float()
    dtype, E, k = case["dtype"], case["E"], case["k"]
    z = x @ w["w_router"].float().T + w["b_router"]
    zs, idx = torch.sort(z, dim=-1, descending=True, stable=True)
    p = torch.exp(zs[:, :k] - zs[:, :1])
    p = p / p.sum(-1, keepdim=True)
    idx = torch.cat([idx[:, :k], torch.full_like(idx[:, :1], E)], 1)
    p = torch.cat([p, torch.ones_like(p[:, :1])], 1)

    def taken(name):
        q = w["w_" + name][idx]
        if dtype == "mxfp4":
            return _mx_values(q, w["s_" + name][idx])
        return _fp8_values(q, w["s_" + name][idx]) if dtype == "fp8" else q.float()

    v = _as_read(x, dtype)[:, None, :, None]
    a, u = (taken("gate") @ v)[..., 0], (taken("up") @ v)[..., 0]
    h = _as_read(a / (1 + torch.exp(-a)) * u, dtype)
    y = (taken("down") @ h[..., None])[..., 0]
    return (p[..., None] * y).sum(1).to(s["x"].dtype)


def run(s):
    case = s["case"]
    if not own:
        return {"norm": _plain_norm, "quant": _plain_quant, "product": _plain_product, "few": _plain_few}[case["op"]](s)
    from sparse_moe_expert_02_gb300 import mx, norm
    if case["op"] == "norm":
        if case["form"] == "pre":
            return norm.pre(s["x"], s["w"], s["b"], kind=case["kind"], eps=1e-6, out=s["out"])
        out, after = norm.post(s["x"], s["res"], s["w"], s["b"], kind=case["kind"], eps=1e-6, gate=s["gate"],
                               gate_by=case["gate"], gate_sigmoid=case["sigmoid"], res_scale=0.75, branch_scale=1.25,
                               next_w=s["next_w"], out=s["out"], next_out=s["next_out"])
        return [out] if after is None else [out, after]
    if case["op"] == "quant":
        return mx.dequantize(mx.quantize(s["x"], out=s["q"]), out=s["back"])
    if case["op"] == "product":
        return mx.matmul(s["a"], s["b"], offsets=s["offsets"], out=s["out"])
    return s["layer"].forward_few(s["x"], out=s["out"])


# ------------------------------------------------------------------- work

def work(case):
    """Each input read once, each output written once; the layer reads the experts that T tokens touch on average."""
    if case["op"] == "norm":
        n = case["T"] * case["D"] * (2 if case["dtype"] == "bf16" else 4)
        post = case["form"] == "post"
        tensors = 2 + post + (post and case["next"]) + (case["gate"] == "full")
        return dict(bytes=n * tensors, flops=case["T"] * case["D"] * (14 if post else 5))
    if case["op"] == "quant":
        n = case["rows"] * case["cols"]
        return dict(bytes=n * ((2 if case["dtype"] == "bf16" else 4) + 17 / 32 + 2), flops=4 * n)
    if case["op"] == "product":
        r, N, K, G = case["rows"], case["N"], case["K"], case["G"]
        p = torch.arange(1, G + 1, dtype=torch.float64) ** -case["zipf"]
        touched = float((1 - (1 - p / p.sum()) ** r).sum())
        return dict(bytes=(r + touched * N) * K * 17 / 32 + 2 * r * N, flops=2.0 * r * N * K)
    T, D, E, I, k = (case[n] for n in ("T", "D", "E", "I", "k"))
    p = torch.arange(1, E + 1, dtype=torch.float64) ** -case["zipf"]
    touched = 1 + float((1 - (1 - p / p.sum()).clamp(min=0) ** (T * k)).sum()) if T > 1 else 1 + k
    per = {"f32": 4, "bf16": 2, "fp8": 1 + 1 / 4096, "mxfp4": 17 / 32}[case["dtype"]]
    act = 4 if case["dtype"] == "f32" else 2
    return dict(bytes=touched * 3 * D * I * per + E * D * act + 2 * T * D * act,
                flops=T * (2.0 * D * E + (k + 1) * 6.0 * D * I))


# -------------------------------------------------- the definition in 64 bits

def _exact_norm(v, w, b, kind):
    mu = v.sum(-1, keepdim=True) / v.shape[-1] if kind == "layer" else torch.zeros_like(v[..., :1])
    d = v - mu
    y = d / torch.sqrt((d * d).sum(-1, keepdim=True) / v.shape[-1] + 1e-6) * w.double()
    return y + b.double() if b is not None else y


def _exact_mx(v):
    """The values that v [R, K] in 64 bits has once it is held in microscaled 4 bits."""
    R, K = v.shape
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)
    b = torch.nn.functional.pad(v, (0, -K % 32)).reshape(R, -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    top = torch.where(top > 0, top, torch.ones_like(top))
    unit = torch.exp2(torch.floor(torch.log2(top)))
    unit = torch.where(2 * unit <= top, 2 * unit, torch.where(unit > top, unit / 2, unit)) / 4
    r = b.abs() / unit
    hi = torch.searchsorted(grid, r.contiguous()).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    dl, dh = r - grid[lo], grid[hi] - r
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (r >= 6)
    return (torch.where(up, grid[hi], grid[lo]) * unit * torch.sign(b)).reshape(R, -1)[:, :K]


def _exact_codes(q, s):
    """The values of packed codes and scales, by the fields of each code."""
    n = torch.stack([q % 16, q // 16], -1).reshape(q.shape[0], -1).double()
    sign = torch.where(n >= 8, -1.0, 1.0)
    m = n % 8
    e, f = torch.floor(m / 2), m % 2
    mag = torch.where(e == 0, f / 2, torch.exp2(e - 1) * (1 + f / 2))
    return sign * mag * torch.exp2(s.double() - 127).repeat_interleave(32, -1)


def _exact_e4m3(v):
    """v [R, K] in 64 bits, quantised by rows and groups of 128 columns; the type rounds 448/amax and its product to 32 bits."""
    b = v.reshape(v.shape[0], -1, 128)
    top = b.abs().amax(-1, keepdim=True)
    top = torch.where(top > 0, top, torch.full_like(top, 448.0))
    r = (b * (448 / top).float().double()).float().double()
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -30))), min=-6.0) - 3)
    return ((torch.round(r / step) * step).clamp(-448, 448) * (top / 448)).reshape(v.shape)


def _exact_few(s):
    case, w, x = s["case"], s["w"], s["x"].double()
    dtype, E, k = case["dtype"], case["E"], case["k"]

    def matrix(name, e):
        q = w["w_" + name][e]
        if dtype == "mxfp4":
            return _exact_codes(q, w["s_" + name][e])
        if dtype == "fp8":
            sc = w["s_" + name][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            return q.view(torch.float8_e4m3fn).double() * sc
        return q.double()

    held = {"mxfp4": _exact_mx, "fp8": _exact_e4m3}.get(dtype, lambda v: v)
    z = (x @ w["w_router"].double().T + w["b_router"].double()).cpu()
    out = torch.zeros_like(x)
    for t in range(x.shape[0]):
        order = sorted(range(E), key=lambda e: (-float(z[t, e]), e))[:k]
        p = torch.softmax(z[t, order], 0)
        v = held(x[t:t + 1])
        for e, weight in [(E, 1.0)] + list(zip(order, p.tolist())):
            a, u = v @ matrix("gate", e).T, v @ matrix("up", e).T
            out[t] += weight * (held(a * torch.sigmoid(a) * u) @ matrix("down", e).T)[0]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        y = _exact_norm(s["x"].double(), s["w"], s["b"], case["kind"])
        if case["form"] == "pre":
            return y
        if s["gate"] is not None:
            a = s["gate"].double()
            a = torch.sigmoid(a) if case["sigmoid"] else a
            y = y * (a.unsqueeze(1) if case["gate"] == "token" else a)
        out = 0.75 * s["res"].double() + 1.25 * y
        if s["next_w"] is None:
            return [out]
        # the next norm is of the stored (rounded) residual stream
        return [out, _exact_norm(out.to(s["x"].dtype).double(), s["next_w"], None, case["kind"])]
    if case["op"] == "quant":
        return _exact_mx(s["x"].double())
    if case["op"] == "product":
        a = _exact_codes(s["aq"], s["as"])
        out = torch.zeros((case["rows"], case["N"]), dtype=torch.float64, device=a.device)
        at = s["offsets"].tolist()
        for i in range(case["G"]):
            if at[i + 1] > at[i]:
                out[at[i]:at[i + 1]] = a[at[i]:at[i + 1]] @ _exact_codes(s["bq"][i], s["bs"][i]).T
        return out
    return _exact_few(s)
