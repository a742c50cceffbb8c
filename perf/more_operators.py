"""Cases and plain forms of the experts' products around the routed-MoE layer.

Three operators, as an expert's feed-forward runs them where the layer call
itself does not: when its weights are trained, and when they are held in four
bits beside 16- or 32-bit activations.

  product   rows grouped by expert times their expert's matrix, and its two
            gradients: ``grouped.matmul`` (out_r = W_g x_r), ``matmul_dx``
            (dx_r = W_g^T dy_r) and ``matmul_dw`` (dW_g = sum over the group's
            rows of dy_r x_r^T)
  act       the gated activation between two of them with the routing weight
            of a row, h = weight * silu(gate) * up (``grouped.swiglu``), and
            its gradient (``grouped.swiglu_grad``)
  int4      rows times a matrix (or one of several, by group) of 4-bit codes
            with a scale, and if asked for a zero point, per 32, 64 or 128
            columns (``int4.matmul``)

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
        # a few decoded tokens over eight experts' up projection: bound by the weights' bytes and by latency
        dict(name="fwd_decode_rows13", op="product", dir="fwd", rows=13, N=1024, K=4096, G=8, zipf=0.0, pad=0, dtype="bf16",
             out="bf16"),
        # a small fp32 layer with sizes that nothing divides, and rows behind the last group
        dict(name="fwd_odd_f32", op="product", dir="fwd", rows=501, N=255, K=513, G=5, zipf=1.2, pad=11, dtype="f32", out="f32"),
        # ragged groups of a mid-sized batch (some empty, one of hundreds of rows): bound by the weights' bytes
        dict(name="fwd_ragged_G64", op="product", dir="fwd", rows=4001, N=1024, K=4096, G=64, zipf=1.2, pad=0, dtype="bf16",
             out="bf16"),
        # a prefill-sized product over a few large experts: bound by the tensor cores
        dict(name="fwd_prefill_G8", op="product", dir="fwd", rows=16384, N=4096, K=4096, G=8, zipf=0.6, pad=0, dtype="bf16",
             out="bf16"),
        # a training step's gradient of the rows: 1638 tokens of ten experts each
        dict(name="dx_train_G64", op="product", dir="dx", rows=16380, N=1024, K=4096, G=64, zipf=0.6, pad=4, dtype="bf16",
             out="bf16"),
        # the same step's gradient of the weights, kept in fp32 for the optimiser
        dict(name="dw_train_G64", op="product", dir="dw", rows=16380, N=1024, K=4096, G=64, zipf=0.6, pad=4, dtype="bf16",
             out="f32"),
        # gradient of odd-sized weights, rows unaligned to 16 bytes
        dict(name="dw_odd_bf16", op="product", dir="dw", rows=777, N=129, K=257, G=7, zipf=1.2, pad=0, dtype="bf16", out="bf16"),
        # the activation of eight tokens' ten experts each
        dict(name="act_decode_rows80", op="act", dir="fwd", rows=80, I=1024, dtype="bf16", weight=True, halves=True),
        # a training step over 8192 tokens of ten experts each: the activation's gradient (HBM-bound)
        dict(name="act_grad_rows81920", op="act", dir="grad", rows=81920, I=1024, dtype="bf16", weight=True, halves=True),
        # one token through one 4-bit projection: latency and 8.7 MB
        dict(name="int4_T1", op="int4", rows=1, N=4096, K=4096, G=1, zipf=0.0, pad=0, group=128, zeros=False, scale="bf16",
             dtype="bf16"),
        # eight tokens over 4-bit experts with zero points, in groups as the permutation leaves them
        dict(name="int4_experts_rows80", op="int4", rows=80, N=1024, K=4096, G=128, zipf=1.0, pad=0, group=64, zeros=True,
             scale="bf16", dtype="bf16"),
        # a prompt of 2047 tokens through the same projection
        dict(name="int4_prompt_rows2047", op="int4", rows=2047, N=4096, K=4096, G=1, zipf=0.0, pad=0, group=128, zeros=False,
             scale="bf16", dtype="bf16"),
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]: half of them odd, half multiples of 8 where there is room for one."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = n | 1 if rng.random() < 0.5 else max(lo, n // 8 * 8)
    return min(hi, max(lo, n))


def draw(rng):
    op = rng.choice(["product", "product", "act", "int4"])
    if op == "product":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        G = rng.choice([1, 1, 2, 5, 8, 17, 64, 128])
        N, K = _size(rng, 16, 4096), _size(rng, 16, 4096)
        while G * N * K > 64 * 1024 * 4096:
            G = G // 2
        rows = _size(rng, 1, 16384)
        if dtype == "f32":  # no tensor cores: a smaller share of the range
            rows = max(1, min(rows, 2 ** 33 // (N * K)))
        return dict(op="product", dir=rng.choice(["fwd", "dx", "dw"]), rows=rows, N=N, K=K, G=G, zipf=rng.choice([0.0, 0.6, 1.2]),
                    pad=rng.choice([0, 0, 3, 64]), dtype=dtype, out="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]))
    if op == "act":
        size = _size(rng, 16, 4096)
        return dict(op="act", dir=rng.choice(["fwd", "grad"]), rows=max(1, min(_size(rng, 1, 81920), 81920 * 512 // size)), I=size,
                    dtype=rng.choice(["bf16", "f32"]), weight=rng.random() < 0.5, halves=rng.random() < 0.5)
    G = rng.choice([1, 1, 3, 16, 128])
    N, K = _size(rng, 16, 4096), 32 * _size(rng, 1, 128)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    rows = rng.choice([rng.randint(1, 16), _size(rng, 1, 2047)])
    if dtype == "f32":
        rows = max(1, min(rows, 2 ** 33 // (N * K)))
    return dict(op="int4", rows=rows, N=N, K=K, G=G, zipf=rng.choice([0.0, 1.0]), pad=rng.choice([0, 0, 5]),
                group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5, scale=rng.choice(["bf16", "f32"]), dtype=dtype)


# ------------------------------------------------------- inputs (seeded)

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _weights(shape, g, std, dtype):
    w = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 26) // (shape[1] * shape[2]))
    for i in range(0, shape[0], step):
        n = min(step, shape[0] - i)
        w[i:i + n] = _randn((n,) + tuple(shape[1:]), g, std)
    return w


def _groups(case, seed):
    """First row of each group and the end of the last: sizes drawn with the popularities of a random ranking, so some are empty."""
    g = torch.Generator().manual_seed(seed)
    p = (torch.randperm(case["G"], generator=g) + 1.0) ** -case["zipf"]
    n = torch.bincount(torch.multinomial(p, case["rows"], replacement=True, generator=g), minlength=case["G"])
    return [0] + n.cumsum(0).tolist()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "act":
        rows, I, dt = case["rows"], case["I"], _DT[case["dtype"]]
        if case["halves"]:  # both products in one buffer, the gate's columns first
            both = _randn((rows, 2 * I), g, 1.5, dt)
            s["gate"], s["up"] = both[:, :I], both[:, I:]
        else:
            s["gate"], s["up"] = _randn((rows, I), g, 1.5, dt), _randn((rows, I), g, 1.5, dt)
        # the routing weights of ten experts a token
        s["weight"] = torch.rand((rows,), generator=g, device="cuda") * 0.2 if case["weight"] else None
        s["out"] = torch.empty((rows, I), dtype=dt, device="cuda")
        if case["dir"] == "grad":
            s["dh"] = _randn((rows, I), g, 0.1, dt)
            s["out2"] = torch.empty((rows, I), dtype=dt, device="cuda")
            s["dweight"] = torch.empty((rows,), device="cuda") if case["weight"] else None
        return s
    rows, N, K, G = case["rows"] + case["pad"], case["N"], case["K"], case["G"]
    s["at"] = _groups(case, seed)
    s["offsets"] = torch.tensor(s["at"], dtype=torch.int32).cuda()
    dt = _DT[case["dtype"]]
    if case["op"] == "product":
        if case["dir"] != "dw":
            s["w"] = _weights((G, N, K), g, K ** -0.5, dt)
        if case["dir"] != "dx":
            s["x"] = _randn((rows, K), g, 1.0, dt)
        if case["dir"] != "fwd":
            s["dy"] = _randn((rows, N), g, 0.1, dt)
        # rows behind the last group keep what they held
        shape = {"fwd": (rows, N), "dx": (rows, K), "dw": (G, N, K)}[case["dir"]]
        s["out"] = torch.zeros(shape, dtype=_DT[case["out"]], device="cuda")
        return s
    nb = -(-K // case["group"])
    s["x"] = _randn((rows, K), g, 1.0, dt)
    s["codes"] = torch.randint(0, 256, (G, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s["scales"] = ((0.5 + torch.rand((G, N, nb), generator=g, device="cuda")) * (K ** -0.5 / 4.6)).to(_DT[case["scale"]])
    s["zeros"] = torch.randint(5, 11, (G, N, nb), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
    s["out"] = torch.zeros((rows, N), dtype=dt, device="cuda")
    if own:
        from sparse_moe_expert_02_gb300 import int4
        s["w"] = int4.I4Tensor(s["codes"], s["scales"], s["zeros"], K, case["group"])
    return s


# ------------------------------------------------------------ plain forms

def _plain_product(s):
    d, at = s["case"]["dir"], s["at"]
    out = s["out"].clone()
    for g in range(len(at) - 1):
        a, b = at[g], at[g + 1]
        if d == "fwd":
            out[a:b] = (s["x"][a:b].float() @ s["w"][g].float().T).to(out.dtype)
        elif d == "dx":
            out[a:b] = (s["dy"][a:b].float() @ s["w"][g].float()).to(out.dtype)
        else:
            out[g] = (s["dy"][a:b].float().T @ s["x"][a:b].float()).to(out.dtype)
    return out


def _plain_act(s):
    a, u = s["gate"].float(), s["up"].float()
    sig = 1 / (1 + torch.exp(-a))
    w = 1.0 if s["weight"] is None else s["weight"][:, None]
    if s["case"]["dir"] == "fwd":
        return (a * sig * u * w).to(s["out"].dtype)
    dh = s["dh"].float()
    out = [(dh * w * u * sig * (1 + a * (1 - sig))).to(s["out"].dtype), (dh * w * a * sig).to(s["out"].dtype)]
    if s["weight"] is not None:
        out.append((dh * a * sig * u).sum(1))
    return out


def _values(codes, scales, zeros, K, group):
    """fp32 values of 4-bit codes [N, K/2]: the even column in the low half of a byte."""
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], K).float()
    z = 8.0 if zeros is None else zeros.float().repeat_interleave(group, 1)[:, :K]
    return (c - z) * scales.float().repeat_interleave(group, 1)[:, :K]


def _plain_int4(s):
    case, at = s["case"], s["at"]
    out = s["out"].clone()
    for g in range(len(at) - 1):
        a, b = at[g], at[g + 1]
        if b > a:
            w = _values(s["codes"][g], s["scales"][g], None if s["zeros"] is None else s["zeros"][g], case["K"], case["group"])
            out[a:b] = (s["x"][a:b].float() @ w.T).to(out.dtype)
    return out


def run(s):
    case = s["case"]
    if not own:
        return {"product": _plain_product, "act": _plain_act, "int4": _plain_int4}[case["op"]](s)
    from sparse_moe_expert_02_gb300 import grouped, int4
    if case["op"] == "product":
        if case["dir"] == "fwd":
            return grouped.matmul(s["x"], s["w"], s["offsets"], out=s["out"])
        if case["dir"] == "dx":
            return grouped.matmul_dx(s["dy"], s["w"], s["offsets"], out=s["out"])
        return grouped.matmul_dw(s["dy"], s["x"], s["offsets"], out=s["out"])
    if case["op"] == "act":
        if case["dir"] == "fwd":
            return grouped.swiglu(s["gate"], s["up"], s["weight"], out=s["out"])
        got = grouped.swiglu_grad(s["dh"], s["gate"], s["up"], s["weight"], dgate=s["out"], dup=s["out2"], dweight=s["dweight"])
        return [t for t in got if t is not None]
    return int4.matmul(s["x"], s["w"], s["offsets"], out=s["out"])


# ------------------------------------------------------------------- work

def _touched(case):
    """Groups that get a row, on average."""
    p = torch.arange(1, case["G"] + 1, dtype=torch.float64) ** -case["zipf"]
    return float((1 - (1 - p / p.sum()).clamp(min=0) ** case["rows"]).sum())


def work(case):
    """Each input read once, each output written once; a product reads the matrices that have a row."""
    if case["op"] == "act":
        n, e = case["rows"] * case["I"], 2 if case["dtype"] == "bf16" else 4
        grad = case["dir"] == "grad"
        return dict(bytes=n * e * (5 if grad else 3) + (case["rows"] * (8 if grad else 4) if case["weight"] else 0),
                    flops=n * (14 if grad else 6))
    rows, N, K, G = case["rows"], case["N"], case["K"], case["G"]
    e = 2 if case["dtype"] == "bf16" else 4
    flops = 2.0 * rows * N * K
    if case["op"] == "int4":
        per = N * (K / 2 + -(-K // case["group"]) * ((2 if case["scale"] == "bf16" else 4) + (1 if case["zeros"] else 0)))
        return dict(bytes=_touched(case) * per + rows * (K + N) * e, flops=flops)
    eo = 2 if case["out"] == "bf16" else 4
    if case["dir"] == "dw":  # every matrix is written, of an empty group too
        return dict(bytes=rows * (N + K) * e + G * N * K * eo, flops=flops)
    i, o = (K, N) if case["dir"] == "fwd" else (N, K)
    return dict(bytes=_touched(case) * N * K * e + rows * (i * e + o * eo), flops=flops)


# -------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "act":
        a, u = s["gate"].double(), s["up"].double()
        silu = a * torch.sigmoid(a)
        r = torch.ones_like(a[:, :1]) if s["weight"] is None else s["weight"].double().unsqueeze(1)
        if case["dir"] == "fwd":
            return r * silu * u
        dh, p = s["dh"].double(), torch.sigmoid(a)
        out = [r * dh * u * (p + silu * torch.sigmoid(-a)), r * dh * silu]
        return out if s["weight"] is None else out + [torch.einsum("ri,ri->r", dh, silu * u)]
    out = s["out"].double()
    first = s["offsets"].tolist()
    for g, (lo, hi) in enumerate(zip(first, first[1:])):
        if case["op"] == "product" and case["dir"] == "dw":
            out[g] = torch.einsum("rn,rk->nk", s["dy"][lo:hi].double(), s["x"][lo:hi].double())
        if lo == hi or (case["op"] == "product" and case["dir"] == "dw"):
            continue
        if case["op"] == "int4":
            q = s["codes"][g].long()
            w = torch.empty((case["N"], case["K"]), dtype=torch.float64, device=q.device)
            w[:, 0::2], w[:, 1::2] = (q % 16).double(), (q // 16).double()
            col = torch.arange(case["K"], device=q.device) // case["group"]
            w = (w - (8 if s["zeros"] is None else s["zeros"][g].double()[:, col])) * s["scales"][g].double()[:, col]
            out[lo:hi] = s["x"][lo:hi].double() @ w.mT
        elif case["dir"] == "fwd":
            out[lo:hi] = s["x"][lo:hi].double() @ s["w"][g].double().mT
        else:
            out[lo:hi] = s["dy"][lo:hi].double() @ s["w"][g].double()
    return out
