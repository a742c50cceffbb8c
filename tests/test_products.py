"""The experts' products on the GPU: rows times their group's matrix and its
gradients, the activation and its gradient, 4-bit weights."""
import pytest
import torch

import product_ref as R
from sparse_moe_expert_02_gb300 import _lib as L, grouped, int4

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def offsets_of(sizes, before=0):
    at = [before]
    for n in sizes:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def operands(op, rows, N, K, G, dtype, seed=0):
    g = gen(seed)
    if op == "fwd":
        return randn(g, rows, K, dtype=dtype), randn(g, G, N, K, dtype=dtype, std=K ** -0.5)
    if op == "dx":
        return randn(g, rows, N, dtype=dtype), randn(g, G, N, K, dtype=dtype, std=N ** -0.5)
    return randn(g, rows, N, dtype=dtype), randn(g, rows, K, dtype=dtype)


def call(op, a, b, offsets, out, **kw):
    fn = {"fwd": grouped.matmul, "dx": grouped.matmul_dx, "dw": grouped.matmul_dw}[op]
    return fn(a, b, offsets, out=out, **kw)


def out_shape(op, rows, N, K, G):
    return {"fwd": (rows, N), "dx": (rows, K), "dw": (G, N, K)}[op]


def check(op, a, b, offsets, out, **kw):
    """Calls and compares, with rows of no group left as they were."""
    held = out.clone()
    word = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = call(op, a, b, offsets, out, err=word, **kw)
    assert got is out and not word.any()
    groups = R.ranges(None if offsets is None else offsets.tolist(), a.shape[0])
    ref, bound = R.product(op, a, b, groups, held, out.dtype, **kw)
    R.close(got, ref, bound)


SIZES = [  # group sizes, rows before the first and after the last, N, K
    ([1], 0, 0, 16, 8), ([1], 0, 0, 1, 1), ([5], 0, 0, 128, 64), ([3, 0, 1, 0, 17], 2, 3, 72, 136), ([64, 65, 63, 0, 128], 0, 0, 256, 192),
    ([0, 0, 0], 4, 1, 24, 40), ([130, 7, 259], 1, 0, 264, 328), ([33] * 40, 0, 5, 136, 72), ([300, 1], 0, 2, 127, 65), ([31, 2, 90], 1, 1, 129, 257),
    ([513], 0, 0, 8, 1000), ([16, 48, 112, 240], 0, 0, 384, 520), ([700, 20], 0, 0, 64, 24), ([2, 1, 1], 0, 0, 1000, 2048),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_product(op, dtype, case):
    sizes, before, after, N, K = SIZES[case]
    rows, G = before + sum(sizes) + after, len(sizes)
    a, b = operands(op, rows, N, K, G, DT[dtype], case)
    for out_dtype in DT.values():
        out = randn(gen(99), *out_shape(op, rows, N, K, G), dtype=out_dtype)
        check(op, a, b, offsets_of(sizes, before), out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("rows,N,K", [(1, 128, 4096), (7, 2048, 1024), (257, 64, 4096), (300, 1025, 63), (1, 4096, 31), (2048, 96, 80)])
def test_product_of_one_group(op, dtype, rows, N, K):
    a, b = operands(op, rows, N, K, 1, DT[dtype], rows)
    b1 = b if op == "dw" else b[0]
    check(op, a, b, None, randn(gen(1), *out_shape(op, rows, N, K, 1), dtype=DT[dtype]))
    got = call(op, a, b1, None, None)
    ref = call(op, a, b, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), None)
    assert got.dtype == DT[dtype] and torch.equal(got, ref.view(got.shape))
    assert got.dim() == 2


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("N,K,G,rows", [(640, 1024, 16, 1999), (1024, 640, 3, 3001), (255, 1031, 9, 1500)])
def test_product_large(op, N, K, G, rows):
    """Many tiles a block, ragged groups, one of them most of the rows."""
    sizes = [rows // (3 * G)] * G
    sizes[G // 2] = rows - sum(sizes) + sizes[0] - 3
    sizes[1] = 0
    sizes[0] += 1
    total = sum(sizes)
    a, b = operands(op, total + 9, N, K, G, torch.bfloat16)
    for out_dtype in DT.values():
        check(op, a, b, offsets_of(sizes, 4), randn(gen(5), *out_shape(op, total + 9, N, K, G), dtype=out_dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["fwd", "dx"])
@pytest.mark.parametrize("left,right", [(0, 8), (8, 8), (3, 4), (1, 0), (5, 64)])
def test_product_of_strided_rows(op, dtype, left, right):
    sizes, N, K = [9, 0, 70], 96, 160
    rows = sum(sizes)
    a, b = operands(op, rows, N, K, 3, DT[dtype])
    wide = randn(gen(3), rows, left + a.shape[1] + right, dtype=DT[dtype])
    wide[:, left:left + a.shape[1]] = a
    shape = out_shape(op, rows, N, K, 3)
    buf = randn(gen(4), rows, left + shape[1] + right, dtype=DT[dtype])
    edges = buf.clone()
    check(op, wide[:, left:left + a.shape[1]], b, offsets_of(sizes), buf[:, left:left + shape[1]])
    assert torch.equal(buf[:, :left], edges[:, :left]) and torch.equal(buf[:, left + shape[1]:], edges[:, left + shape[1]:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("left,right", [(0, 8), (8, 16), (3, 4), (1, 0)])
def test_weight_gradient_of_strided_rows(dtype, left, right):
    sizes, N, K = [9, 0, 70, 200], 96, 160
    rows = sum(sizes)
    a, b = operands("dw", rows, N, K, 4, DT[dtype])
    wa, wb = (randn(gen(i), rows, left + t.shape[1] + right, dtype=DT[dtype]) for i, t in ((6, a), (7, b)))
    wa[:, left:left + N], wb[:, left:left + K] = a, b
    check("dw", wa[:, left:left + N], wb[:, left:left + K], offsets_of(sizes), randn(gen(8), 4, N, K, dtype=DT[dtype]))


def test_weights_at_an_odd_address():
    sizes, N, K = [9, 30], 96, 160
    for op in ("fwd", "dx"):
        a, b = operands(op, 39, N, K, 2, torch.bfloat16)
        flat = torch.empty(b.numel() + 5, dtype=b.dtype, device="cuda")
        w = flat[5:].view_as(b)
        w.copy_(b)
        check(op, a, w, offsets_of(sizes), randn(gen(1), *out_shape(op, 39, N, K, 2)))
    a, b = operands("dw", 39, N, K, 2, torch.bfloat16)
    flat = torch.zeros(2 * N * K + 3, device="cuda")
    check("dw", a, b, offsets_of(sizes), flat[3:].view(2, N, K))
    assert not flat[:3].any()


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nothing_leaks_from_other_rows_groups_or_columns(op, dtype, bad):
    """Infinities and NaN in rows of no group, in an empty group's matrix and in the columns beside a strided view."""
    sizes, before, N, K = [20, 0, 37, 1], 3, 104, 72
    rows = before + sum(sizes) + 6
    a, b = operands(op, rows, N, K, 4, DT[dtype])
    wide = torch.full((rows, a.shape[1] + 8), bad, dtype=DT[dtype], device="cuda")
    wide[before:rows - 6, :a.shape[1]] = a[before:rows - 6]
    a = wide[:, :a.shape[1]]
    if op == "dw":
        b[:before] = bad
        b[rows - 6:] = bad
    else:
        b[1] = bad
    out = torch.zeros(out_shape(op, rows, N, K, 4), device="cuda")
    call(op, a, b, offsets_of(sizes, before), out)
    assert torch.isfinite(out).all()
    check(op, a, b, offsets_of(sizes, before), out)


@pytest.mark.parametrize("op", ["fwd", "dx"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_bad_row_spoils_itself_alone(op, dtype):
    sizes, N, K = [20, 37], 104, 72
    a, b = operands(op, 57, N, K, 2, DT[dtype])
    out = call(op, a, b, offsets_of(sizes), None)
    a[20, 5] = float("nan")
    a[40, 7] = float("inf")
    bad = call(op, a, b, offsets_of(sizes), None)
    keep = [r for r in range(57) if r not in (20, 40)]
    assert torch.isnan(bad[20]).all() and not torch.isfinite(bad[40]).any()
    assert torch.equal(bad[keep], out[keep])


def test_a_bad_row_spoils_its_own_groups_gradient_alone():
    sizes = [20, 37, 12]
    for dtype in DT.values():
        a, b = operands("dw", 69, 40, 24, 3, dtype)
        a[25, 3] = float("inf")
        got = call("dw", a, b, offsets_of(sizes), None)
        assert torch.isfinite(got[[0, 2]]).all() and not torch.isfinite(got[1, 3]).any() and torch.isfinite(got[1, 4:]).all()


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
def test_offsets_outside_the_rows_are_cut(op):
    a, b = operands(op, 50, 48, 56, 4, torch.bfloat16)
    for at in ([-7, 10, 10, 48, 2000], [0, 0, 0, 0, 0], [50, 60, 70, 80, 90], [5, 5, 50, 51, 2 ** 31 - 1]):
        check(op, a, b, torch.tensor(at, dtype=torch.int32, device="cuda"), randn(gen(1), *out_shape(op, 50, 48, 56, 4)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(96, 160), (65, 33)])
def test_weight_gradient_accumulates(dtype, out_dtype, N, K):
    sizes = [70, 0, 3, 129]
    a, b = operands("dw", 202, N, K, 4, DT[dtype])
    out = randn(gen(2), 4, N, K, dtype=DT[out_dtype], std=20.0)
    empty = out[1].clone()
    check("dw", a, b, offsets_of(sizes), out, accumulate=True)
    assert torch.equal(out[1], empty)


def test_no_rows():
    for dtype in DT.values():
        x, w = torch.empty((0, 24), dtype=dtype, device="cuda"), torch.ones((2, 16, 24), dtype=dtype, device="cuda")
        at = torch.zeros(3, dtype=torch.int32, device="cuda")
        assert grouped.matmul(x, w, at).shape == (0, 16) and grouped.matmul_dx(x[:, :16], w, at).shape == (0, 24)
        dw = grouped.matmul_dw(x[:, :16].contiguous(), x, at, out=w.clone())
        assert dw.shape == (2, 16, 24) and not dw.any()
        assert torch.equal(grouped.matmul_dw(x[:, :16].contiguous(), x, at, out=w.clone(), accumulate=True), w)


def test_rows_far_apart():
    """Row strides whose offsets pass 32 bits."""
    stride, N, K = (1 << 29) + 8, 40, 48
    buf = torch.empty(5 * stride, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((5, K), (stride, 1))
    out = buf.as_strided((5, N), (stride, 1), 4096)
    x.copy_(randn(gen(1), 5, K))
    w = randn(gen(2), 2, N, K, dtype=torch.bfloat16)
    check("fwd", x, w, offsets_of([2, 3]), out)
    check("dx", out, w, offsets_of([2, 3]), torch.zeros((5, K), device="cuda"))
    check("dw", out, x, offsets_of([2, 3]), torch.zeros((2, N, K), device="cuda"))
    odd = buf.as_strided((5, K), (stride - 1, 1), 3)
    odd.copy_(randn(gen(3), 5, K))
    check("fwd", odd, w, offsets_of([2, 3]), torch.zeros((5, N), device="cuda"))


def test_weights_past_32_bits():
    """The last matrices lie beyond 2^32 bytes and 2^31 elements."""
    G, N, K = 520, 2048, 2048
    w = torch.empty((G, N, K), dtype=torch.bfloat16, device="cuda")
    w[:2] = randn(gen(1), 2, N, K)
    w[-1:] = randn(gen(2), 1, N, K)
    x = randn(gen(3), 12, K, dtype=torch.bfloat16)
    at = torch.full((G + 1,), 7, dtype=torch.int32, device="cuda")
    at[0], at[1], at[-1] = 0, 5, 12
    rows = [(0, 5, 0), (5, 7, 1), (7, 12, G - 1)]
    for op, out in (("fwd", grouped.matmul(x, w, at)), ("dx", grouped.matmul_dx(x, w, at))):
        for lo, hi, g in rows:
            ref, bound = R.product(op, x[lo:hi], w[g:g + 1], [(0, hi - lo)], torch.zeros((hi - lo, 2048), device="cuda"), torch.bfloat16)
            R.close(out[lo:hi], ref, bound)
    dw = grouped.matmul_dw(x, x, at, out=w)
    for lo, hi, g in rows:
        ref, bound = R.product("dw", x[lo:hi], x[lo:hi], [(0, hi - lo)], torch.zeros((1, N, K), device="cuda"), torch.bfloat16)
        R.close(dw[g:g + 1], ref, bound)
    assert not dw[2:G - 1].any()


def test_products_are_the_same_every_time():
    for dtype in DT.values():
        for op in ("fwd", "dx", "dw"):
            a, b = operands(op, 517, 200, 264, 5, dtype)
            at = offsets_of([100, 0, 300, 16, 101])
            first = call(op, a, b, at, None)
            for _ in range(3):
                assert torch.equal(call(op, a, b, at, None), first)


# ------------------------------------------------------------- activation

ACT = [(1, 1), (1, 8), (3, 33), (80, 1024), (17, 4096), (2500, 72), (1300, 513), (5, 10000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("rows,I", ACT)
def test_swiglu(dtype, halves, rows, I):
    both = randn(gen(rows), rows, 2 * I, dtype=DT[dtype], std=3.0)
    gate, up = (both[:, :I], both[:, I:]) if halves else (both[:, :I].contiguous(), both[:, I:].contiguous())
    weight = torch.rand(rows, generator=gen(1), device="cuda")
    for w in (None, weight):
        for out_dtype in DT.values():
            R.close(grouped.swiglu(gate, up, w, out_dtype=out_dtype), *R.swiglu(gate, up, w, out_dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("rows,I", ACT)
def test_swiglu_grad(dtype, halves, rows, I):
    both = randn(gen(rows), rows, 2 * I, dtype=DT[dtype], std=3.0)
    gate, up = (both[:, :I], both[:, I:]) if halves else (both[:, :I].contiguous(), both[:, I:].contiguous())
    dh = randn(gen(2), rows, I, dtype=DT[dtype])
    weight = torch.rand(rows, generator=gen(1), device="cuda")
    for w in (None, weight):
        dg, du, dw = grouped.swiglu_grad(dh, gate, up, w)
        refs = R.swiglu_grad(dh, gate, up, w)
        R.close(dg, *refs[0])
        R.close(du, *refs[1])
        assert (dw is None) == (w is None)
        if w is not None:
            R.close(dw, *refs[2])
    only = grouped.swiglu_grad(dh, gate, up, None, dweight=torch.empty(rows, device="cuda"))[2]
    R.close(only, *R.swiglu_grad(dh, gate, up, None)[2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swiglu_grad_is_the_difference_of_swiglu(dtype):
    """Central differences of the 64-bit definition, so that formula and code do not share a slip."""
    rows, I, h = 6, 40, 1e-5
    gate, up, dh = (randn(gen(i), rows, I, dtype=DT[dtype]) for i in range(3))
    weight = torch.rand(rows, generator=gen(4), device="cuda")
    loss = lambda g, u, w: (R.swiglu(g, u, w, torch.float32)[0] * dh.double())
    g, u, w = gate.double(), up.double(), weight.double()
    dg, du, dw = grouped.swiglu_grad(dh, gate, up, weight)
    # differences are off by h^2 of the third derivative, below 1e-9 here, and 1e-11 of rounding
    tol = 1e-8 + 4 * R.half_step(DT[dtype]) + 2.0 ** -18
    assert ((loss(g + h, u, w) - loss(g - h, u, w)) / (2 * h) - dg.double()).abs().max() <= tol * (dh * up).abs().max()
    assert ((loss(g, u + h, w) - loss(g, u - h, w)) / (2 * h) - du.double()).abs().max() <= tol * (dh * gate).abs().max()
    assert ((loss(g, u, w + h) - loss(g, u, w - h)).sum(1) / (2 * h) - dw.double()).abs().max() <= tol * (dh * gate * up).abs().sum(1).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_swiglu_in_place(dtype):
    both = randn(gen(0), 300, 2 * 136, dtype=DT[dtype], std=2.0)
    w = torch.rand(300, generator=gen(1), device="cuda")
    dh = randn(gen(2), 300, 136, dtype=DT[dtype])
    gate, up = both[:, :136], both[:, 136:]
    h, (dg, du, dw) = grouped.swiglu(gate, up, w), grouped.swiglu_grad(dh, gate, up, w)
    copy = both.clone()
    a, b = copy[:, :136], copy[:, 136:]
    got = grouped.swiglu_grad(dh, a, b, w, dgate=a, dup=b)
    assert torch.equal(got[0], dg) and torch.equal(got[1], du) and torch.equal(got[2], dw) and torch.equal(copy, torch.cat([dg, du], 1))
    copy = both.clone()
    assert torch.equal(grouped.swiglu(copy[:, :136], copy[:, 136:], w, out=copy[:, 136:]), h) and torch.equal(copy[:, :136], gate)


def test_swiglu_at_the_ends_of_the_range():
    g = torch.tensor([[-200.0, -89.0, -87.0, -30.0, 0.0, 30.0, 88.0, 200.0, 3e38]], device="cuda")
    for dtype in DT.values():
        gate = g.to(dtype)
        up = torch.full_like(gate, 0.5)
        got = grouped.swiglu(gate, up)
        assert torch.isfinite(got).all()
        R.close(got, *R.swiglu(gate, up, None, dtype))
        dg, du, dw = grouped.swiglu_grad(up, gate, up, torch.ones(1, device="cuda"))
        assert torch.isfinite(dg).all() and torch.isfinite(du).all()
        R.close(dg[:, :8], *(t[:, :8] for t in R.swiglu_grad(up, gate, up, None)[0]))
    bad = torch.ones((3, 40), device="cuda")
    bad[1, 3] = float("nan")
    got = grouped.swiglu(bad, torch.ones_like(bad))
    assert int(torch.isnan(got).sum()) == 1
    dg, du, dw = grouped.swiglu_grad(torch.ones_like(bad), bad, torch.ones_like(bad), torch.ones(3, device="cuda"))
    assert int(torch.isnan(dg).sum()) == 1 and torch.isnan(dw).tolist() == [False, True, False]


def test_activation_of_no_rows():
    e = torch.empty((0, 16), device="cuda")
    assert grouped.swiglu(e, e).shape == (0, 16)
    assert grouped.swiglu_grad(e, e, e, torch.empty(0, device="cuda"))[2].shape == (0,)


# ----------------------------------------------------------------- 4 bits

def weights4(G, N, K, group, zeros, scale, seed=0):
    nb = -(-K // group)
    g = gen(seed)
    codes = torch.randint(0, 256, (G, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((0.5 + torch.rand((G, N, nb), generator=g, device="cuda")) * K ** -0.5).to(DT[scale])
    z = torch.randint(0, 16, (G, N, nb), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return int4.I4Tensor(codes, scales, z, K, group)


def check4(x, w, offsets, out):
    held = out.clone()
    word = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = int4.matmul(x, w, offsets, out=out, err=word)
    assert got is out and not word.any()
    groups = R.ranges(None if offsets is None else offsets.tolist(), x.shape[0])
    G = w.codes.shape[0]
    v = torch.stack([R.int4_values(w.codes[g], w.scales[g], None if w.zeros is None else w.zeros[g], w.group) for g in range(G)])
    ref, bound = R.product("fwd", x, v, groups, held, out.dtype)
    # K products and, group by group, a scale each: K / 32 more roundings at most, which n 2^-23 has room for beside
    # sums that round to nearest; bf16 rows, many of them: the values of the weights rounded to bf16
    if x.dtype == torch.bfloat16 and x.shape[0] > 16:
        for g, (lo, hi) in enumerate(groups):
            bound[lo:hi] += R.half_step(torch.bfloat16) * (1 + 2.0 ** -7) * (x[lo:hi].double().abs() @ v[g].abs().mT)
    R.close(got, ref, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group,zeros,scale", [(128, False, "bf16"), (64, True, "bf16"), (32, True, "f32"), (128, True, "f32"), (32, False, "bf16")])
@pytest.mark.parametrize("sizes,before,after,N,K", [
    ([1], 0, 0, 16, 32), ([1], 0, 0, 1, 64), ([7], 0, 0, 200, 288), ([3, 0, 1, 8, 9], 1, 2, 64, 160), ([16], 0, 0, 33, 4096),
    ([17, 40, 0, 130], 0, 3, 72, 416), ([300], 0, 0, 130, 96), ([1] * 30, 0, 0, 24, 1024), ([2, 5], 0, 0, 520, 2080)])
def test_int4_matmul(dtype, group, zeros, scale, sizes, before, after, N, K):
    rows = before + sum(sizes) + after
    w = weights4(len(sizes), N, K, group, zeros, scale)
    x = randn(gen(1), rows, K, dtype=DT[dtype])
    for out_dtype in DT.values():
        check4(x, w, offsets_of(sizes, before), randn(gen(2), rows, N, dtype=out_dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 8, 9, 16, 17, 33, 64, 65, 256, 700])
def test_int4_matmul_of_one_matrix(dtype, rows):
    w = weights4(1, 648, 1184, 128, False, "bf16")
    x = randn(gen(rows), rows, 1184, dtype=DT[dtype])
    check4(x, w, None, randn(gen(2), rows, 648, dtype=DT[dtype]))
    one = int4.I4Tensor(w.codes[0], w.scales[0], None, w.cols, w.group)
    assert torch.equal(int4.matmul(x, one), int4.matmul(x, w))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [5, 40, 300])
@pytest.mark.parametrize("left,right", [(0, 8), (3, 4), (1, 0)])
def test_int4_matmul_of_strided_rows(dtype, rows, left, right):
    w = weights4(1, 56, 224, 64, True, "bf16")
    wide = torch.full((rows, left + 224 + right), float("nan"), dtype=DT[dtype], device="cuda")
    wide[:, left:left + 224] = randn(gen(1), rows, 224)
    buf = randn(gen(2), rows, left + 56 + right, dtype=DT[dtype])
    edges = buf.clone()
    check4(wide[:, left:left + 224], w, None, buf[:, left:left + 56])
    assert torch.equal(buf[:, :left], edges[:, :left]) and torch.equal(buf[:, left + 56:], edges[:, left + 56:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", [[3, 0, 5, 1], [30, 0, 50, 40]])
def test_int4_nothing_leaks(dtype, sizes):
    w = weights4(4, 40, 96, 32, True, "f32")
    w.scales[1] = float("nan")
    rows = 2 + sum(sizes) + 3
    x = torch.full((rows, 96), float("inf"), dtype=DT[dtype], device="cuda")
    x[2:rows - 3] = randn(gen(1), rows - 5, 96)
    out = torch.zeros((rows, 40), device="cuda")
    check4(x, w, offsets_of(sizes, 2), out)
    assert torch.isfinite(out).all()
    clean = out.clone()
    x[2, 9] = float("nan")
    int4.matmul(x, w, offsets_of(sizes, 2), out=out)
    assert torch.isnan(out[2]).all() and torch.equal(out[3:], clean[3:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("inf"), -3.3e38, 3e-39])
def test_int4_rows_at_the_ends_of_the_range(dtype, value):
    """An infinity, numbers next to the largest and subnormal ones come out as the products say."""
    w = weights4(1, 16, 64, 64, False, "f32")
    w.scales.fill_(0.25)
    x = torch.zeros((2, 64), dtype=DT[dtype], device="cuda")
    x[0, 5] = value
    x[1, 6] = 1.0
    got = int4.matmul(x, w, out_dtype=torch.float32).double()
    v = R.int4_values(w.codes[0], w.scales[0], None, 64)
    want = x[0, 5].double() * v[:, 5]
    big = want.abs() > torch.finfo(torch.float32).max
    want = torch.where(big & torch.isfinite(want), want.sign() * float("inf"), want)
    assert torch.allclose(got[0], want, rtol=2.0 ** -22, atol=0, equal_nan=True) and torch.equal(got[1], v[:, 6])


def test_int4_weights_past_32_bits():
    G, N, K = 1024, 2048, 4096  # 4 GB of codes
    w = int4.empty((G, N), K, 128)
    few = weights4(3, N, K, 128, False, "bf16")
    for i, g in enumerate((0, 700, G - 1)):
        w.codes[g], w.scales[g] = few.codes[i], few.scales[i]
    x = randn(gen(1), 21, K, dtype=torch.bfloat16)
    at = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    at[1:] = 4
    at[701:] = 9
    at[G] = 21
    got, ref = int4.matmul(x, w, at), int4.matmul(x, few, offsets_of([4, 5, 12]))
    assert torch.equal(got, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_int4_quantize(dtype, scale, group, zeros):
    x = randn(gen(0), 37, 288, dtype=DT[dtype]) * torch.exp(2 * randn(gen(1), 37, 1)).to(DT[dtype])
    x[0, :128] = 0
    x[1, 40] = float("nan")
    x[2, 140] = float("-inf")
    x[3] = x[3].abs() + 1
    x[4] = -x[3]
    x[5] = torch.arange(288, device="cuda") % 31 - 15  # ties
    x[6] = 1e-44
    x[7] = x[7] * 1e-39
    x[8] = x[8].sign() * 3.3e38
    wide = torch.empty((37, 300), dtype=DT[dtype], device="cuda")
    wide[:, 7:295] = x
    q = int4.quantize(wide[:, 7:295], group, zeros, DT[scale])
    codes, scales, z = R.int4_quantize(x, group, zeros, DT[scale])
    assert torch.equal(torch.nan_to_num(q.scales.cpu(), nan=-1), torch.nan_to_num(scales, nan=-1))
    assert torch.equal(q.codes.cpu(), codes) and (not zeros or torch.equal(q.zeros.cpu(), z))
    v = R.int4_values(q.codes, q.scales, q.zeros, group).cpu()
    for out_dtype in DT.values():
        back = int4.dequantize(q, out_dtype)
        R.close(back, v, R.half_step(out_dtype) * torch.nan_to_num(v.abs()) + 1e-45 + (1e-40 if out_dtype == torch.bfloat16 else 0))
        buf = torch.zeros((37, 291), dtype=out_dtype, device="cuda")
        int4.dequantize(q, out=buf[:, 3:])
        assert torch.equal(torch.nan_to_num(buf[:, 3:]), torch.nan_to_num(back)) and not buf[:, :3].any()


def test_int4_quantized_weights_by_group():
    w = randn(gen(0), 3, 40, 160)
    q = int4.quantize(w, 64)
    assert q.shape == (3, 40, 160) and int4.dequantize(q).shape == (3, 40, 160)
    x = randn(gen(1), 9, 160)
    check4(x, q, offsets_of([2, 0, 7]), torch.zeros((9, 40), device="cuda"))
    e = int4.quantize(torch.empty((0, 64), device="cuda"))
    assert int4.dequantize(e).shape == (0, 64) and int4.matmul(torch.empty((0, 160), device="cuda"), q, offsets_of([0, 0, 0])).shape == (0, 40)


# ------------------------------------------------------- used as they would be

def test_experts_trained_on_the_layers_permutation():
    """A step of the experts' feed-forward over routed rows: forward with the routing weights in the activation, every
    gradient, two micro-batches added up; in fp32, against the 64-bit step."""
    T, D, E, I, k = 70, 96, 6, 64, 3
    g = gen(0)
    wg, wu, wd = (randn(g, *s, std=s[2] ** -0.5) for s in ((E, I, D), (E, I, D), (E, D, I)))
    dwg, dwu, dwd = (torch.zeros_like(w) for w in (wg, wu, wd))
    exact = [torch.zeros_like(w, dtype=torch.float64) for w in (wg, wu, wd)]
    for batch in range(2):
        x, dout = randn(g, T, D), randn(g, T, D)
        idx = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(batch * T + t))[:k] for t in range(T)]).int().cuda()
        p = torch.rand((T, k), generator=g, device="cuda")
        counts, offsets, tiles = (torch.empty(E + n, dtype=torch.int32, device="cuda") for n in (1, 2, 2))
        inv, src = torch.empty(T * k, dtype=torch.int32, device="cuda"), torch.empty(T * k + T, dtype=torch.int32, device="cuda")
        assert L.moe_permute_index_noalloc(idx, T, E, k, counts, offsets, tiles, inv, src) == 0
        at, tok = offsets[:E + 1], src[:T * k].long()
        w = torch.empty(T * k, device="cuda")
        w[inv.long()] = p.flatten()
        xp = x[tok]
        gu = torch.empty((T * k, 2 * I), device="cuda")
        gate, up = grouped.matmul(xp, wg, at, out=gu[:, :I]), grouped.matmul(xp, wu, at, out=gu[:, I:])
        h = grouped.swiglu(gate, up, w)
        out = torch.zeros((T, D), device="cuda").index_add_(0, tok, grouped.matmul(h, wd, at))
        dy = dout[tok]
        grouped.matmul_dw(dy, h, at, out=dwd, accumulate=True)
        dh = grouped.matmul_dx(dy, wd, at)
        dgate, dup, dw = grouped.swiglu_grad(dh, gate, up, w)
        grouped.matmul_dw(dgate, xp, at, out=dwg, accumulate=True)
        grouped.matmul_dw(dup, xp, at, out=dwu, accumulate=True)
        dx = torch.zeros((T, D), device="cuda").index_add_(0, tok, grouped.matmul_dx(dgate, wg, at) + grouped.matmul_dx(dup, wu, at))
        # the same in 64 bits, pair by pair, by autograd
        leaves = [t.double().requires_grad_() for t in (x, wg, wu, wd, p)]
        X, G, U, W, P = leaves
        a, u = torch.einsum("td,tkid->tki", X, G[idx.long()]), torch.einsum("td,tkid->tki", X, U[idx.long()])
        ref = torch.einsum("tki,tkdi,tk->td", a * torch.sigmoid(a) * u, W[idx.long()], P)
        grads = torch.autograd.grad(ref, leaves, dout.double())
        for i in range(3):
            exact[i] += grads[i + 1]
        # three products and an activation of 32 bits: the sums' terms stay below a few units
        for got, want in ((out, ref), (dx, grads[0]), (dw[inv.long()].view(T, k), grads[4])):
            assert (got.double() - want).abs().max() <= 1e-5 * want.abs().max()
    for got, want in zip((dwg, dwu, dwd), exact):
        assert (got.double() - want).abs().max() <= 1e-5 * want.abs().max()


def test_experts_served_from_four_bits():
    """A few tokens' experts from 4-bit weights, captured once and replayed for other tokens and another routing."""
    D, E, I, rows = 256, 8, 128, 24
    up4, gate4, down4 = (int4.quantize(randn(gen(i), *s, std=s[2] ** -0.5), 64, zeros=i == 1) for i, s in
                         enumerate(((E, I, D), (E, I, D), (E, D, I))))
    x, p = torch.zeros((rows, D), dtype=torch.bfloat16, device="cuda"), torch.zeros(rows, device="cuda")
    at = torch.zeros(E + 1, dtype=torch.int32, device="cuda")

    def step():
        gate, up = int4.matmul(x, gate4, at, out_dtype=torch.float32), int4.matmul(x, up4, at, out_dtype=torch.float32)
        return int4.matmul(grouped.swiglu(gate, up, p, out_dtype=torch.bfloat16), down4, at)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for i, sizes in enumerate(([3, 3, 3, 3, 3, 3, 3, 3], [0, 20, 0, 4, 0, 0, 0, 0], [1, 0, 0, 0, 0, 0, 0, 23])):
        x.copy_(randn(gen(10 + i), rows, D))
        p.copy_(torch.rand(rows, generator=gen(20 + i), device="cuda"))
        at.copy_(offsets_of(sizes))
        graph.replay()
        assert torch.equal(y, step())
        value = lambda q: torch.stack([R.int4_values(q.codes[g], q.scales[g], None if q.zeros is None else q.zeros[g], q.group) for g in range(E)])
        G, U, W = value(gate4), value(up4), value(down4)
        e = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(sizes, device="cuda"))
        a, u = torch.einsum("rd,rid->ri", x.double(), G[e]), torch.einsum("rd,rid->ri", x.double(), U[e])
        ref = torch.einsum("ri,rdi->rd", p.double()[:, None] * a * torch.sigmoid(a) * u, W[e])
        # h, out and (in groups of many rows) the weights rounded to bf16 once each
        assert (y.double() - ref).abs().max() <= 4 * R.half_step(torch.bfloat16) * ref.abs().max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_products_on_two_streams_and_in_a_graph(dtype):
    """Calls in flight at the same time share nothing; a captured step follows its offsets."""
    N, K, G, rows = 136, 264, 4, 333
    ops = {op: operands(op, rows, N, K, G, DT[dtype]) for op in ("fwd", "dx", "dw")}
    at = offsets_of([100, 33, 0, 200])
    want = {op: call(op, *ab, at, None) for op, ab in ops.items()}
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, (op, ab) in zip(streams, ops.items()):
            with torch.cuda.stream(s):
                got.append((op, call(op, *ab, at, None)))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[op]) for op, t in got)
    outs = {op: torch.zeros_like(want[op]) for op in ops}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for op, ab in ops.items():
            call(op, *ab, at, outs[op])
    for sizes in ([100, 33, 0, 200], [0, 0, 1, 2], [333, 0, 0, 0]):
        at.copy_(offsets_of(sizes))
        for t in outs.values():
            t.zero_()
        graph.replay()
        for op, ab in ops.items():
            assert torch.equal(outs[op], call(op, *ab, at, torch.zeros_like(outs[op])))
