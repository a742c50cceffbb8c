"""The operators of the block -- norms, microscaled 4-bit quantisation and
product, the layer for a few tokens, MoEBlock -- against 64-bit definitions.

Tolerances: fp32 arithmetic over n terms is allowed n * 2^-22 of the sum of
the terms' magnitudes (any order of summation, products in any order), a store
to bf16 2^-8 of the value (half an ulp is 2^-9).  Codes and scales must match
bit for bit.  The layer is held to the bounds its types are specified with.
"""
import numpy as np
import pytest
import torch

import block_ref as R
import oracle
from parity_util import experts_for_tokens, rel_max_err
from sparse_moe_expert_02_gb300 import MoEBlock, MoELayer, mx, norm, synth
from sparse_moe_expert_02_gb300 import _lib as L

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
ULP = {F32: 2.0 ** -23, BF16: 2.0 ** -8}


def rand(*shape, seed=0, dtype=F32, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


# ------------------------------------------------------------------- norms

def norm_tol(v, kind, eps, w, w_offset, ref, dtype):
    """Error allowed for N(v): the mean's and the variance's fp32 sums, then three products."""
    n = v.shape[-1]
    spread = np.abs(v).max(-1, keepdims=True)
    rstd = 1 / np.sqrt((v - (v.mean(-1, keepdims=True) if kind == "layer" else 0)).__pow__(2).mean(-1, keepdims=True) + eps)
    gain = np.abs(1.0 if w is None else w + w_offset)
    steps = np.log2(max(n, 2)) + 16  # a thread's 16 elements, then a tree
    return steps * 2.0 ** -23 * (np.abs(ref) + spread * rstd * gain) + ULP[dtype] * np.abs(ref) + 1e-30


def check_norm(got, v, kind, eps, w, b, w_offset):
    ref = R.norm(v, kind, eps, w, b, w_offset)
    tol = norm_tol(v, kind, eps, w, w_offset, ref, got.dtype) + (0 if b is None else 2.0 ** -22 * np.abs(b))
    assert (np.abs(f64(got) - ref) <= tol).all(), np.abs(f64(got) - ref).max()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("xt,ot", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (5, 33), (2, 512), (4, 520), (9, 1000), (7, 4096), (3, 4104), (2, 16384),
                                 (2, 16383)])
def test_norm_pre(kind, xt, ot, T, D):
    x, w, b = rand(T, D, seed=1, dtype=xt, std=3) + 1, rand(D, seed=2, dtype=xt), rand(D, seed=3, dtype=xt)
    out = torch.empty(T, D, dtype=ot, device="cuda")
    norm.pre(x, w, b, kind=kind, eps=1e-5, w_offset=1.0, out=out)
    check_norm(out, f64(x), kind, 1e-5, f64(w), f64(b), 1.0)
    norm.pre(x, kind=kind, eps=1e-5, out=out)
    check_norm(out, f64(x), kind, 1e-5, None, None, 0.0)


@pytest.mark.parametrize("gate_by", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("kind,next_kind", [("rms", "rms"), ("layer", "none"), ("none", "layer"), ("rms", None)])
@pytest.mark.parametrize("T,D,yt,rt,nt", [(5, 77, F32, F32, F32), (6, 264, BF16, BF16, BF16), (33, 2048, BF16, F32, BF16),
                                          (3, 4097, F32, BF16, F32)])
def test_norm_post(gate_by, sigmoid, kind, next_kind, T, D, yt, rt, nt):
    y, r = rand(T, D, seed=1, dtype=yt, std=2), rand(T, D, seed=2, dtype=rt)
    w, nw = rand(D, seed=3, dtype=yt), rand(D, seed=4)
    gate = {"none": None, "channel": rand(D, seed=5, dtype=yt), "token": rand(T, seed=5, dtype=yt),
            "full": rand(T, D, seed=5, dtype=yt)}[gate_by]
    nxt = torch.empty(T, D, dtype=nt, device="cuda") if next_kind else None
    out, n = norm.post(y, r, w, kind=kind, eps=1e-6, gate=gate, gate_by=gate_by, gate_sigmoid=sigmoid, res_scale=0.5,
                       branch_scale=-1.5, next_w=nw if next_kind else None, next_norm=next_kind is not None,
                       next_kind=next_kind, next_out=nxt)
    assert (n is None) == (next_kind in (None, "none"))  # "none": no next norm
    g = 1.0
    if gate is not None:
        g = f64(gate)
        g = 1 / (1 + np.exp(-g)) if sigmoid else g
        g = g[:, None] if gate_by == "token" else g
    wn = None if kind == "none" else f64(w)
    branch = R.norm(f64(y), kind, 1e-6, wn)
    ref = 0.5 * f64(r) - 1.5 * g * branch
    tol = 1.5 * np.abs(g) * (norm_tol(f64(y), kind, 1e-6, wn, 0.0, branch, F32) + 2.0 ** -20 * np.abs(branch))
    tol = tol + 2.0 ** -22 * np.abs(f64(r)) + ULP[rt] * np.abs(ref)
    assert (np.abs(f64(out) - ref) <= tol).all()
    if n is not None:
        check_norm(n, f64(out), next_kind, 1e-6, None if next_kind == "none" else f64(nw), None, 0.0)


def test_norm_strided_rows_in_place_and_other_stream():
    T, D = 37, 640
    big_y, big_r = rand(T, 3 * D, seed=1, dtype=BF16), rand(T, 2 * D + 8, seed=2)
    y, r = big_y[:, D:2 * D], big_r[:, 8:8 + D]
    keep, keep_y = big_r.clone(), big_y.clone()
    w = rand(D, seed=3, dtype=BF16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, _ = norm.post(y, r, w, out=r)
    s.synchronize()
    assert out.data_ptr() == r.data_ptr()
    fresh, _ = norm.post(y, keep[:, 8:8 + D], w)
    assert torch.equal(fresh, r)
    assert torch.equal(big_y, keep_y)
    keep[:, 8:8 + D] = fresh
    assert torch.equal(big_r, keep)  # nothing outside the view
    # rows at an odd offset (2-byte alignment): the same values by the unaligned path
    a = norm.pre(big_y[:, 1:1 + D], w)
    assert torch.equal(a, norm.pre(big_y[:, 1:1 + D].contiguous(), w))


def test_norm_rows_do_not_mix_and_extremes_follow_the_formula():
    x = rand(6, 96, seed=1)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 3.0
    out = f64(norm.pre(x, eps=1e-6))
    assert (out[1] == 0).all() and np.isnan(out[2]).all()
    assert np.isnan(out[3, 7]) and (np.delete(out[3], 7) == 0).all()
    assert np.isfinite(out[[0, 4, 5]]).all()
    ln = f64(norm.pre(x, kind="layer", eps=1e-6))
    assert (ln[4] == 0).all() and (ln[1] == 0).all()
    assert norm.pre(x[:0]).shape == (0, 96)


def test_norm_refusals():
    x = rand(2, 64)
    for bad in (lambda: norm.pre(x.half()), lambda: norm.pre(x, kind="batch"), lambda: norm.pre(x, rand(63)),
                lambda: norm.pre(x.t()), lambda: norm.pre(x, out=rand(2, 63)), lambda: norm.pre(x.cpu()),
                lambda: norm.pre(x, rand(64), rand(64, dtype=BF16)), lambda: norm.post(x, x, gate=rand(3), gate_by="token"),
                lambda: norm.post(x, x, gate=rand(64), gate_by="row"), lambda: norm.post(x, rand(2, 65))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: norm.pre(x, eps=-1.0), lambda: norm.pre(x, eps=float("nan")), lambda: norm.pre(rand(1, 16385))):
        with pytest.raises(L.MoEError):
            bad()


# ---------------------------------------------------- microscaled 4 bits

def special_rows(cols):
    """Rows at the format's edges: ties, saturation, subnormals, zeros, the largest and smallest values."""
    rows = []
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.5, 6.0, 7.0, 7.99, 4.0, 0.24, 0.26], np.float32)
    for s in (1.0, 2.0 ** -126, 2.0 ** 100, 3.0, 2.0 ** -20):
        r = np.zeros(cols, np.float32)
        for i in range(cols):
            r[i] = ties[i % len(ties)] * s * (-1) ** (i // 3)
        rows.append(r)
    rows.append(np.zeros(cols, np.float32))
    rows.append(np.full(cols, -0.0, np.float32))
    rows.append(np.full(cols, np.finfo(np.float32).max, np.float32))
    rows.append(np.full(cols, np.float32(1e-45)))
    rows.append(np.where(np.arange(cols) % 32 == 3, np.float32(1.1754944e-38), np.float32(1e-44)))
    for bad in (np.nan, np.inf, -np.inf):
        r = np.linspace(-3, 3, cols).astype(np.float32)
        r[cols // 2] = bad
        rows.append(r)
    return np.stack(rows).astype(np.float32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (2, 32), (5, 33), (7, 250), (13, 4096), (2, 8191)])
def test_mx_quantize_and_back(dtype, rows, cols):
    x = rand(rows, cols, seed=rows, dtype=dtype, std=2)
    q = mx.quantize(x)
    codes, scales = R.mx_quantize(f64(x).astype(np.float32))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    want = R.mx_values(codes, scales)[:, :cols]
    for dt in (F32, BF16):
        assert np.array_equal(f64(mx.dequantize(q, dt)), want)


@pytest.mark.parametrize("cols", [32, 64, 250])
def test_mx_edges(cols):
    x = special_rows(cols)
    q = mx.quantize(torch.from_numpy(x).cuda())
    codes, scales = R.mx_quantize(x)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    got, want = f64(mx.dequantize(q, F32)), R.mx_values(codes, scales)[:, :cols]
    assert np.array_equal(got, want, equal_nan=True)


def test_mx_strided_leading_shape_and_empty():
    big = rand(9, 200, seed=1, dtype=BF16)
    v = big[:, 3:3 + 64]
    a, b = mx.quantize(v), mx.quantize(v.contiguous())
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    w = rand(2, 3, 64, seed=2)
    q = mx.quantize(w)
    assert q.shape == (2, 3, 64)
    flat = mx.quantize(w.view(6, 64))
    assert torch.equal(q.codes.view(6, -1), flat.codes)
    assert mx.dequantize(q).shape == (2, 3, 64)
    wide = torch.zeros(6, 100, device="cuda")
    mx.dequantize(flat, out=wide[:, 5:69])
    assert torch.equal(wide[:, 5:69], mx.dequantize(flat, F32)) and (wide[:, :5] == 0).all() and (wide[:, 69:] == 0).all()
    assert mx.quantize(rand(0, 64)).shape == (0, 64)


def random_mx(shape, seed):
    q = mx.quantize(rand(*shape, seed=seed))
    return q, R.mx_values(q.codes.cpu().numpy(), q.scales.cpu().numpy())


def check_product(out, a, b, rows=slice(None)):
    """out[rows] against a @ b.T with the summation bound."""
    a = a[rows]
    ref = a @ b.T
    tol = (a.shape[1] * 2.0 ** -22) * (np.abs(a) @ np.abs(b).T) + ULP[out.dtype] * np.abs(ref)
    got = f64(out[rows])
    assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("rows,N,K", [(1, 1, 32), (1, 128, 4096), (3, 130, 96), (16, 64, 256), (17, 257, 544), (129, 100, 320),
                                      (300, 520, 1056), (260, 768, 512)])
def test_mx_matmul_dense(out_dtype, rows, N, K):
    a, av = random_mx((rows, K), 1)
    b, bv = random_mx((N, K), 2)
    out = mx.matmul(a, b, out_dtype=out_dtype)
    check_product(out, av, bv)


@pytest.mark.parametrize("sizes", [[5, 0, 1, 130, 0], [0, 0, 3], [64, 64, 64, 64], [1, 1, 1, 1, 1, 1, 1], [300, 2, 0, 17, 128]])
@pytest.mark.parametrize("N,K", [(96, 128), (264, 800)])
def test_mx_matmul_grouped(sizes, N, K):
    G, rows = len(sizes), sum(sizes)
    a, av = random_mx((rows, K), 3)
    b, bv = random_mx((G, N, K), 4)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    out = mx.matmul(a, b, offsets=torch.from_numpy(off).cuda())
    for g in range(G):
        if sizes[g]:
            check_product(out, av, bv[g], slice(off[g], off[g + 1]))


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("rows,N,K", [(2600, 4104, 224), (5000, 2050, 64), (130, 33000, 96)])
def test_mx_matmul_many_tiles_a_cta(out_dtype, rows, N, K):
    a, av = random_mx((rows, K), 11)
    b, bv = random_mx((N, K), 12)
    check_product(mx.matmul(a, b, out_dtype=out_dtype), av, bv)


@pytest.mark.parametrize("average", [40, 100, 260])
@pytest.mark.parametrize("N,K", [(1030, 352)])
def test_mx_matmul_grouped_many_tiles_a_cta(average, N, K):
    G = 24
    sizes = np.random.default_rng(average).integers(0, 2 * average, G)
    sizes[5] = 0
    rows = int(sizes.sum())
    a, av = random_mx((rows, K), 13)
    b, bv = random_mx((G, N, K), 14)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    out = mx.matmul(a, b, offsets=torch.from_numpy(off).cuda(), out_dtype=BF16)
    for g in range(G):
        if sizes[g]:
            check_product(out, av, bv[g], slice(off[g], off[g + 1]))


def test_mx_matmul_rows_of_no_group_strided_out_and_bad_offsets():
    a, av = random_mx((40, 64), 5)
    b, bv = random_mx((2, 48, 64), 6)
    wide = torch.full((40, 60), 7.0, device="cuda")
    out = wide[:, 4:52]
    mx.matmul(a, b, offsets=torch.tensor([3, 20, 31], dtype=torch.int32, device="cuda"), out=out)
    check_product(out, av, bv[0], slice(3, 20))
    check_product(out, av, bv[1], slice(20, 31))
    assert (wide[:3] == 7).all() and (wide[31:] == 7).all() and (wide[:, :4] == 7).all() and (wide[:, 52:] == 7).all()
    # entries outside [0, rows] are clamped to it, descending ones hold no rows
    got = mx.matmul(a, b, offsets=torch.tensor([-5, 10, 900], dtype=torch.int32, device="cuda"))
    check_product(got, av, bv[0], slice(0, 10))
    check_product(got, av, bv[1], slice(10, 40))
    keep = torch.full((40, 48), 9.0, device="cuda")
    mx.matmul(a, b, offsets=torch.tensor([30, 12, 12], dtype=torch.int32, device="cuda"), out=keep)
    assert (keep == 9).all()


def test_mx_matmul_nan_scale_stays_in_its_row():
    x = rand(20, 128, seed=7)
    x[4, 40] = float("nan")
    a = mx.quantize(x)
    b, bv = random_mx((33, 128), 8)
    out = f64(mx.matmul(a, b))
    assert np.isnan(out[4]).all() and np.isfinite(np.delete(out, 4, 0)).all()


def test_mx_refusals():
    a, _ = random_mx((4, 64), 1)
    b, _ = random_mx((2, 8, 64), 2)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for bad in (lambda: mx.matmul(a, mx.empty(8, 96)), lambda: mx.matmul(a, b, offsets=off.long()),
                lambda: mx.matmul(a, b, offsets=off[:2]), lambda: mx.matmul(mx.empty(4, 48), mx.empty(8, 48)),
                lambda: mx.quantize(rand(2, 64).half()), lambda: mx.quantize(rand(2, 64), out=mx.empty(2, 32)),
                lambda: mx.dequantize(a, torch.float16), lambda: mx.quantize(rand(2, 64).cpu()),
                lambda: mx.MXTensor(a.codes, a.scales, 65)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(L.MoEError):
        mx.matmul(a, b)  # several groups, no offsets


def test_operators_in_a_row_see_each_other():
    # each call reads what the one before wrote and overwrites what the one before read
    def chain(r, w, b, wait):
        x, z, q = torch.empty_like(r), torch.empty_like(r), mx.empty(r.shape[0], r.shape[1])
        for _ in range(20):
            for step in (lambda: norm.pre(r, w, out=x), lambda: mx.quantize(x, out=q), lambda: mx.matmul(q, b, out=z),
                         lambda: norm.post(z, r, w, res_scale=0.5, out=r, next_w=w, next_out=x), lambda: mx.quantize(x, out=q),
                         lambda: mx.dequantize(q, out=z), lambda: norm.post(z, r, None, kind="none", branch_scale=0.25, out=r)):
                step()
                if wait:
                    torch.cuda.synchronize()
        return r

    for rows, D in ((1, 512), (7, 1024), (200, 2048)):
        b, _ = random_mx((D, D), 21)
        r, w = rand(rows, D, seed=22).to(BF16), rand(D, seed=23).to(BF16)
        assert torch.equal(chain(r.clone(), w, b, False), chain(r.clone(), w, b, True))


# ------------------------------------------------- the layer for few tokens

TOL = {"f32": 1e-4, "bf16": 1e-2, "fp8": 5e-2, "mxfp4": 5e-2}


def few_case(dtype, T, D, E, I, k, zipf, seed=0, flags=0, out_dtype="f32"):
    shape = synth.LayerShape("few", T, D, E, I, k, "fp8" if dtype == "mxfp4" else dtype, zipf)
    inp = synth.make_inputs(shape, seed=seed, device="cuda")
    layer = MoELayer(D, E, I, k, dtype, inp, T_max=max(T, 1), has_router_bias=shape.has_bias, flags=flags,
                     out_dtype=out_dtype)
    return shape, inp, layer


def few_check(dtype, shape, inp, layer, out):
    T, E, k = shape.T, shape.E, shape.top_k
    z = oracle.logits(inp["x"].cpu(), inp["w_router"].cpu(), inp["b_router"].cpu() if shape.has_bias else None)
    v = layer.ws_view(T, "blob", torch.int32, (2, T, k)).cpu().numpy()
    logits = f64(layer.ws_view(T, "logits", torch.float32, (T, E)))
    assert np.abs(logits - z).max() <= 2e-4 * max(1.0, np.abs(z).max())
    idx, w = oracle.topk(logits, k)
    assert np.array_equal(v[0], idx)
    assert np.allclose(v[1].view(np.float32), w, rtol=1e-6, atol=1e-7)
    if dtype == "mxfp4":
        val = lambda n: R.mx_values(layer.w["w_" + n].cpu().numpy(), layer.w["s_" + n].cpu().numpy())  # noqa: E731
        ref = R.mx_layer(f64(inp["x"]), idx, w, val("gate"), val("up"), val("down"))
    else:
        ex, sub = experts_for_tokens(idx, inp, dtype, E)
        ref = oracle.moe_tokens(inp["x"].cpu(), sub, w, ex)
    extra = 2.0 ** -8 * np.abs(ref).max() / np.sqrt(np.mean(ref ** 2)) if out.dtype == BF16 else 0.0
    assert rel_max_err(f64(out), ref) <= TOL[dtype] + extra


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("T,D,E,I,k,zipf", [(1, 512, 32, 256, 4, None), (1, 256, 1, 128, 1, None), (5, 512, 32, 256, 4, 1.2),
                                            (16, 768, 20, 128, 10, 1.0), (9, 256, 33, 384, 32, None),
                                            (8, 1280, 64, 256, 2, 1.2)])
def test_few_layer(dtype, T, D, E, I, k, zipf):
    shape, inp, layer = few_case(dtype, T, D, E, I, k, zipf)
    out = layer.forward_few(inp["x"])
    layer.check()
    few_check(dtype, shape, inp, layer, out)
    # and again: nothing of the first call is left to disturb the second
    assert torch.equal(out, layer.forward_few(inp["x"]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("T,D,E,I,k,zipf", [(2, 1024, 8, 2176, 3, None), (1, 512, 5, 2176, 4, None), (1, 4096, 24, 1024, 10, None),
                                            (16, 512, 700, 128, 20, None), (12, 512, 6, 4096, 4, 1.0)])
def test_few_layer_many_tiles_a_warp(dtype, T, D, E, I, k, zipf):
    shape, inp, layer = few_case(dtype, T, D, E, I, k, zipf, seed=3)
    out = layer.forward_few(inp["x"])
    layer.check()
    few_check(dtype, shape, inp, layer, out)
    assert torch.equal(out, layer.forward_few(inp["x"]))


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_few_agrees_with_moe_forward_and_takes_its_options(dtype):
    shape, inp, layer = few_case(dtype, 7, 512, 48, 256, 6, 1.0)
    T, E, k = 7, 48, 6
    blob, logits = torch.empty(2, T, k, dtype=torch.int32, device="cuda"), torch.empty(T, E, device="cuda")
    a = layer.forward_few(inp["x"], blob_out=blob, logits_out=logits)
    words = torch.empty(T, k, dtype=torch.int32, device="cuda")
    L.moe_pack_routing_words(layer.plan, T, layer.ws, words)
    assert torch.equal(words & 0xFFFF, blob[0])
    b = layer.forward(inp["x"])
    layer.check()
    assert rel_max_err(f64(a), f64(b)) <= 2 * TOL[dtype]
    assert torch.equal(layer.forward_few(inp["x"]), a)  # after a moe_forward on the same workspace
    assert torch.equal(blob[0], layer.ws_view(T, "blob", torch.int32, (2, T, k))[0])
    assert rel_max_err(f64(logits), oracle.logits(inp["x"].cpu(), inp["w_router"].cpu(), inp["b_router"].cpu())) <= 1e-4


@pytest.mark.parametrize("flags", [L.MOE_FLAG_DOWN_HILO, L.MOE_FLAG_FORCE_SIMT])
def test_few_layer_under_flags(flags):
    shape, inp, layer = few_case("bf16", 3, 256, 16, 128, 2, None, flags=flags)
    out = layer.forward_few(inp["x"])
    few_check("bf16", shape, inp, layer, out)


@pytest.mark.parametrize("dtype", ["bf16", "mxfp4"])
def test_few_bf16_output_other_stream_and_graph(dtype):
    shape, inp, layer = few_case(dtype, 4, 512, 32, 256, 4, None, out_dtype="bf16")
    out = layer.forward_few(inp["x"])
    few_check(dtype, shape, inp, layer, out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = torch.empty_like(out)
    with torch.cuda.stream(s):
        layer.forward_few(inp["x"], out=again)
    s.synchronize()
    assert torch.equal(out, again)
    x = inp["x"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward_few(x, out=again)
    x.copy_(x.flip(0))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out.flip(0))
    layer.check()


def test_few_ties_nonfinite_logits_and_refusals():
    shape, inp, layer = few_case("bf16", 4, 256, 16, 128, 4, None)
    x = inp["x"].clone()
    x[2] = 0  # every logit equal: the lowest indices
    layer.forward_few(x)
    layer.check()
    blob = layer.ws_view(4, "blob", torch.int32, (2, 4, 4))
    assert blob[0, 2].tolist() == [0, 1, 2, 3]
    x[1, 3] = float("inf")
    layer.forward_few(x)
    with pytest.raises(L.MoEError) as e:
        layer.check()
    assert e.value.status == L.MOE_ERR_NONFINITE
    layer.forward_few(inp["x"])  # the next call clears it
    layer.check()
    assert layer.forward_few(inp["x"][:0]).shape == (0, 256)
    big = MoELayer(256, 16, 128, 4, "bf16", inp, T_max=64)
    with pytest.raises(L.MoEError) as e:
        big.forward_few(torch.zeros(17, 256, dtype=BF16, device="cuda"))
    assert e.value.status == L.MOE_ERR_UNSUPPORTED


# ------------------------------------------- the 4-bit layer at every size

@pytest.mark.parametrize("T,D,E,I,k,zipf", [(1, 256, 16, 128, 2, None), (40, 512, 32, 256, 4, 1.2), (300, 384, 20, 128, 3, 1.0),
                                            (1100, 256, 24, 128, 2, None)])
def test_mxfp4_layer_forward(T, D, E, I, k, zipf):
    shape, inp, layer = few_case("mxfp4", T, D, E, I, k, zipf)
    out = layer.forward(inp["x"])
    layer.check()
    # y is rounded to bf16 before the sum: 2^-9 of each of the k + 1 terms, inside the type's bound
    few_check("mxfp4", shape, inp, layer, out)
    v = layer.views(T)
    src = v["src_tok"].long()
    q = mx.quantize(inp["x"])
    assert torch.equal(v["xq"], q.codes) and torch.equal(v["xq_scale"], q.scales)
    assert torch.equal(v["xp"], q.codes[src[:T * k]]) and torch.equal(v["xp_scale"], q.scales[src[:T * k]])
    assert torch.equal(layer.forward(inp["x"]), out)
    if T <= L.MOE_FEW_MAX:
        assert rel_max_err(f64(layer.forward_few(inp["x"])), f64(out)) <= 2 * TOL["mxfp4"]


def test_mxfp4_stages_agree_with_forward():
    shape, inp, layer = few_case("mxfp4", 70, 256, 16, 128, 2, 1.0)
    x = inp["x"]
    out = layer.forward(x)
    layer.init_ws()
    layer.route(x)
    layer.permute(x)
    layer.gemm_gateup(x)
    layer.gemm_down(70)
    assert torch.equal(layer.unpermute(70), out)


# --------------------------------------------------------------- MoEBlock

@pytest.mark.parametrize("dtype", ["bf16", "mxfp4"])
def test_block_runs_the_operators_together(dtype):
    shape, inp, layer = few_case(dtype, 6, 512, 32, 256, 4, 1.0, out_dtype="bf16")
    D = 512
    pre_w, post_w, next_w, gate = (rand(D, seed=s, dtype=BF16) for s in (11, 12, 13, 14))
    block = MoEBlock(layer, pre_w=pre_w, post_w=post_w, next_w=next_w, gate=gate, gate_sigmoid=True, res_scale=0.9,
                     branch_scale=0.5, w_offset=1.0)
    r = rand(6, D, seed=15, std=2)
    r2, n2 = block.forward(r)
    assert r2.dtype == F32 and n2.dtype == BF16
    n = norm.pre(r, pre_w, w_offset=1.0, out=torch.empty(6, D, dtype=BF16, device="cuda"))
    y = layer.forward_few(n)
    ref = 0.9 * f64(r) + 0.5 / (1 + np.exp(-f64(gate))) * R.norm(f64(y), "rms", 1e-6, f64(post_w), None, 1.0)
    assert np.abs(f64(r2) - ref).max() <= 1e-5 * np.abs(ref).max()
    check_norm(n2, f64(r2), "rms", 1e-6, f64(next_w), None, 1.0)
    again, none = block.forward(r, n=n, next_norm=False)
    assert none is None and torch.equal(again, r2)


def test_block_prefill_runs_moe_forward():
    shape, inp, layer = few_case("mxfp4", 50, 256, 16, 128, 2, None, out_dtype="bf16")
    block = MoEBlock(layer, post_kind="none", next_kind="none")
    r = rand(50, 256, seed=1, dtype=BF16)
    r2, none = block.forward(r)
    n = norm.pre(r)
    assert none is None and torch.equal(r2, norm.post(layer.forward(n), r, kind="none")[0])
