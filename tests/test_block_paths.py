"""Paths of the block operators that small sizes do not reach, against the same
64-bit definitions and with the tolerances of test_block_ops."""
import numpy as np
import pytest
import torch

import block_ref as R
import oracle
from parity_util import rel_max_err
from sparse_moe_expert_02_gb300 import MoEBlock, MoELayer, mx, norm
from sparse_moe_expert_02_gb300 import _lib as L
from test_block_ops import (BF16, F32, TOL, ULP, check_norm, check_product, f64, few_case, few_check, norm_tol, rand,
                            random_mx)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,T", [(43136, 2), (49152, 5)])
def test_few_takes_rows_too_wide_for_shared_memory(D, T):
    shape, inp, layer = few_case("f32", T, D, 4, 64, 2, None)
    out = layer.forward_few(inp["x"])
    layer.check()
    few_check("f32", shape, inp, layer, out)
    assert torch.equal(out, layer.forward(inp["x"]))


def test_few_fp32_activation_is_accurate():
    # one expert and identity down weights: out[i] = silu(a[i]) * u[i], with a and u exact.  fp32 arithmetic: the
    # exponential within 2 ulp, then a sum, a product and a quotient of half an ulp each; 4 ulp of the result
    D, a = 512, torch.linspace(-60, 60, 512)
    u = torch.linspace(0.5, 2, D)
    eye, zero = torch.eye(D), torch.zeros(D, D)
    gate, up = zero.clone(), zero.clone()
    gate[:, 0], up[:, 0] = a, u
    w = {"w_router": torch.zeros(1, D), "w_gate": torch.stack([gate, zero]), "w_up": torch.stack([up, zero]),
         "w_down": torch.stack([eye, zero])}
    layer = MoELayer(D, 1, D, 1, "f32", {n: t.cuda() for n, t in w.items()}, T_max=4)
    x = torch.zeros(3, D, device="cuda")
    x[:, 0] = 1
    ref = (a.double() / (1 + torch.exp(-a.double())) * u.double()).cuda()
    out = layer.forward_few(x)
    layer.check()
    assert ((out.double() - ref).abs() <= 4 * 2.0 ** -23 * ref.abs()).all(), ((out.double() - ref) / ref).abs().max()


@pytest.mark.parametrize("gate_by", ["channel", "token", "full"])
def test_block_takes_a_gate_by_call_and_biases(gate_by):
    shape, inp, layer = few_case("bf16", 24, 256, 16, 128, 2, None, out_dtype="bf16")
    D = 256
    pre_w, pre_b, post_w, post_b, next_w, next_b = (rand(D, seed=s, dtype=BF16) for s in range(31, 37))
    block = MoEBlock(layer, kind="layer", pre_w=pre_w, pre_b=pre_b, post_w=post_w, post_b=post_b, next_w=next_w, next_b=next_b,
                     gate_by=gate_by, gate_sigmoid=True, branch_scale=0.5)
    for T in (3, 20, 1):
        r = rand(T, D, seed=T)
        gate = rand(*{"channel": (D,), "token": (T,), "full": (T, D)}[gate_by], seed=40 + T)
        n = norm.pre(r, pre_w, pre_b, kind="layer", out=torch.empty(T, D, dtype=BF16, device="cuda"))
        y = layer.forward_few(n) if T <= 16 else layer.forward(n)
        want = norm.post(y, r, post_w, post_b, kind="layer", gate=gate, gate_by=gate_by, gate_sigmoid=True, branch_scale=0.5,
                         next_w=next_w, next_b=next_b, next_out=torch.empty(T, D, dtype=BF16, device="cuda"))
        got = block.forward(r, gate=gate)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # an own gate stays what calls without one use
        assert torch.equal(block.forward(r)[0], norm.post(y, r, post_w, post_b, kind="layer", branch_scale=0.5)[0])


# ------------------------------------------------------------ long prompts

# Row counts from which a block of bf16 takes row after row (three at least): 456 times the blocks an SM holds.
LONG_POST = [(4777, 520, BF16, BF16, BF16), (2001, 4096, BF16, BF16, BF16), (1500, 4104, F32, F32, BF16), (7301, 1024, BF16, F32, F32),
             (3003, 2056, F32, BF16, BF16), (900, 8192, F32, F32, F32), (7301, 1032, BF16, BF16, F32), (1000, 8192, BF16, BF16, BF16),
             (500, 14336, BF16, BF16, BF16)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,D,xt,ot", [(4777, 520, F32, F32), (2900, 4096, BF16, BF16), (1537, 4104, F32, BF16), (500, 16384, BF16, F32),
                                       (9200, 1024, BF16, BF16), (5001, 520, BF16, F32), (1900, 4104, BF16, BF16)])
def test_norm_pre_of_a_long_prompt(kind, T, D, xt, ot):
    wide = rand(T, D + 16, seed=1, dtype=xt, std=3)
    x, w, b = wide[:, 8:8 + D], rand(D, seed=2), rand(D, seed=3)
    room = torch.full((T, D + 8), 7.0, dtype=ot, device="cuda")
    out = room[:, :D]
    norm.pre(x, w, b, kind=kind, eps=1e-5, w_offset=1.0, out=out)
    check_norm(out, f64(x), kind, 1e-5, f64(w), f64(b), 1.0)
    assert (room[:, D:] == 7).all()


@pytest.mark.parametrize("gate_by", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("T,D,yt,rt,nt", LONG_POST)
def test_norm_post_of_a_long_prompt_in_place(gate_by, T, D, yt, rt, nt):
    y, w, nw, b = rand(T, D + 8, seed=1, dtype=yt, std=2)[:, 8:], rand(D, seed=3), rand(D, seed=4), rand(D, seed=6)
    wide = rand(T, D + 8, seed=2, dtype=rt)
    r, keep = wide[:, :D], wide.clone()
    gate = {"none": None, "channel": rand(D, seed=5), "token": rand(T, seed=5), "full": rand(T, D + 8, seed=5, dtype=yt)[:, :D]}[gate_by]
    out, n = norm.post(y, r, w, b, kind="layer", eps=1e-6, gate=gate, gate_by=gate_by, gate_sigmoid=True, res_scale=0.5,
                       branch_scale=-1.5, next_w=nw, next_kind="rms", next_out=torch.empty(T, D, dtype=nt, device="cuda"), out=r)
    assert out.data_ptr() == r.data_ptr() and torch.equal(wide[:, D:], keep[:, D:])
    g = 1.0 if gate is None else 1 / (1 + np.exp(-f64(gate)))
    g = g[:, None] if gate_by == "token" else g
    branch = R.norm(f64(y), "layer", 1e-6, f64(w), f64(b))
    ref = 0.5 * f64(keep[:, :D]) - 1.5 * g * branch
    tol = 1.5 * np.abs(g) * (norm_tol(f64(y), "layer", 1e-6, f64(w), 0.0, branch, F32) + 2.0 ** -20 * np.abs(branch) + 2.0 ** -22 * np.abs(f64(b)))
    tol = tol + 2.0 ** -22 * np.abs(f64(keep[:, :D])) + ULP[rt] * np.abs(ref)
    assert (np.abs(f64(out) - ref) <= tol).all()
    check_norm(n, f64(out), "rms", 1e-6, f64(nw), None, 0.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols,ld", [(5003, 4096, 4096), (2501, 4096, 4096), (5003, 4096, 4104), (701, 4001, 4001), (20003, 33, 40)])
def test_mx_of_many_elements(dtype, rows, cols, ld):
    # more than a pass of the grid: against calls of a few rows each, and some rows against the definition
    x = rand(rows, ld, seed=1, dtype=dtype, std=2)[:, :cols]
    q = mx.quantize(x)
    step = 300
    for r in range(0, rows, step):
        part = mx.quantize(x[r:r + step])
        assert torch.equal(q.codes[r:r + step], part.codes) and torch.equal(q.scales[r:r + step], part.scales)
    some = [0, 1, rows // 2, rows - 2, rows - 1]
    codes, scales = R.mx_quantize(f64(x[some]).astype(np.float32))
    assert np.array_equal(q.codes[some].cpu().numpy(), codes) and np.array_equal(q.scales[some].cpu().numpy(), scales)
    room = torch.zeros(rows, ld + 8, dtype=dtype, device="cuda")
    mx.dequantize(q, out=room[:, :cols])
    assert (room[:, cols:] == 0).all()
    for r in range(0, rows, step):
        assert torch.equal(room[r:r + step, :cols], mx.dequantize(mx.MXTensor(q.codes[r:r + step], q.scales[r:r + step], cols), dtype))
    assert np.array_equal(f64(room[some, :cols]), R.mx_values(codes, scales)[:, :cols])


# K of 2048 and 4096: scales in 16-byte loads; 1152: 4-byte; 2880 and 2848: single bytes.
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("rows,N,K", [(3001, 4104, 4096), (2900, 4100, 1152), (2600, 4104, 2880)])
def test_mx_matmul_of_a_long_prompt(out_dtype, rows, N, K):
    a, av = random_mx((rows, K), 11)
    b, bv = random_mx((N, K), 12)
    check_product(mx.matmul(a, b, out_dtype=out_dtype), av, bv)


@pytest.mark.parametrize("average", [20, 60, 300])
@pytest.mark.parametrize("N,K", [(1032, 2048), (1030, 1152), (520, 2848)])
def test_mx_matmul_grouped_with_long_rows(average, N, K):
    G = 33
    sizes = np.random.default_rng(average).integers(0, 2 * average, G)
    sizes[[0, 7, 32]] = 0, 1, 0
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    a, av = random_mx((int(off[-1]), K), 13)
    b, bv = random_mx((G, N, K), 14)
    out = mx.matmul(a, b, offsets=torch.from_numpy(off).cuda(), out_dtype=F32)
    for g in range(G):
        if sizes[g]:
            check_product(out, av, bv[g], slice(off[g], off[g + 1]))


def test_mxfp4_layer_of_a_long_prompt():
    # h is of more than a pass of the grid; some tokens against the definition
    T, D, E, I, k = 1100, 256, 4, 4096, 2
    shape, inp, layer = few_case("mxfp4", T, D, E, I, k, 1.0)
    out = layer.forward(inp["x"])
    layer.check()
    some = torch.tensor([0, 1, 2, 500, 777, 1097, 1098, 1099], device="cuda")
    logits = f64(layer.ws_view(T, "logits", torch.float32, (T, E)))[some.cpu().numpy()]
    idx, w = oracle.topk(logits, k)
    val = lambda n: R.mx_values(layer.w["w_" + n].cpu().numpy(), layer.w["s_" + n].cpu().numpy())  # noqa: E731
    ref = R.mx_layer(f64(inp["x"][some]), idx, w, val("gate"), val("up"), val("down"))
    assert rel_max_err(f64(out[some]), ref) <= TOL["mxfp4"]


# --------------------------------------- few tokens in launches of fewer still

@pytest.mark.parametrize("dtype,D", [("bf16", 7168), ("fp8", 7168), ("mxfp4", 7168), ("f32", 3584), ("bf16", 16384), ("f32", 16384)])
@pytest.mark.parametrize("T", [16, 13])
def test_few_layer_of_wide_rows(dtype, D, T):
    shape, inp, layer = few_case(dtype, T, D, 6, 128, 2, None, seed=2)
    out = layer.forward_few(inp["x"])
    layer.check()
    few_check(dtype, shape, inp, layer, out)
    assert torch.equal(out, layer.forward_few(inp["x"]))
    x = inp["x"].clone()
    x[T - 1, 3] = float("inf")  # in the last launch: reported, and its own row only (others add up in another order at most)
    got = layer.forward_few(x)
    with pytest.raises(L.MoEError) as e:
        layer.check()
    assert e.value.status == L.MOE_ERR_NONFINITE
    assert rel_max_err(f64(got[:T - 1]), f64(out[:T - 1])) <= 1e-5


def test_block_takes_the_layer_that_pays():
    shape, inp, layer = few_case("mxfp4", 16, 1024, 32, 512, 10, None, out_dtype="bf16")
    block = MoEBlock(layer)
    for T in (4, 16):
        r = rand(T, 1024, seed=T, dtype=BF16)
        n = norm.pre(r)
        y = layer.forward_few(n) if T == 4 else layer.forward(n)
        assert torch.equal(block.forward(r, next_norm=False)[0], norm.post(y, r)[0])


# ------------------------------------------------------- graphs and streams

@pytest.mark.parametrize("rows,D", [(1, 512), (7, 1024), (301, 1023), (2000, 2048)])
def test_operators_captured_with_copies_and_a_second_stream(rows, D):
    # launches, copies, memsets and an event's wait between the operators, eagerly and as a graph replayed on new inputs
    K = D // 32 * 32
    b, _ = random_mx((D, K), 21)
    w = rand(D, seed=23)
    r, x, z = (torch.empty(rows, D, device="cuda") for _ in range(3))
    side_out, back = torch.empty(rows, D, dtype=BF16, device="cuda"), torch.empty(rows, K, dtype=BF16, device="cuda")
    q = mx.empty(rows, K)
    side, done = torch.cuda.Stream(), torch.cuda.Event()

    def step():
        main = torch.cuda.current_stream()
        norm.pre(r, w, out=x)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            norm.pre(x, w, kind="layer", out=side_out)
            done.record()
        mx.quantize(x[:, :K], out=q)
        z.zero_()
        mx.matmul(q, b, out=z)
        mx.dequantize(q, out=back)
        main.wait_event(done)
        norm.post(z, r, w, gate=side_out, gate_by="full", res_scale=0.5, out=r)
        x.copy_(r)
        norm.post(x, r, None, kind="none", branch_scale=0.25, out=r)

    inputs = [rand(rows, D, seed=30 + i) for i in range(3)]
    want = []
    for v in inputs:
        r.copy_(v)
        step()
        want.append((r.clone(), back.clone(), side_out.clone()))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    for v, (a, c, d) in zip(inputs, want):
        r.copy_(v)
        g.replay()
        assert torch.equal(r, a) and torch.equal(back, c) and torch.equal(side_out, d)


def test_few_fp32_sums_are_no_single_chain():
    # h = silu(8) * up . x of 4096 random terms.  A chain of n fp32 additions is off by some 2.5e-8 sqrt(n/2) of the sum
    # (rms; half an ulp uniformly, partial sums growing): 1.1e-6 for one of 4096, 2e-7 for one of 128 blocks of 32,
    # whose own chains are of far smaller sums; silu adds 1.2e-7.  Between the two: 5e-7
    T, D, I = 3, 4096, 512
    x = rand(T, D, seed=1)
    x[:, 0] = 8
    gate, up = torch.zeros(2, I, D, device="cuda"), rand(2, I, D, seed=2)
    gate[:, :, 0], up[:, :, 0] = 1, 0
    layer = MoELayer(D, 1, I, 1, "f32", {"w_router": rand(1, D, seed=3), "w_gate": gate, "w_up": up, "w_down": rand(2, D, I, seed=4)}, T_max=T)
    layer.forward_few(x)
    layer.check()
    h = f64(layer.ws_view(T, "few", F32, (2 * T, I)))
    ref = 8 / (1 + np.exp(-8.0)) * np.concatenate([f64(x) @ f64(up[e]).T for e in (0, 1)])
    assert np.sqrt(np.mean((h - ref) ** 2) / np.mean(ref ** 2)) <= 5e-7
