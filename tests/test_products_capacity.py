"""The experts' products on buffers of fixed capacity, as captured steps and
shards of the experts have them: few of the rows in use, in few of the groups.

A row's result does not depend on the rows and groups beside it, so it is the
same, bit by bit, as in a buffer of the rows in use alone, as long as both
calls are few-row ones (at most max(8 G, 32) rows of the buffer)."""
import pytest
import torch

import product_ref as R
from sparse_moe_expert_02_gb300 import grouped, int4
from test_products import DT, check, gen, offsets_of, operands, randn, weights4

pytestmark = pytest.mark.gpu


def exact4(x, w, offsets, out):
    """int4.matmul of few rows, which multiplies the weights' values themselves: off by the sums' roundings and the
    output's alone (K products and a scale for every 32 of them, which the bound's n 2^-23 has room for)."""
    assert x.shape[0] <= max(8 * w.codes.shape[0], 32)
    held, word = out.clone(), torch.zeros(4, dtype=torch.int32, device="cuda")
    assert int4.matmul(x, w, offsets, out=out, err=word) is out and not word.any()
    v = torch.stack([R.int4_values(w.codes[g], w.scales[g], None if w.zeros is None else w.zeros[g], w.group) for g in range(w.codes.shape[0])])
    R.close(out, *R.product("fwd", x, v, R.ranges(offsets.tolist(), x.shape[0]), held, out.dtype))


def sizes_in_use(kind, G):
    """Groups of the rows in use: spread, all in one group (the first, one between, the last), or none."""
    n = [0] * G
    if kind == "spread":
        for i, g in enumerate((1, G // 3, G // 2, G - 2)):
            n[g] += (1, 2, 4, 3)[i]
    elif kind != "none":
        n[{"first": 0, "between": G // 2, "last": G - 1}[kind]] = 24
    return n


@pytest.mark.parametrize("group,zeros,scale", [(128, False, "bf16"), (64, True, "bf16"), (32, True, "f32")])
@pytest.mark.parametrize("kind", ["spread", "first", "between", "last", "none"])
@pytest.mark.parametrize("G,N,K", [(128, 1000, 1024), (128, 1024, 384), (128, 1024, 1024), (128, 4096, 1024), (64, 4096, 384), (800, 64, 128)])
def test_int4_few_rows_in_use(G, N, K, kind, group, zeros, scale):
    rows = 1024 if G == 128 else 8 * G
    sizes = sizes_in_use(kind, G)
    used = sum(sizes)
    w = weights4(G, N, K, group, zeros, scale)
    x = torch.full((rows, K), float("nan"), dtype=torch.bfloat16, device="cuda")  # rows of no group are not read
    x[:used] = randn(gen(1), used, K)
    for out_dtype in DT.values():
        out = randn(gen(2), rows, N, dtype=out_dtype)
        held = out.clone()
        exact4(x, w, offsets_of(sizes), out)
        assert torch.equal(out[used:], held[used:])
        if used:
            assert torch.equal(out[:used], int4.matmul(x[:used].contiguous(), w, offsets_of(sizes), out_dtype=out_dtype))


@pytest.mark.parametrize("kind", ["spread", "between", "none"])
@pytest.mark.parametrize("N,K", [(1000, 1024), (1024, 384), (72, 200)])
def test_few_rows_in_use(N, K, kind):
    G, rows = 128, 1024
    sizes = sizes_in_use(kind, G)
    used = sum(sizes)
    x, w = operands("fwd", rows, N, K, G, torch.bfloat16)
    x[used:] = float("nan")
    for out_dtype in DT.values():
        out = randn(gen(2), rows, N, dtype=out_dtype)
        held = out.clone()
        check("fwd", x, w, offsets_of(sizes), out)
        assert torch.equal(out[used:], held[used:])
        if used:
            assert torch.equal(out[:used], grouped.matmul(x[:used].contiguous(), w, offsets_of(sizes), out_dtype=out_dtype))


def test_a_captured_step_of_fixed_capacity():
    """One capture; replayed for a full buffer, a few rows, none, and rows in other places of the buffer."""
    G, rows, N, K = 128, 1024, 1024, 512
    w = weights4(G, N, K, 64, True, "bf16")
    x, at = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda"), torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    out = torch.zeros((rows, N), device="cuda")
    int4.matmul(x, w, at, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        int4.matmul(x, w, at, out=out)
    full = [8] * G
    for i, (sizes, before) in enumerate(((full, 0), (sizes_in_use("spread", G), 0), (sizes_in_use("none", G), 0), (sizes_in_use("last", G), 997),
                                         (sizes_in_use("spread", G), 500), (full, 0))):
        x.copy_(randn(gen(i), rows, K))
        at.copy_(offsets_of(sizes, before))
        out.fill_(i)
        graph.replay()
        want = torch.full_like(out, i)
        exact4(x, w, at, want)
        assert torch.equal(out, want)
