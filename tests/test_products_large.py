"""The experts' products at sizes where every block works through several tiles
and its rings of stages go round: against 64 bits, with the bounds of
product_ref."""
import pytest
import torch

import product_ref as R
from sparse_moe_expert_02_gb300 import grouped, int4
from test_products import DT, check, check4, gen, offsets_of, operands, out_shape, randn, weights4

pytestmark = pytest.mark.gpu


def ragged(rows, G, seed):
    """G sizes that sum to rows: one empty, one of a single row, the others uneven and odd."""
    g = torch.Generator().manual_seed(seed)
    p = torch.rand(G, generator=g) + 0.2
    n = [int(v) | 1 for v in (p / p.sum() * (rows - 40)).tolist()]
    n[0], n[1] = 0, 1
    n[-1] += rows - sum(n)
    return n


@pytest.mark.parametrize("op,rows,N,K,G", [
    ("fwd", 9001, 1024, 320, 5), ("fwd", 5003, 1152, 200, 7), ("fwd", 12007, 256, 72, 6), ("fwd", 3001, 2048, 1000, 40), ("fwd", 4999, 4096, 136, 1),
    ("dx", 9001, 320, 1024, 5), ("dx", 5003, 200, 1152, 7), ("dx", 3001, 1000, 2048, 40), ("dx", 4999, 136, 4096, 1), ("dx", 700, 72, 4224, 12),
    ("dw", 5003, 1024, 1024, 6), ("dw", 6007, 640, 2304, 9), ("dw", 2403, 384, 4096, 6), ("dw", 2999, 1024, 2048, 40), ("dw", 2047, 2048, 2304, 1),
    ("fwd", 6001, 1031, 333, 5), ("dx", 6001, 333, 1031, 5), ("dw", 5001, 513, 1030, 5), ("dw", 5001, 1024, 1030, 5)])
def test_product_of_many_tiles(op, rows, N, K, G):
    a, b = operands(op, rows + 3, N, K, G, torch.bfloat16)
    at = offsets_of(ragged(rows, G, rows) if G > 1 else [rows], 2)
    for out_dtype in DT.values():
        check(op, a, b, at, randn(gen(5), *out_shape(op, rows + 3, N, K, G), dtype=out_dtype))
    if op == "dw":
        for out_dtype in DT.values():
            check(op, a, b, at, randn(gen(6), G, N, K, dtype=out_dtype), accumulate=True)


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("rows,N,K,G", [(3001, 500, 333, 5), (900, 1000, 1024, 3), (2001, 129, 260, 20)])
def test_fp32_product_of_many_tiles(op, rows, N, K, G):
    a, b = operands(op, rows + 3, N, K, G, torch.float32)
    check(op, a, b, offsets_of(ragged(rows, G, rows), 2), randn(gen(5), *out_shape(op, rows + 3, N, K, G)))


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
def test_nothing_leaks_between_many_tiles(op):
    """Infinities beside the groups and in an empty group's matrix, pairs of CTAs at work."""
    rows, N, K, G = 4003, 1024, 1024, 6
    a, b = operands(op, rows + 7, N, K, G, torch.bfloat16)
    sizes = ragged(rows, G, 1)
    a[:2], a[rows + 2:] = float("inf"), float("nan")
    if op == "dw":
        b[:2], b[rows + 2:] = float("nan"), float("inf")
    else:
        b[0] = float("nan")
    out = torch.zeros(out_shape(op, rows + 7, N, K, G), dtype=torch.bfloat16, device="cuda")
    check(op, a, b, offsets_of(sizes, 2), out)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group,zeros,scale", [(128, False, "bf16"), (64, True, "bf16"), (32, True, "f32")])
@pytest.mark.parametrize("rows,N,K,G", [(2600, 1536, 1024, 2), (2047, 4096, 416, 1), (5000, 328, 2048, 3)])
def test_int4_matmul_of_many_tiles(dtype, group, zeros, scale, rows, N, K, G):
    rows = rows if dtype == "bf16" else rows // 8
    x = randn(gen(1), rows + 3, K, dtype=DT[dtype])
    w = weights4(G, N, K, group, zeros, scale)
    sizes = [rows] if G == 1 else [rows // 3, rows - rows // 3] + [0] * (G - 2)
    out = randn(gen(2), rows + 3, N, dtype=DT[dtype])
    check4(x, w, offsets_of(sizes, 1), out)
    for _ in range(4):
        again = out.clone()
        assert torch.equal(int4.matmul(x, w, offsets_of(sizes, 1), out=again), out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group,zeros,scale", [(128, False, "bf16"), (64, True, "bf16"), (32, True, "f32"), (32, False, "bf16")])
@pytest.mark.parametrize("G,N,K", [(40, 2048, 1280), (30, 1000, 1024), (40, 1004, 1280), (5, 4096, 8192), (3, 528, 16384)])
def test_int4_few_rows_of_many_tiles(dtype, group, zeros, scale, G, N, K):
    sizes = [(3 * i) % 9 for i in range(G)]
    rows = sum(sizes)
    x = randn(gen(1), rows, K, dtype=DT[dtype])
    w = weights4(G, N, K, group, zeros, scale)
    out = randn(gen(2), rows, N, dtype=DT[dtype])
    check4(x, w, offsets_of(sizes), out)
    for _ in range(3):
        assert torch.equal(int4.matmul(x, w, offsets_of(sizes)), out)


@pytest.mark.parametrize("G,N,K", [(40, 2048, 1280), (30, 1000, 1024), (40, 1004, 1280), (5, 4096, 8192), (1, 4096, 4096), (60, 520, 1000)])
def test_few_rows_of_many_tiles(G, N, K):
    sizes = [(3 * i) % 9 + (G == 1) for i in range(G)]
    rows = sum(sizes)
    x, w = operands("fwd", rows, N, K, G, torch.bfloat16)
    for out_dtype in DT.values():
        check("fwd", x, w, offsets_of(sizes), randn(gen(2), rows, N, dtype=out_dtype))
    first = grouped.matmul(x, w, offsets_of(sizes))
    for _ in range(3):
        assert torch.equal(grouped.matmul(x, w, offsets_of(sizes)), first)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("op,rows,N,K,G", [("dx", 45, 2536, 41, 1), ("fwd", 33, 20, 5000, 1), ("fwd", 70, 40, 1111, 3), ("dw", 3001, 33, 65, 1), ("dw", 1501, 70, 40, 4),
                                           ("dx", 1, 4096, 8, 1)])
def test_product_of_few_tiles_and_long_sums(op, rows, N, K, G, dtype):
    a, b = operands(op, rows + 3, N, K, G, DT[dtype])
    at = offsets_of(ragged(rows, G, rows) if G > 1 else [rows], 2)
    for out_dtype in DT.values():
        check(op, a, b, at, randn(gen(5), *out_shape(op, rows + 3, N, K, G), dtype=out_dtype))
        if op == "dw":
            check(op, a, b, at, randn(gen(5), G, N, K, dtype=out_dtype), accumulate=True)
    first = {"fwd": grouped.matmul, "dx": grouped.matmul_dx, "dw": grouped.matmul_dw}[op](a, b, at)
    again = {"fwd": grouped.matmul, "dx": grouped.matmul_dx, "dw": grouped.matmul_dw}[op](a, b, at)
    lo, hi = int(at[0]), int(at[-1])
    assert torch.equal(first[lo:hi] if op != "dw" else first, again[lo:hi] if op != "dw" else again)


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("each", [3, 20])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_most_groups(op, each, dtype):
    """1025 groups, every third of them empty."""
    G, N, K = 1025, 40, 72
    sizes = [each * (i % 3) for i in range(G)]
    rows = sum(sizes)
    a, b = operands(op, rows, N, K, G, DT[dtype])
    check(op, a, b, offsets_of(sizes), randn(gen(1), *out_shape(op, rows, N, K, G)))
    if op == "fwd":
        x = randn(gen(3), rows, 96, dtype=DT[dtype])
        check4(x, weights4(G, N, 96, 32, True, "bf16"), offsets_of(sizes), randn(gen(2), rows, N, dtype=DT[dtype]))


@pytest.mark.parametrize("group,zeros,scale", [(128, False, "bf16"), (64, True, "bf16"), (32, True, "f32"), (32, False, "bf16")])
@pytest.mark.parametrize("G,N,K", [(128, 1000, 1024), (100, 1024, 384), (200, 960, 128), (60, 2056, 1024)])
def test_int4_few_rows_of_short_columns(group, zeros, scale, G, N, K):
    sizes = [(5 * i) % 11 for i in range(G)]
    rows = sum(sizes)
    x = randn(gen(1), rows, K, dtype=torch.bfloat16)
    w = weights4(G, N, K, group, zeros, scale)
    for out_dtype in DT.values():
        check4(x, w, offsets_of(sizes), randn(gen(2), rows, N, dtype=out_dtype))
    out = int4.matmul(x, w, offsets_of(sizes))
    for _ in range(3):
        assert torch.equal(int4.matmul(x, w, offsets_of(sizes)), out)
    x[7] = float("nan")
    bad = int4.matmul(x, w, offsets_of(sizes))
    keep = [r for r in range(rows) if r != 7]
    assert torch.isnan(bad[7]).all() and torch.equal(bad[keep], out[keep])
