"""4-bit products of a few rows whose result is no finite number: NaN where the
row or the feature's scales hold one, what the products say where a group's sum
overflows before its scale, and neither takes a call out of proportion."""
import pytest
import torch

import product_ref as R
from sparse_moe_expert_02_gb300 import int4
from test_products import DT, gen, offsets_of, randn, weights4

pytestmark = pytest.mark.gpu


def microseconds(f):
    for _ in range(3):
        f()
    t = []
    for _ in range(5):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        f()
        end.record()
        torch.cuda.synchronize()
        t.append(begin.elapsed_time(end) * 1e3)
    return sorted(t)[2]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,N,K,group", [(64, 1024, 4096, 64), (64, 1024, 4064, 128), (128, 1024, 1024, 128)])
@pytest.mark.parametrize("where", ["all", "first", "last", "scale"])
def test_nan_rows(G, N, K, group, dtype, where):
    """The call takes at most five times that of finite rows (30 times, where each result was summed again)."""
    sizes = [(3 * i) % 4 for i in range(G)]
    rows = sum(sizes)
    w = weights4(G, N, K, group, True, "bf16")
    x = randn(gen(1), rows, K, dtype=DT[dtype])
    at = offsets_of(sizes)
    clean = int4.matmul(x, w, at)
    usual = microseconds(lambda: int4.matmul(x, w, at, out=clean))
    bad = torch.zeros((rows, N), dtype=torch.bool, device="cuda")
    if where == "scale":
        w.scales[:, 5, -1] = float("nan")
        bad[:, 5] = True
    else:
        hit = slice(None) if where == "all" else slice(0, rows, 3)
        x[hit, {"all": slice(None), "first": 0, "last": K - 1}[where]] = float("nan")
        bad[hit] = True
    got = int4.matmul(x, w, at)
    assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], clean[~bad])
    assert microseconds(lambda: int4.matmul(x, w, at, out=got)) <= 5 * max(usual, 20)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,group", [(40, 256, 128), (24, 160, 64), (64, 1024, 32)])
def test_sums_that_overflow_before_their_scale(N, K, group, dtype):
    """Rows of large numbers and small scales: finite results; infinities where the row holds one; NaN beside them."""
    G, rows = 3, 9
    w = weights4(G, N, K, group, True, "f32")
    w.scales.mul_(1e-3)
    x = randn(gen(2), rows, K, dtype=DT[dtype]).abs()
    x[::2] *= 3e37
    x[4, 3], x[5, 7], x[6, 9] = float("inf"), float("nan"), float("-inf")
    x[6, 10] = float("inf")
    out = torch.zeros((rows, N), device="cuda")
    at = offsets_of([4, 0, 5])
    int4.matmul(x, w, at, out=out)
    v = torch.stack([R.int4_values(w.codes[g], w.scales[g], w.zeros[g], group) for g in range(G)])
    R.close(out, *R.product("fwd", x, v, R.ranges(at.tolist(), rows), torch.zeros_like(out), out.dtype))
    assert torch.isfinite(out[0]).all() and out[0].abs().max() > 1e36
