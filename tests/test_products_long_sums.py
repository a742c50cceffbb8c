"""Sums that take longer than a device wait may: a gradient of the weights over
all rows of one group, which one block sums (the other groups' blocks have
nothing to do)."""
import pytest
import torch

from sparse_moe_expert_02_gb300 import grouped

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,rows", [(9, 9, 260_000_003), (8, 8, 650_000_001)])
def test_dw_of_one_long_group(N, K, rows):
    """Rows of -1, 0 and 1: partial sums stay below 2^24, so the result is the exact one."""
    G, group = 80, 33
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    x, dy = (torch.empty((rows, c), dtype=torch.bfloat16, device="cuda") for c in (K, N))
    ref, step = torch.zeros((N, K), dtype=torch.float64, device="cuda"), 1 << 23
    for a in range(0, rows, step):
        b = min(rows, a + step)
        for t in (x, dy):
            t[a:b] = torch.randint(-1, 2, (b - a, t.shape[1]), generator=g, device="cuda", dtype=torch.int8)
        ref += dy[a:b].double().mT @ x[a:b].double()
    at = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    at[group + 1:] = rows
    word = torch.zeros(4, dtype=torch.int32, device="cuda")
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    got = grouped.matmul_dw(dy, x, at, out_dtype=torch.float32, err=word)
    end.record()
    assert not word.any() and torch.equal(got[group].double(), ref)
    assert not got[:group].any() and not got[group + 1:].any()
    print(f"{rows} rows: {begin.elapsed_time(end):.0f} ms")
