"""The experts' products behind kernels that write what they read: every input
(rows, offsets, codes, scales, zero points, weights, gradients) is overwritten
by the library's own kernels right before the product, on one stream and without
a wait of the host, over the same memory again and again."""
import pytest
import torch

from sparse_moe_expert_02_gb300 import _lib as L, grouped, int4
from test_products import DT, gen, randn

pytestmark = pytest.mark.gpu

ROUNDS = 12


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K", [(9, 256), (9, 160), (150, 256), (150, 161)])
def test_products_behind_the_kernels_that_write_their_inputs(dtype, T, K):
    E, k, N, group = 6, 3, 72, 32
    rows, coded, dt = T * k, K % 32 == 0, DT[dtype]
    g = gen(T + K)
    gates, ups = [randn(g, rows, K, dtype=dt) for _ in range(ROUNDS)], [randn(g, rows, K, dtype=dt) for _ in range(ROUNDS)]
    ws, dys = [randn(g, E, N, K, dtype=dt, std=K ** -0.5) for _ in range(ROUNDS)], [randn(g, rows, N, dtype=dt) for _ in range(ROUNDS)]
    idx = [torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(i * T + t))[:k] for t in range(T)]).int().cuda() for i in range(ROUNDS)]
    counts, offsets, tiles = (torch.empty(E + n, dtype=torch.int32, device="cuda") for n in (1, 2, 2))
    inv, src = torch.empty(T * k, dtype=torch.int32, device="cuda"), torch.empty(T * k + T, dtype=torch.int32, device="cuda")
    x, w, q = torch.empty((rows, K), dtype=dt, device="cuda"), torch.empty((E, N, K), dtype=dt, device="cuda"), None
    dy = torch.empty((rows, N), dtype=dt, device="cuda")
    if coded:
        q = int4.empty((E, N), K, group, True)

    def inputs(i):
        assert L.moe_permute_index_noalloc(idx[i], T, E, k, counts, offsets, tiles, inv, src) == 0
        grouped.swiglu(gates[i], ups[i], out=x)
        grouped.swiglu(dys[i], dys[i], out=dy)
        if coded:
            int4.quantize(ws[i], out=q)
            int4.dequantize(q, out=w)
        else:
            w.copy_(ws[i])

    def products():
        at = offsets[:E + 1]
        got = [grouped.matmul(x, w, at), grouped.matmul_dx(dy, w, at), grouped.matmul_dw(dy, x, at)]
        return got + [int4.matmul(x, q, at)] if coded else got

    want = []
    for i in range(ROUNDS):
        inputs(i)
        torch.cuda.synchronize()
        want.append(products())
        torch.cuda.synchronize()
    got = []
    for i in range(ROUNDS):
        inputs(i)
        got.append(products())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
    assert not any(torch.equal(a, b) for x, y in zip(want, want[1:]) for a, b in zip(x, y))
