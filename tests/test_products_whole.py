"""The experts' products of numbers whose sums 32 bits hold without a rounding,
in whatever order they are summed: the outputs have to equal the 64-bit ones.  A
column left out, taken twice or put in another's place shows, and so does a
weight rounded where it is to be multiplied as it is.

Rows are -1, 0 or 1.  4-bit values are (code - zero) scale, |code - zero| <= 15,
scale 1 + i/128: multiples of 2^-7 below 30, so sums of up to 2^12 of them stay
below 2^17 and take 24 bits at most.  Where many rows let the values be rounded
to bf16, scales are 1, 2 or 4 and the values whole numbers up to 60.  Weights
and gradients of the wide products are whole numbers up to 3."""
import pytest
import torch

import product_ref as R
from sparse_moe_expert_02_gb300 import grouped, int4

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def draw(seed, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=torch.Generator().manual_seed(seed))


def rows_of(seed, *shape, dtype=torch.bfloat16):
    return draw(seed, -1, 1, *shape).to(dtype)


def weights(G, N, K, group, zeros, scale, whole, seed=0):
    """(codes, scales, zeros) on the CPU."""
    nb = -(-K // group)
    s = 2.0 ** draw(seed + 1, 0, 2, G, N, nb) if whole else 1 + draw(seed + 1, 0, 127, G, N, nb) / 128
    z = draw(seed + 2, 0, 15, G, N, nb).to(torch.uint8) if zeros else None
    return draw(seed, 0, 255, G, N, K // 2).to(torch.uint8), s.to(DT[scale]), z


def values(codes, scales, zeros, group):
    return torch.stack([R.int4_values(codes[g], scales[g], None if zeros is None else zeros[g], group) for g in range(codes.shape[0])])


def by_group(x, v, sizes):
    at = torch.tensor([0] + sizes).cumsum(0).tolist()
    return torch.cat([x[a:b] @ v[g].mT for g, (a, b) in enumerate(zip(at, at[1:]))])


def test_a_planted_mistake_shows():
    """On the CPU, in the definition: weights rounded to bf16, and a column left out."""
    x = rows_of(5, 40, 1024).double()
    for group, zeros, scale in ((128, False, "bf16"), (32, True, "f32")):
        v = values(*weights(1, 64, 1024, group, zeros, scale, False), group)[0]
        ref = x @ v.mT
        assert torch.equal(ref, ref.float().double()) and torch.equal(ref, (x.float() @ v.float().mT).double())
        assert ((x @ v.bfloat16().double().mT) != ref).any(1).all()
        keep = torch.ones(1024, dtype=torch.bool)
        keep[777] = False
        hit = x[:, 777] != 0
        assert ((x[:, keep] @ v[:, keep].mT) != ref)[hit].any(1).all()


def offsets_of(sizes, before=0):
    return (torch.tensor([0] + sizes).cumsum(0) + before).int().cuda()


def shifted(t, by):
    """t on the GPU, at an address by elements off an aligned one."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
    buf[by:].copy_(t.flatten())
    return buf[by:].view(t.shape)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group,zeros,scale", [(128, False, "bf16"), (64, True, "bf16"), (32, True, "f32"), (128, True, "f32"), (32, False, "bf16")])
@pytest.mark.parametrize("sizes,N,K", [
    ([1], 4096, 4096), ([31], 40, 2048), ([32], 648, 1184), ([7], 200, 288), ([(3 * i) % 9 for i in range(40)], 1004, 1280),
    ([(5 * i) % 11 for i in range(128)], 1024, 1024), ([(5 * i) % 11 for i in range(100)], 1024, 384), ([(5 * i) % 11 for i in range(200)], 960, 128),
    ([(5 * i) % 11 for i in range(100)], 1000, 896), ([3, 0, 17, 1], 72, 4096)])
def test_int4_of_few_rows(sizes, N, K, group, zeros, scale, dtype):
    rows, G = sum(sizes), len(sizes)
    assert rows <= max(32, 8 * G)
    c, s, z = weights(G, N, K, group, zeros, scale, False)
    x = rows_of(9, rows, K, dtype=DT[dtype])
    ref = by_group(x.double(), values(c, s, z, group), sizes).float()
    w = int4.I4Tensor(c.cuda(), s.cuda(), None if z is None else z.cuda(), K, group)
    assert torch.equal(int4.matmul(x.cuda(), w, offsets_of(sizes), out_dtype=torch.float32).cpu(), ref)
    # addresses that rule out copies in bulk: of rows, or of scales and zero points
    assert torch.equal(int4.matmul(shifted(x, 1), w, offsets_of(sizes), out_dtype=torch.float32).cpu(), ref)
    w = int4.I4Tensor(c.cuda(), shifted(s, 1), None if z is None else shifted(z, 3), K, group)
    assert torch.equal(int4.matmul(x.cuda(), w, offsets_of(sizes), out_dtype=torch.float32).cpu(), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("group,zeros,scale", [(128, False, "bf16"), (64, True, "bf16"), (32, True, "f32")])
@pytest.mark.parametrize("sizes,N,K", [([33], 136, 96), ([700], 648, 1184), ([2047], 520, 416), ([5, 0, 300, 1, 77], 1000, 2048), ([90] * 7, 4096, 160)])
def test_int4_of_many_rows(sizes, N, K, group, zeros, scale):
    rows, G = sum(sizes), len(sizes)
    assert rows > max(32, 8 * G)
    c, s, z = weights(G, N, K, group, zeros, scale, True)
    x = rows_of(9, rows, K)
    ref = by_group(x.double(), values(c, s, z, group), sizes).float()
    w = int4.I4Tensor(c.cuda(), s.cuda(), None if z is None else z.cuda(), K, group)
    for rows_at in (x.cuda(), shifted(x, 1)):
        assert torch.equal(int4.matmul(rows_at, w, offsets_of(sizes), out_dtype=torch.float32).cpu(), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,N,K", [
    ([13], 1024, 4096), ([2, 0, 3, 1, 7], 1024, 2048), ([5, 9], 520, 1000), ([77, 0, 130], 129, 257), ([700, 20, 0, 333], 1024, 320),
    ([1200, 1801], 640, 2304), ([999], 255, 1031), ([64] * 40, 136, 1024)])
def test_wide_products(sizes, N, K, dtype):
    rows, G, dt = sum(sizes), len(sizes), DT[dtype]
    x, dy, w = rows_of(1, rows, K), draw(2, -3, 3, rows, N), draw(3, -3, 3, G, N, K)
    at = offsets_of(sizes)
    put = lambda t: t.to(dt).cuda()
    got = grouped.matmul(put(x), put(w), at, out_dtype=torch.float32)
    assert torch.equal(got.cpu(), by_group(x.double(), w.double(), sizes).float())
    got = grouped.matmul_dx(put(dy), put(w), at, out_dtype=torch.float32)
    assert torch.equal(got.cpu(), by_group(dy.double(), w.double().mT, sizes).float())
    first = torch.tensor([0] + sizes).cumsum(0).tolist()
    ref = torch.stack([dy[a:b].double().mT @ x[a:b].double() for a, b in zip(first, first[1:])]).float()
    got = grouped.matmul_dw(put(dy), put(x), at, out_dtype=torch.float32)
    assert torch.equal(got.cpu(), ref)
    grouped.matmul_dw(put(dy), put(x), at, out=got, accumulate=True)
    assert torch.equal(got.cpu(), 2 * ref)
