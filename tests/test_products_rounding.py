"""4-bit values in bf16 from fp32 scales are rounded once: scales whose product
with a code lies next to a tie of bf16, so close that 32 bits round it onto the
tie, and a second rounding from there would go to the even neighbour, on the
wrong side or on the right one."""
import pytest
import torch

from sparse_moe_expert_02_gb300 import int4


def nearest_bf16(v):
    """64-bit v (normal) to eight significant bits, ties to even."""
    m, e = torch.frexp(v)
    return torch.ldexp(torch.round(m * 256) / 256, e)


def next_to_ties():
    """(factors d, fp32 scales s): d s rounds in 32 bits to a tie of bf16 that it is not."""
    d = torch.arange(3, 16, dtype=torch.float64)[:, None]
    tie = (torch.arange(128, 256, dtype=torch.float64)[None, :] + 0.5) / 256
    s = (tie / d).float()
    hit = ((s * d.float()).double() == tie) & (s.double() * d != tie)
    return d.expand_as(s)[hit], s[hit]


def test_scales_next_to_ties():
    d, s = next_to_ties()
    v = d * s.double()
    twice, once = v.float().bfloat16().double(), nearest_bf16(v)
    assert d.numel() > 500 and (twice != once).sum() > 200 and (twice == once).sum() > 200
    w = torch.tensor([1.0, -1.00390625, 1.00390625, 1.01171875], dtype=torch.float64)  # ties themselves, to even
    assert nearest_bf16(w).tolist() == [1.0, -1.0, 1.0, 1.015625]


def coded(zeros):
    """[64, 32 n]: groups of 32 columns, codes of +d and -d in turn as far as the zero point allows, and d of all others."""
    d, s = next_to_ties()
    n = s.numel() // 64
    d, s = d[:64 * n].view(64, n).long(), s[:64 * n].view(64, n)
    z = torch.zeros_like(d) if zeros else torch.full_like(d, 8)
    if not zeros:
        d = torch.where(d > 7, -d + 8, d)  # -7 .. 7; those made of others are ordinary values
    codes = (d + z)[:, :, None].expand(64, n, 32).reshape(64, 32 * n).clone()
    codes[:, 5::32] = torch.arange(64)[:, None] % 16
    if zeros:
        z[:, ::2] = 15
        codes.view(64, n, 32)[:, ::2] = 15 - codes.view(64, n, 32)[:, ::2]
    value = (codes.view(64, n, 32) - z[:, :, None]) * s[:, :, None].double()
    packed = (codes[:, 0::2] | codes[:, 1::2] << 4).to(torch.uint8)
    return packed, s, z.to(torch.uint8) if zeros else None, value.view(64, 32 * n)


@pytest.mark.gpu
@pytest.mark.parametrize("zeros", [False, True])
def test_int4_values_are_rounded_once(zeros):
    packed, s, z, value = coded(zeros)
    K = value.shape[1]
    q = int4.I4Tensor(packed.cuda(), s.cuda(), None if z is None else z.cuda(), K, 32)
    want = torch.where(value == 0, value, nearest_bf16(value))
    assert torch.equal(int4.dequantize(q).double().cpu(), want)
    assert torch.equal(int4.dequantize(q, torch.float32).cpu(), value.float())
    # a row that takes one column: what the product of many rows multiplies
    x = torch.eye(K, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(int4.matmul(x, q, out_dtype=torch.float32).double().cpu(), want.mT)
    # and few rows: the values themselves
    assert torch.equal(int4.matmul(x[:32], q, out_dtype=torch.float32).cpu(), value.float().mT[:32])


@pytest.mark.gpu
def test_int4_values_of_infinite_and_of_the_largest_scales():
    s = torch.tensor([[float("inf"), float("nan"), 3.4e38, 2.0 ** -149, 2.0 ** -126, 0.0]])
    codes = torch.arange(192) % 16
    q = int4.I4Tensor((codes[0::2] | codes[1::2] << 4).to(torch.uint8).view(1, 96).cuda(), s.cuda(), None, 192, 32)
    value = ((codes.view(6, 32) - 8) * s.view(6, 1).double()).view(1, 192)
    got, wide = int4.dequantize(q).float().cpu(), int4.dequantize(q, torch.float32).cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(value)) and torch.equal(torch.isnan(wide), torch.isnan(value))
    assert torch.equal(torch.nan_to_num(wide, 1.0), torch.nan_to_num(value.float(), 1.0))
    # (every product here is a number of 32 bits or past their range: one more rounding is the only one)
    assert torch.equal(torch.nan_to_num(got, 1.0), torch.nan_to_num(value.float().bfloat16().float(), 1.0))
