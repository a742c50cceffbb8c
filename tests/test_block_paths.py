"""Paths of the block operators that small sizes do not reach, against the same
64-bit definitions and with the tolerances of test_block_ops."""
import pytest
import torch

from sparse_moe_expert_02_gb300 import MoEBlock, MoELayer, norm
from test_block_ops import BF16, few_case, few_check, rand

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
