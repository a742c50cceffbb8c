"""Paths of the block operators that small sizes do not reach, against the same
64-bit definitions and with the tolerances of test_block_ops."""
import pytest
import torch

from sparse_moe_expert_02_gb300 import MoELayer
from test_block_ops import few_case, few_check

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
