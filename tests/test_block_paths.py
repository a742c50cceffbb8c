"""Paths of the block operators that small sizes do not reach, against the same
64-bit definitions and with the tolerances of test_block_ops."""
import pytest
import torch

from test_block_ops import few_case, few_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,T", [(43136, 2), (49152, 5)])
def test_few_takes_rows_too_wide_for_shared_memory(D, T):
    shape, inp, layer = few_case("f32", T, D, 4, 64, 2, None)
    out = layer.forward_few(inp["x"])
    layer.check()
    few_check("f32", shape, inp, layer, out)
    assert torch.equal(out, layer.forward(inp["x"]))
