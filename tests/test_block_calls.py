"""How Python reaches the block operators: what the C module refuses and how it
calls the library."""
import pytest
import torch

from sparse_moe_expert_02_gb300 import mx
from test_block_host import Stub, stub_mx


@pytest.mark.parametrize("err", [Stub(1, dtype=torch.int32), Stub(3, dtype=torch.int32), Stub(0, dtype=torch.int32), Stub(4),
                                 Stub(4, dtype=torch.int64), Stub(16, dtype=torch.uint8), Stub(4, dtype=torch.int32, stride=(2,)),
                                 torch.zeros(4, dtype=torch.int32)])
def test_product_refuses_an_error_word_it_would_write_past(err):
    with pytest.raises(ValueError):
        mx.matmul(stub_mx(4), stub_mx(8), out=Stub(4, 8), err=err)


@pytest.mark.gpu
def test_product_takes_an_error_word():
    a, b = (mx.quantize(torch.randn(n, 96, device="cuda")) for n in (5, 7))
    word = torch.zeros(6, dtype=torch.int32, device="cuda")
    assert torch.equal(mx.matmul(a, b, err=word[:4]), mx.matmul(a, b))
    mx.matmul(a, b, err=word)
    assert not word.any()
