"""Host side of the experts' products (no GPU): argument checks of the C entry
points and of the Python functions, and the tests' own 64-bit definitions."""
import ctypes
import importlib.util
import shutil

import pytest
import torch

import product_ref as R
from sparse_moe_expert_02_gb300 import _lib as L, grouped, int4
from test_block_host import Stub as BlockStub

OK, INVALID, UNSUPPORTED = L.MOE_OK, L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(G=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(offsets=0, G=2), INVALID),
    (dict(G=1026), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(K=(1 << 20) + 1, ld_x=1 << 21), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(out_dtype=3), UNSUPPORTED), (dict(x=0), INVALID),
    (dict(x=18), INVALID), (dict(w=2), INVALID), (dict(ld_x=7), INVALID), (dict(out=0), INVALID), (dict(ld_out=11), INVALID),
    (dict(offsets=6), INVALID), (dict(err=6), INVALID), (dict(rows=0, x=0, w=0, out=0), OK)])
def test_grouped_gemm_checks_before_any_launch(change, status):
    a = dict(x=16, ld_x=8, w=16, dtype=0, offsets=4, rows=3, G=1, N=12, K=8, out=16, out_dtype=0, ld_out=12, err=0) | change
    assert L.lib().moe_grouped_gemm(*a.values(), None) == status
    if not {"ld_x", "ld_out"} & set(change):
        b = a | dict(ld_x=12, ld_out=8)
        assert L.lib().moe_grouped_gemm_dx(*b.values(), None) == status


def test_the_gradients_row_strides_are_checked():
    a = dict(dy=16, ld=12, w=16, dtype=0, offsets=4, rows=3, G=1, N=12, K=8, out=16, out_dtype=0, ld_out=8, err=0)
    assert L.lib().moe_grouped_gemm_dx(*(a | dict(ld=11)).values(), None) == INVALID
    assert L.lib().moe_grouped_gemm_dx(*(a | dict(ld_out=7)).values(), None) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(G=2, offsets=0), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(out_dtype=2), UNSUPPORTED),
    (dict(dy=0), INVALID), (dict(x=0), INVALID), (dict(ld_dy=11), INVALID), (dict(ld_x=7), INVALID), (dict(dw=0), INVALID),
    (dict(dw=0, rows=0), INVALID), (dict(dw=18), INVALID), (dict(err=2), INVALID), (dict(K=0), INVALID)])
def test_grouped_gemm_dw_checks_before_any_launch(change, status):
    a = dict(dy=16, ld_dy=12, x=16, ld_x=8, dtype=0, offsets=4, rows=3, G=1, N=12, K=8, dw=16, out_dtype=0, accumulate=0, err=0) | change
    assert L.lib().moe_grouped_gemm_dw(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(I=0), INVALID), (dict(I=(1 << 20) + 1), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(gate=0), INVALID),
    (dict(ld_up=7), INVALID), (dict(weight=2), INVALID), (dict(out=18), INVALID), (dict(out_dtype=5), UNSUPPORTED), (dict(ld_out=7), INVALID),
    (dict(rows=0, gate=0, up=0, out=0), OK)])
def test_swiglu_checks_before_any_launch(change, status):
    a = dict(gate=16, ld_gate=8, up=16, ld_up=8, dtype=0, weight=0, rows=3, I=8, out=16, out_dtype=0, ld_out=8) | change
    assert L.lib().moe_swiglu(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(dh=0), INVALID), (dict(ld_dgate=7), INVALID), (dict(dup=0), INVALID),
    (dict(dweight=6), INVALID), (dict(weight=6), INVALID), (dict(rows=0, dh=0, dup=0), OK)])
def test_swiglu_grad_checks_before_any_launch(change, status):
    a = dict(dh=16, ld_dh=8, gate=16, ld_gate=8, up=16, ld_up=8, dtype=0, weight=0, rows=3, I=8, dgate=16, ld_dgate=8, dup=16, ld_dup=8,
             dweight=0) | change
    assert L.lib().moe_swiglu_grad(*a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVALID), (dict(K=48), UNSUPPORTED), (dict(K=0), INVALID), (dict(group=16), UNSUPPORTED), (dict(group=0), UNSUPPORTED),
    (dict(scale_dtype=2), UNSUPPORTED), (dict(codes=8), INVALID), (dict(scales=0), INVALID), (dict(scales=18), INVALID), (dict(x=0), INVALID),
    (dict(ld_x=63), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(ld_out=7), INVALID), (dict(G=2, offsets=0), INVALID), (dict(err=6), INVALID),
    (dict(rows=0, x=0, codes=0, scales=0, out=0), OK)])
def test_int4_gemm_checks_before_any_launch(change, status):
    a = dict(x=16, dtype=0, ld_x=64, codes=16, scales=16, scale_dtype=0, zeros=0, group=32, offsets=4, rows=3, G=1, N=8, K=64, out=16,
             out_dtype=0, ld_out=8, err=0) | change
    assert L.lib().moe_int4_gemm(*a.values(), None) == status


def test_int4_quantize_checks_before_any_launch():
    lib = L.lib()
    q = dict(x=16, dtype=0, ld=64, rows=3, cols=64, group=32, codes=16, scales=16, scale_dtype=0, zeros=0)
    for change, status in ((dict(rows=-1), INVALID), (dict(cols=40), UNSUPPORTED), (dict(ld=63), INVALID), (dict(dtype=3), UNSUPPORTED),
                           (dict(codes=0), INVALID), (dict(group=256), UNSUPPORTED), (dict(rows=0, x=0, codes=0), OK)):
        assert lib.moe_int4_quantize(*(q | change).values(), None) == status
    d = dict(codes=16, scales=16, scale_dtype=0, zeros=0, group=32, rows=3, cols=64, out=16, out_dtype=0, ld=64)
    for change, status in ((dict(rows=-1), INVALID), (dict(cols=40), UNSUPPORTED), (dict(ld=63), INVALID), (dict(out_dtype=3), UNSUPPORTED),
                           (dict(scales=0), INVALID), (dict(rows=0, out=0, codes=0), OK)):
        assert lib.moe_int4_dequantize(*(d | change).values(), None) == status


class Stub(BlockStub):
    """A tensor of the current device, or of another one."""

    def __init__(self, *shape, dtype=torch.float32, stride=None, device=0):
        super().__init__(*shape, dtype=dtype, stride=stride)
        self.index = device

    def get_device(self):
        return self.index


@pytest.fixture(autouse=True)
def device_zero(monkeypatch, tmp_path):
    """The module asks torch for the current device, which needs a GPU: a copy of it that is told."""
    if torch.cuda.is_available():
        return
    L.lib()
    copy = shutil.copy(L._build.FAST, tmp_path)
    spec = importlib.util.spec_from_file_location("_fastcall", copy)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    lib = L.lib()
    at = lambda *names: tuple(ctypes.cast(getattr(lib, "moe_" + n), ctypes.c_void_p).value for n in names)
    m.init((torch.float32, torch.bfloat16, torch.uint8, torch.int32), lambda: 0, lambda device: 0,
           at("norm_pre", "norm_post", "mx_quantize", "mx_dequantize", "mx_gemm"),
           at("grouped_gemm", "grouped_gemm_dx", "grouped_gemm_dw", "swiglu", "swiglu_grad", "int4_quantize", "int4_dequantize", "int4_gemm"))
    monkeypatch.setattr(L, "_fast", m)


def I32(*shape):
    return Stub(*shape, dtype=torch.int32)


def stub4(*lead, cols=64, group=32, zeros=True, scale=torch.float32):
    nb = -(-cols // group)
    return int4.I4Tensor(torch.empty(*lead, cols // 2, dtype=torch.uint8), torch.empty(*lead, nb, dtype=scale),
                         torch.empty(*lead, nb, dtype=torch.uint8) if zeros else None, cols, group)


def as_stub(q):
    q.codes, q.scales = Stub(*q.codes.shape, dtype=torch.uint8), Stub(*q.scales.shape, dtype=q.scales.dtype)
    if q.zeros is not None:
        q.zeros = Stub(*q.zeros.shape, dtype=torch.uint8)
    return q


def test_products_refuse_before_any_launch():
    x, w, out, at = Stub(6, 8), Stub(3, 5, 8), Stub(6, 5), I32(4)
    dy = Stub(6, 5)
    bf = torch.bfloat16
    for bad in (lambda: grouped.matmul(torch.zeros(6, 8), w, at, out=out), lambda: grouped.matmul(Stub(6, 7), w, at, out=out),
                lambda: grouped.matmul(x, w, None, out=out), lambda: grouped.matmul(x, w, I32(3), out=out),
                lambda: grouped.matmul(x, w, Stub(4), out=out), lambda: grouped.matmul(x, w, Stub(4, dtype=torch.int64), out=out),
                lambda: grouped.matmul(x, w, I32(2, 2), out=out), lambda: grouped.matmul(x, w, at, out=Stub(5, 5)),
                lambda: grouped.matmul(x, w, at, out=Stub(6, 6)), lambda: grouped.matmul(x, Stub(3, 5, 8, dtype=bf), at, out=out),
                lambda: grouped.matmul(Stub(6, 8, dtype=torch.float16), w, at, out=out), lambda: grouped.matmul(Stub(6, 8, stride=(16, 2)), w, at, out=out),
                lambda: grouped.matmul(x, Stub(3, 5, 8, stride=(80, 16, 1)), at, out=out), lambda: grouped.matmul(x, Stub(8), at, out=out),
                lambda: grouped.matmul(x, w, at, out=out, err=I32(3)), lambda: grouped.matmul(x, w, at, out=out, err=Stub(4)),
                lambda: grouped.matmul(x, w, at, out=Stub(6, 5, device=1)), lambda: grouped.matmul(x, Stub(3, 5, 8, device=1), at, out=out),
                lambda: grouped.matmul(x, w, Stub(4, dtype=torch.int32, device=1), out=out),
                lambda: grouped.matmul_dx(dy, w, at, out=out), lambda: grouped.matmul_dx(x, w, at, out=x),
                lambda: grouped.matmul_dw(dy, x, at, out=Stub(2, 5, 8)), lambda: grouped.matmul_dw(dy, x, at, out=Stub(3, 8, 5)),
                lambda: grouped.matmul_dw(dy, x, None, out=Stub(3, 5, 8)), lambda: grouped.matmul_dw(Stub(5, 5), x, at, out=w),
                lambda: grouped.matmul_dw(Stub(6, 5, dtype=bf), x, at, out=w), lambda: grouped.matmul_dw(dy, x, at, accumulate=True),
                lambda: grouped.matmul_dw(dy, x, at, out=Stub(3, 5, 8, dtype=torch.float16)),
                lambda: grouped.matmul_dw(dy, Stub(6, 8, device=1), at, out=w)):
        with pytest.raises(ValueError):
            bad()


def test_rows_that_lie_over_one_another_are_refused():
    x, w = Stub(6, 8, stride=(0, 1)), Stub(1, 5, 8)
    with pytest.raises(L.MoEError):
        grouped.matmul(x, w, None, out=Stub(6, 5))
    with pytest.raises(L.MoEError):
        grouped.matmul(Stub(6, 8), w, None, out=Stub(6, 5, stride=(4, 1)))


def test_activation_refuses_before_any_launch():
    x, w = Stub(6, 8), Stub(6)
    for bad in (lambda: grouped.swiglu(x, Stub(6, 7), out=x), lambda: grouped.swiglu(x, Stub(6, 8, dtype=torch.bfloat16), out=x),
                lambda: grouped.swiglu(x, x, Stub(5), out=x), lambda: grouped.swiglu(x, x, Stub(6, dtype=torch.bfloat16), out=x),
                lambda: grouped.swiglu(x, x, Stub(6, stride=(2,)), out=x), lambda: grouped.swiglu(x, x, out=Stub(5, 8)),
                lambda: grouped.swiglu(x, x, out=Stub(6, 8, dtype=torch.float16)), lambda: grouped.swiglu(x, x, out=Stub(6, 8, device=2)),
                lambda: grouped.swiglu_grad(Stub(6, 7), x, x, w, x, x, w), lambda: grouped.swiglu_grad(x, x, x, w, x, x, Stub(7)),
                lambda: grouped.swiglu_grad(x, x, x, w, Stub(6, 8, dtype=torch.bfloat16), x, w),
                lambda: grouped.swiglu_grad(Stub(6, 8, dtype=torch.bfloat16), x, x, w, x, x, w),
                lambda: grouped.swiglu_grad(x, x, x, w, x, x, Stub(6, device=1))):
        with pytest.raises(ValueError):
            bad()


def test_int4_refuses_before_any_launch():
    u8 = torch.uint8
    for bad in (lambda: stub4(5, cols=48), lambda: stub4(5, group=16), lambda: stub4(5, scale=torch.float16),
                lambda: int4.I4Tensor(torch.empty(5, 32, dtype=u8), torch.empty(5, 3), None, 64, 32),
                lambda: int4.I4Tensor(torch.empty(5, 32, dtype=u8), torch.empty(4, 2), None, 64, 32),
                lambda: int4.I4Tensor(torch.empty(5, 32, dtype=torch.int8), torch.empty(5, 2), None, 64, 32),
                lambda: int4.I4Tensor(torch.empty(5, 32, dtype=u8), torch.empty(5, 2), torch.empty(5, 2), 64, 32),
                lambda: int4.I4Tensor(torch.empty(5, 32, dtype=u8), torch.empty(5, 2), torch.empty(5, 1, dtype=u8), 64, 32),
                lambda: int4.I4Tensor(torch.empty(32, dtype=u8), torch.empty(2), None, 64, 32)):
        with pytest.raises(ValueError):
            bad()
    w, x, at = as_stub(stub4(3, 5)), Stub(6, 64), I32(4)
    other = as_stub(stub4(3, 5))
    other.scales = Stub(3, 5, 2, device=1)
    for bad in (lambda: int4.matmul(Stub(6, 32), w, at, out=Stub(6, 5)), lambda: int4.matmul(x, w, None, out=Stub(6, 5)),
                lambda: int4.matmul(x, w, I32(3), out=Stub(6, 5)), lambda: int4.matmul(x, w, at, out=Stub(6, 4)),
                lambda: int4.matmul(x, w, at, out=Stub(5, 5)), lambda: int4.matmul(Stub(6, 64, dtype=torch.float16), w, at, out=Stub(6, 5)),
                lambda: int4.matmul(x, as_stub(stub4(2, 3, 5)), at, out=Stub(6, 5)), lambda: int4.matmul(x, other, at, out=Stub(6, 5)),
                lambda: int4.quantize(Stub(5, 96), out=as_stub(stub4(5))), lambda: int4.quantize(Stub(4, 64), out=as_stub(stub4(5))),
                lambda: int4.dequantize(as_stub(stub4(5)), out=Stub(5, 32)),
                lambda: int4.dequantize(as_stub(stub4(5)), out=Stub(5, 64, device=1))):
        with pytest.raises(ValueError):
            bad()


def test_the_definitions_by_hand():
    x = torch.tensor([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    w = torch.tensor([[[1.0, 0.0], [0.0, 1.0], [1.0, 1.0]], [[2.0, 0.0], [0.0, 2.0], [0.0, 0.0]]])
    held = torch.full((3, 3), -1.0)
    ref, _ = R.product("fwd", x, w, R.ranges([0, 1, 2], 3), held, torch.float32)
    assert ref.tolist() == [[1, 2, 3], [6, 8, 0], [-1, -1, -1]]
    dy = torch.tensor([[1.0, 1.0, 1.0], [1.0, 2.0, 3.0], [9.0, 9.0, 9.0]])
    assert R.product("dx", dy, w, R.ranges([0, 1, 2], 3), held[:, :2], torch.float32)[0].tolist() == [[2, 2], [2, 4], [-1, -1]]
    dw, _ = R.product("dw", dy, x, R.ranges([0, 2, 2], 3), torch.zeros(2, 3, 2), torch.float32)
    assert dw[0].tolist() == [[4, 6], [7, 10], [10, 14]] and not dw[1].any()
    assert R.ranges([-4, 2, 1, 99], 5) == [(0, 2), (2, 2), (1, 5)]
    assert R.int4_values(torch.tensor([[0x98, 0x0F]], dtype=torch.uint8), torch.tensor([[0.5]]), None, 32).tolist() == [[0, 0.5, 3.5, -4]]
    q, s, z = R.int4_quantize(torch.tensor([[7.0, -3.5, 0.5, 1.5] + [0.0] * 28]), 32, False, torch.float32)
    assert s.item() == 1.0 and q[0, :2].tolist() == [0x4F, 0xA8]
