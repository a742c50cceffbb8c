"""Host side of the block operators (no GPU): packed structs, argument checks
of the C entry points, and the 64-bit definitions the GPU tests use."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import block_ref as R
from sparse_moe_expert_02_gb300 import _lib as L, mx, norm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_packed_structs_match_the_header(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe.h"\n'
                   'int main(void) { printf("%zu %zu %zu %zu %zu %zu %zu\\n", sizeof(moe_norm), sizeof(moe_post), '
                   'offsetof(moe_norm, w), offsetof(moe_post, res_scale), offsetof(moe_post, gate), '
                   'offsetof(moe_post, ld_gate), sizeof(moe_ws_layout)); return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [L.NORM_STRUCT.size, L.POST_STRUCT.size, 16, 64, 88, 96, ctypes.sizeof(L.moe_ws_layout)]


def pack_norm(kind=1, eps=1e-6, off=0.0, dt=0, w=0, b=0):
    return L.NORM_STRUCT.pack(kind, eps, off, dt, w, b)


@pytest.mark.parametrize("norm,args,status", [
    (None, (16, 0, 64, 2, 64, 16, 0, 64), L.MOE_ERR_INVALID_ARG),
    (pack_norm(kind=5), (16, 0, 64, 2, 64, 16, 0, 64), L.MOE_ERR_INVALID_ARG),
    (pack_norm(eps=-1.0), (16, 0, 64, 2, 64, 16, 0, 64), L.MOE_ERR_INVALID_ARG),
    (pack_norm(dt=2, w=16), (16, 0, 64, 2, 64, 16, 0, 64), L.MOE_ERR_UNSUPPORTED),
    (pack_norm(w=18), (16, 0, 64, 2, 64, 16, 0, 64), L.MOE_ERR_INVALID_ARG),
    (pack_norm(), (16, 2, 64, 2, 64, 16, 0, 64), L.MOE_ERR_UNSUPPORTED),
    (pack_norm(), (16, 0, 64, 2, 64, 16, 7, 64), L.MOE_ERR_UNSUPPORTED),
    (pack_norm(), (0, 0, 64, 2, 64, 16, 0, 64), L.MOE_ERR_INVALID_ARG),
    (pack_norm(), (16, 0, 63, 2, 64, 16, 0, 64), L.MOE_ERR_INVALID_ARG),
    (pack_norm(), (18, 0, 64, 2, 64, 16, 0, 64), L.MOE_ERR_INVALID_ARG),
    (pack_norm(), (16, 0, 64, -1, 64, 16, 0, 64), L.MOE_ERR_INVALID_ARG),
    (pack_norm(), (16, 0, 64, 2, 0, 16, 0, 64), L.MOE_ERR_INVALID_ARG),
    (pack_norm(), (16, 0, 16385, 2, 16385, 16, 0, 16385), L.MOE_ERR_UNSUPPORTED),
    (pack_norm(), (0, 0, 64, 0, 64, 0, 0, 64), L.MOE_OK),
])
def test_norm_pre_checks_before_any_launch(norm, args, status):
    assert L.lib().moe_norm_pre(norm, *args, None) == status


def pack_post(norm=(1, 1e-6, 0.0, 0, 0, 0), nxt=(0, 0.0, 0.0, 0, 0, 0), by=0, gd=0, gate=0, gl=0):
    return L.POST_STRUCT.pack(*norm, *nxt, 1.0, 1.0, by, gd, 0, gate, gl)


@pytest.mark.parametrize("post,change,status", [
    (pack_post(by=9), {}, L.MOE_ERR_INVALID_ARG),
    (pack_post(by=1, gd=2, gate=16), {}, L.MOE_ERR_UNSUPPORTED),
    (pack_post(by=1), {}, L.MOE_ERR_INVALID_ARG),
    (pack_post(by=3, gate=16, gl=63), {}, L.MOE_ERR_INVALID_ARG),
    (pack_post(nxt=(1, 1e-6, 0.0, 0, 0, 0)), {}, L.MOE_ERR_INVALID_ARG),  # a next norm without next_out
    (pack_post(), dict(res=0), L.MOE_ERR_INVALID_ARG),
    (pack_post(), dict(out=32, ld_out=80), L.MOE_ERR_INVALID_ARG),  # out = res at another stride
    (pack_post(), dict(res_dtype=3), L.MOE_ERR_UNSUPPORTED),
    (pack_post(), dict(T=0), L.MOE_OK),
])
def test_norm_post_checks_before_any_launch(post, change, status):
    a = dict(y=16, dtype=0, ld_y=64, res=32, res_dtype=0, ld_res=64, T=2, D=64, out=48, ld_out=64, next_out=0,
             next_dtype=0, ld_next=0) | change
    assert L.lib().moe_norm_post(post, *a.values(), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), L.MOE_ERR_INVALID_ARG), (dict(G=0), L.MOE_ERR_INVALID_ARG), (dict(K=48), L.MOE_ERR_UNSUPPORTED),
    (dict(offsets=0, G=2), L.MOE_ERR_INVALID_ARG), (dict(G=1026), L.MOE_ERR_UNSUPPORTED), (dict(a=8), L.MOE_ERR_INVALID_ARG),
    (dict(out_dtype=2), L.MOE_ERR_UNSUPPORTED), (dict(ld_out=7), L.MOE_ERR_INVALID_ARG), (dict(b_scale=0), L.MOE_ERR_INVALID_ARG),
    (dict(offsets=6), L.MOE_ERR_INVALID_ARG), (dict(err=6), L.MOE_ERR_INVALID_ARG), (dict(rows=0), L.MOE_OK),
])
def test_mx_gemm_checks_before_any_launch(change, status):
    a = dict(a=16, a_scale=1, b=16, b_scale=1, offsets=4, rows=3, G=1, N=8, K=64, out=16, out_dtype=0, ld_out=8, err=0) | change
    assert L.lib().moe_mx_gemm(*a.values(), None) == status


def test_mx_quantize_checks_before_any_launch():
    lib = L.lib()
    assert lib.moe_mx_quantize(16, 0, 64, -1, 64, 16, 16, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_mx_quantize(16, 2, 64, 1, 64, 16, 16, None) == L.MOE_ERR_UNSUPPORTED
    assert lib.moe_mx_quantize(16, 0, 63, 1, 64, 16, 16, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_mx_quantize(16, 0, 64, 1, 64, 8, 16, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_mx_quantize(0, 0, 64, 0, 64, 0, 0, None) == L.MOE_OK
    assert lib.moe_mx_dequantize(16, 0, 1, 64, 16, 0, 64, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_forward_few(None, None, None, 1, None, None, None, None, 0, None) == L.MOE_ERR_INVALID_ARG


def test_reference_quantiser_rounds_to_the_nearest_code():
    g = np.random.default_rng(0)
    x = g.normal(size=(4, 64)).astype(np.float32)
    q, s = R.mx_quantize(x)
    v = R.mx_values(q, s)
    unit = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, -1)
    grid = np.concatenate([-R.E2M1[::-1], R.E2M1])
    best = np.abs(x[..., None] / unit[..., None] - grid).min(-1)
    assert np.allclose(np.abs(x / unit - v / unit), best)
    assert np.array_equal(R.mx_values(*R.mx_quantize(v.astype(np.float32))), v)  # what is representable stays


class Stub:
    """What the operators read of a device tensor; the address is never used."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.float32, stride=None):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.strides = stride or tuple(int(np.prod(shape[i + 1:])) for i in range(len(shape)))
        self.device = torch.device("cpu")

    def stride(self):
        return self.strides

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return self.strides == tuple(int(np.prod(self.shape[i + 1:])) for i in range(len(self.shape)))

    def data_ptr(self):
        return 4096


def stub_mx(*lead, cols=64):
    t = object.__new__(mx.MXTensor)
    nb = -(-cols // 32)
    t.codes, t.scales, t.cols = Stub(*lead, 16 * nb, dtype=torch.uint8), Stub(*lead, nb, dtype=torch.uint8), cols
    return t


def test_operators_refuse_before_any_launch():
    x, w = Stub(4, 64), Stub(64)
    for bad in (lambda: norm.pre(torch.zeros(4, 64), out=x), lambda: norm.pre(x, out=Stub(4, 65)), lambda: norm.pre(x, out=Stub(5, 64)),
                lambda: norm.pre(Stub(4, 64, dtype=torch.float16), out=x), lambda: norm.pre(Stub(4, 8, 8), out=x),
                lambda: norm.pre(Stub(4, 64, stride=(128, 2)), out=x), lambda: norm.pre(x, Stub(63), out=x),
                lambda: norm.pre(x, Stub(64, stride=(2,)), out=x), lambda: norm.pre(x, w, Stub(64, dtype=torch.bfloat16), out=x),
                lambda: norm.pre(x, w, kind="max", out=x),
                lambda: norm.post(x, Stub(3, 64), out=x), lambda: norm.post(x, x, out=Stub(4, 64, dtype=torch.bfloat16)),
                lambda: norm.post(x, x, out=x, gate=Stub(4)), lambda: norm.post(x, x, out=x, gate=w, gate_by="token"),
                lambda: norm.post(x, x, out=x, gate=Stub(4, 63), gate_by="full"), lambda: norm.post(x, x, out=x, gate=w, gate_by="row"),
                lambda: norm.post(x, x, out=x, next_w=Stub(65), next_out=x), lambda: norm.post(x, x, out=x, next_out=Stub(4, 32)),
                lambda: mx.quantize(x, out=stub_mx(4, cols=96)), lambda: mx.quantize(x, out=stub_mx(3)),
                lambda: mx.quantize(Stub(4, 64, dtype=torch.int32), out=stub_mx(4)),
                lambda: mx.quantize(Stub(2, 4, 64), out=stub_mx(4, 2)),
                lambda: mx.dequantize(stub_mx(4), out=Stub(4, 65)), lambda: mx.dequantize(stub_mx(2, 2), out=Stub(4, 64)),
                lambda: mx.matmul(stub_mx(4), stub_mx(8, cols=96), out=Stub(4, 8)), lambda: mx.matmul(stub_mx(4), stub_mx(8), out=Stub(4, 9)),
                lambda: mx.matmul(stub_mx(4, cols=48), stub_mx(8, cols=48), out=Stub(4, 8)),
                lambda: mx.matmul(stub_mx(2, 4), stub_mx(8), out=Stub(4, 8)), lambda: mx.matmul(stub_mx(4), stub_mx(1, 2, 8), out=Stub(4, 8)),
                lambda: mx.matmul(stub_mx(4), stub_mx(2, 8), offsets=Stub(2, dtype=torch.int32), out=Stub(4, 8)),
                lambda: mx.matmul(stub_mx(4), stub_mx(2, 8), offsets=Stub(3), out=Stub(4, 8))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        L.fast().norm_pre(x, w)
    with pytest.raises(AttributeError):
        norm.pre(x, 3.0, out=x)
