"""How Python reaches the block operators: what the C module refuses and how it
calls the library."""
import ctypes
import importlib.util
import os
import shutil
import subprocess
import sysconfig

import pytest
import torch

from sparse_moe_expert_02_gb300 import _lib as L
from sparse_moe_expert_02_gb300 import build as B
from sparse_moe_expert_02_gb300 import MoELayer, mx
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


def test_the_interpreter_lock_is_free_while_the_library_runs(tmp_path):
    # entry points that report whether they were called with the lock, behind a copy of the module
    fakes = tmp_path / "fakes.c"
    fakes.write_text("#include <Python.h>\nint probe(void) { return PyGILState_Check() ? 99 : 0; }\n")
    so = tmp_path / "fakes.so"
    subprocess.run(["gcc", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"], str(fakes), "-o", str(so)], check=True)
    address = ctypes.cast(ctypes.CDLL(str(so)).probe, ctypes.c_void_p).value
    B.build()
    copy = tmp_path / os.path.basename(B.FAST)
    shutil.copy(B.FAST, copy)
    spec = importlib.util.spec_from_file_location("_fastcall", copy)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.init((torch.float32, torch.bfloat16, torch.uint8, torch.int32), lambda: 0, lambda device: 0, (address,) * 5)
    x, q, b = Stub(4, 64), stub_mx(4), stub_mx(8)
    assert m.norm_pre(x, None, None, 1, 1e-6, 0.0, x) == 0
    assert m.norm_post(x, x, x, None, 1, 1e-6, 0.0, None, None, 0, None, None, 1.0, 1.0, 0, None, False) == 0
    assert m.mx_quantize(x, q.codes, q.scales, 64) == 0
    assert m.mx_dequantize(q.codes, q.scales, 64, x) == 0
    assert m.mx_gemm(q.codes, q.scales, 64, b.codes, b.scales, 64, None, Stub(4, 8), None) == 0


def test_the_library_builds_where_python_has_no_headers(tmp_path, monkeypatch):
    L.lib()  # the real one
    cc = tmp_path / "nvcc"  # makes the file after -o
    cc.write_text('#!/bin/sh\nwhile [ $# -gt 1 ]; do [ "$1" = -o ] && echo made > "$2"; shift; done\n')
    cc.chmod(0o755)
    monkeypatch.setenv("NVCC", str(cc))
    for name in ("BUILD", "LIB", "FAST"):
        monkeypatch.setattr(B, name, str(tmp_path / "b" / os.path.basename(getattr(B, name)) if name != "BUILD" else tmp_path / "b"))
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    with monkeypatch.context() as m:
        m.setattr(B.sysconfig, "get_paths", lambda: paths)
        # a compiler that finds no Python.h
        cc.write_text('#!/bin/sh\ncase "$*" in *fastcall.c*) exit 1;; esac\n' + cc.read_text().split("\n", 1)[1])
        assert B.build() == B.LIB and os.path.exists(B.LIB) and not os.path.exists(B.FAST)
        os.utime(B.LIB, (1, 1))
        B.build()
        assert os.stat(B.LIB).st_mtime == 1  # nothing to do
        m.setattr(L, "_fast", None)
        with pytest.raises(RuntimeError, match="Python.h"):
            mx.quantize(Stub(4, 64), out=stub_mx(4))
    if B.python_headers():  # then the module is made, although the library is up to date
        cc.write_text(cc.read_text().replace("exit 1", ":"))
        B.build()
        assert os.path.exists(B.FAST)


def test_few_tokens_go_to_the_faster_kernel():
    def pays(dtype, T, D=4096, I=1024, k=10):
        layer = object.__new__(MoELayer)
        layer.dtype, layer.D, layer.I, layer.top_k, layer.plan = dtype, D, I, k, None
        return layer.few_pays(T)

    for dtype in ("f32", "bf16", "fp8", "mxfp4"):
        assert pays(dtype, 1) and pays(dtype, 1, 7168, 2048, 8) and pays(dtype, 16, 512, 256, 4) and not pays(dtype, 17, 512, 256, 4)
    # both sides as measured
    assert pays("bf16", 12) and not pays("bf16", 16) and pays("bf16", 4, 7168, 2048, 8) and not pays("bf16", 8, 7168, 2048, 8)
    assert pays("fp8", 8) and not pays("fp8", 12) and not pays("fp8", 8, 7168, 2048, 8)
    assert pays("mxfp4", 8) and not pays("mxfp4", 9) and not pays("mxfp4", 16, 2048, 768, 8) and not pays("mxfp4", 8, 7168, 2048, 8)
    assert pays("f32", 16) and pays("f32", 16, 7168, 2048, 8)
