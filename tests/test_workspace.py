"""A workspace sized for T_max tokens serves every smaller T."""
import glob
import os
import subprocess

import pytest
import torch

from sparse_moe_expert_02_gb300 import MoELayer, synth
from sparse_moe_expert_02_gb300 import build as B

# The layout as the library computes it, for every T up to a few thousand on
# GPUs of several sizes: the size never shrinks, and each part that depends on
# how T is worked on holds what that takes.
HARNESS = r"""
#include "api.cu"
int main() {
    const int shapes[][4] = {{4096, 512, 1024, 10}, {1024, 64, 4096, 2}, {512, 32, 256, 4}, {2048, 256, 768, 8},
                             {256, 1, 128, 1}, {7168, 256, 2048, 8}, {256, 1024, 128, 32}, {384, 700, 128, 3}};
    int bad = 0;
    for (auto& sh : shapes)
        for (int dt = 0; dt < 4; ++dt)
            for (unsigned flags : {0u, MOE_FLAG_DOWN_HILO})
                for (int sms : {8, 132, 152}) {
                    moe_config c = {};
                    c.T_max = 1 << 20; c.D = sh[0]; c.E = sh[1]; c.I = sh[2]; c.top_k = sh[3]; c.dtype = dt; c.flags = flags;
                    size_t last = 0;
                    for (int T = 1; T <= 6000; ++T) {
                        moe_ws_layout L;
                        layout(c, sms, T, &L);
                        const int64_t TK = (int64_t)T * c.top_k;
                        const int S = route_splits(c, T, sms);
                        const bool ok = L.total >= last && L.xq % 4 == 0 &&
                            L.hist + moe::cdiv(TK, moe::perm_chunk(TK)) * c.E * 4 <= (dt == MOE_FP8_E4M3_B128 ? L.xq : L.xp) &&
                            (S > 1 ? L.logits_part > L.y && L.logits_part + (size_t)S * T * c.E * 4 <= L.tiles2 : L.logits_part == 0) &&
                            (T > MOE_FEW_MAX || L.few + (size_t)(TK + T) * c.I * 4 <= L.total);
                        if (!ok && bad++ < 20)
                            printf("D %d E %d I %d k %d dtype %d flags %u SMs %d T %d: %zu after %zu\n", c.D, c.E, c.I, c.top_k, dt, flags, sms, T, L.total, last);
                        last = L.total;
                    }
                }
    return bad != 0;
}
"""


def test_workspace_size_never_shrinks_as_tokens_grow(tmp_path):
    B.build()
    src, exe = tmp_path / "layout.cu", tmp_path / "layout"
    src.write_text(HARNESS)
    objs = [o for o in glob.glob(os.path.join(B.BUILD, "*.o")) if os.path.basename(o) != "api.o"]
    subprocess.run([B.nvcc()] + B.ARCH + ["-O1", "-std=c++17", "--expt-relaxed-constexpr", "-I", B.INCLUDE, "-I", B.CSRC, str(src)]
                   + objs + ["-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("D,E,I,k", [(512, 32, 256, 4), (256, 16, 1024, 2)])
def test_smaller_batches_run_on_the_workspace_of_the_largest(dtype, D, E, I, k):
    shape = synth.LayerShape("ws", 16, D, E, I, k, "fp8" if dtype == "mxfp4" else dtype, 1.0)
    inp = synth.make_inputs(shape, seed=5, device="cuda")
    want = {}
    for T_max in (16, 17, 18, 20, 24, 48):
        layer = MoELayer(D, E, I, k, dtype, inp, T_max=T_max, has_router_bias=shape.has_bias)
        for T in (16, 15):
            for name, call in (("all", layer.forward), ("few", layer.forward_few)):
                out = call(inp["x"][:T])
                layer.check()
                assert torch.equal(out, want.setdefault((T, name), out))
