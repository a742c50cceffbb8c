"""Single-GPU (sm_103a) routed Mixture-of-Experts FFN layer.

The layer -- router, top-k with renormalised softmax weights, expert-grouped
permutation, SwiGLU expert GEMMs on the tensor cores, unpermutation with the
shared-expert add -- runs in the CUDA kernels of libmoe (include/moe.h),
reached through the ctypes binding in ``_lib``.  ``MoELayer`` holds one layer's
weights and workspace on the device; ``MoEBlock`` puts the norms, the gate and
the residual stream of a decoder block around it; ``norm`` and ``mx`` hold the
norms and the microscaled 4-bit operators by themselves; ``grouped`` holds the
experts' products with their gradients and the activation between them,
``int4`` products with 4-bit integer weights; ``synth`` draws seeded synthetic
inputs.
"""
from .layer import MoELayer  # noqa: F401
from .block import MoEBlock  # noqa: F401
from . import grouped, int4, mx, norm, synth  # noqa: F401
