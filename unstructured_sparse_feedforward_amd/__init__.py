"""Activation-sparse ReLU feedforward layer for AMD MI355X (gfx950).

The compute lives in libsffn.so (HIP kernels behind the C ABI of
include/sffn.h); :mod:`.binding` marshals torch tensors into it,
:mod:`.mxfp4` and :mod:`.mxfp8` do so for the 4- and 8-bit matrices,
:mod:`.norm` for the residual norm between layers, :mod:`.moe` and
:mod:`.router` for the expert layer and its router, and :mod:`.workloads`
draws the seeded synthetic inputs.
"""
from .binding import SparseFFN, SffnError, load_library  # noqa: F401
from .moe import SparseMoE  # noqa: F401
from .mxfp4 import (MXTensor, mx_dequantize, mx_empty, mx_matmul,  # noqa: F401
                    mx_quantize)
from .mxfp8 import MX8Tensor, mx8_dequantize, mx8_empty, mx8_quantize  # noqa: F401
from .norm import rms_norm, rms_norm_backward  # noqa: F401
from .router import MoERouter  # noqa: F401
