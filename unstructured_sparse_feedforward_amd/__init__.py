"""Activation-sparse ReLU feedforward layer for AMD MI355X (gfx950).

The compute lives in libsffn.so (HIP kernels behind the C ABI of
include/sffn.h); :mod:`.binding` marshals torch tensors into it,
:mod:`.mxfp4` does so for the 4-bit matrices and :mod:`.moe` for the expert
layer, and :mod:`.workloads` draws the seeded synthetic inputs.
"""
from .binding import SparseFFN, SffnError, load_library  # noqa: F401
from .moe import SparseMoE  # noqa: F401
from .mxfp4 import (MXTensor, mx_dequantize, mx_empty, mx_matmul,  # noqa: F401
                    mx_quantize)
