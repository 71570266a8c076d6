"""Microscaled 4-bit floats: the tensor-level calls over ``include/mhr_mxfp4.h``.

    quantize_mxfp4(x, axis=1, values=False, stream=None) -> MxFp4Matrix [, values]
    matmul_mxfp4(a, b, out=None, out_dtype=torch.float32, stream=None) -> C
    moe_mxfp4(x, router, up, down, top, out=None, stream=None) -> y, experts, weights

As in ``matmul``: argument checks and marshalling only, row-major CUDA tensors
(the last dimension contiguous), launches on ``stream`` (default: the current
torch stream) without synchronising, ``GemmError`` for a status other than
``MHR_OK``. On a stream other than the current one the caller orders the use
of the returned tensors itself.

The checks, the outputs' allocation and the C call are in the compiled
``csrc/torch_binding.cpp``: the smallest calls take a few microseconds on the GPU.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import GemmError, load

try:
    from . import _torch_binding
except ImportError as e:
    raise RuntimeError("the torch binding is missing or does not load: build it with "
                       "memory_hierarchy_reuse_gb300.build.build()") from e

#: mhr_dtype of the element types that plain matrices may have
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class MxFp4Matrix(NamedTuple):
    """A ``rows`` x ``cols`` matrix in 4 bits (the layout is in mhr_mxfp4.h).

    ``data``: uint8, ``rows`` x at least 16 * ceil(cols / 32), rows contiguous
    and a multiple of 16 bytes apart; ``scales``: uint8, contiguous,
    ``mxfp4_scale_bytes(rows, cols)`` bytes.
    """

    data: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int


def mxfp4_scale_bytes(rows: int, cols: int) -> int:
    """Bytes of the scales of a rows x cols matrix."""
    return -(-rows // 128) * -(-cols // 128) * 512


_lib = load()
_torch_binding.init(*(ctypes.cast(f, ctypes.c_void_p).value
                      for f in (_lib.gemm_mxfp4_quantize, _lib.gemm_mxfp4,
                                _lib.gemm_mxfp4_quantized, _lib.gemm_mxfp4_moe)),
                    MxFp4Matrix, GemmError)


def quantize_mxfp4(x, axis: int = 1, values: bool = False, stream=None):
    """Quantise a 2-D tensor (float32, bfloat16 or float16) to MXFP4.

    ``axis`` is the one that blocks of 32 run along: 1 packs ``x`` itself (the
    left operand of a product), 0 packs ``x.T`` (a K x N right operand, as
    ``matmul_mxfp4`` takes it). With ``values`` also returns a tensor like
    ``x`` holding what the codes stand for.
    """
    return _torch_binding.quantize(x, axis, values, stream)


def matmul_mxfp4(a, b, out=None, out_dtype=torch.float32, stream=None):
    """C = a @ B for a 4-bit B, given as the packed N x K matrix ``b`` of its transpose.

    ``a``: an M x K ``MxFp4Matrix``, or a tensor (float32, bfloat16, float16) that is
    quantised along its rows on the way. ``out`` (M x N, float32, bfloat16 or float16; of
    ``out_dtype`` when omitted) is overwritten and returned.
    """
    return _torch_binding.matmul(a, b, out, DTYPES.get(out_dtype, -1), stream)


def moe_mxfp4(x, router, up, down, top: int, out=None, stream=None):
    """A mixture-of-experts layer over 4-bit experts for up to 64 tokens, in one kernel.

    ``x``: T x H bfloat16; ``router``: E x H bfloat16; ``up``: the packed 2 E I x H matrix of
    the experts' gate and up weights (expert e: I gate rows, then I up rows); ``down``: the
    packed E H x I matrix (expert e: H rows). Returns ``y`` (T x H bfloat16), the chosen
    experts (T x top int32, best first, ties to the lowest index) and their weights (T x top
    float32, a softmax over the chosen): y_t = sum of weight * down_e (silu(gate_e x_t) *
    (up_e x_t)).
    """
    return _torch_binding.moe(x, router, up, down, top, out, stream)
