"""Microscaled 4-bit floats: the tensor-level calls over ``include/mhr_mxfp4.h``.

    quantize_mxfp4(x, axis=1, values=False, stream=None) -> MxFp4Matrix [, values]
    matmul_mxfp4(a, b, out=None, out_dtype=torch.float32, stream=None) -> C
    moe_mxfp4(x, router, up, down, top, out=None, stream=None) -> y, experts, weights

As in ``matmul``: argument checks and marshalling only, row-major CUDA tensors
(the last dimension contiguous), launches on ``stream`` (default: the current
torch stream) without synchronising, ``GemmError`` for a status other than
``MHR_OK``. On a stream other than the current one the caller orders the use
of the returned tensors itself.

The smallest calls take a few microseconds on the GPU, so the checks here read
each attribute once and the stream as a raw handle (0.1 us, against 1.9 us
through a Stream object on the Grace host).
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import MHR_OK, GemmError, load

#: mhr_dtype of the element types that plain matrices may have
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

_raw_stream = torch._C._cuda_getCurrentRawStream
_empty, _u8, _bf16 = torch.empty, torch.uint8, torch.bfloat16


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


def _plain(t, name):
    """rows, cols and row pitch of a row-major matrix."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    pitch, step = t.stride()
    if step != 1 and rows > 0 and cols > 1:
        raise ValueError(f"{name} must be row-major (last dimension contiguous)")
    return rows, cols, (pitch if rows > 1 and pitch > cols else cols)


def _packed(q, name):
    """data and scales pointers and bytes a row of an MxFp4Matrix."""
    data, scales, rows, cols = q
    if data.dtype is not _u8 or scales.dtype is not _u8:
        raise TypeError(f"{name}: data and scales must be uint8")
    have, width, pitch = _plain(data, name)
    if have != rows or width < -(-cols // 32) * 16:
        raise ValueError(f"{name}: data must be rows x 16 * ceil(cols / 32) bytes")
    if not scales.is_contiguous() or scales.numel() < mxfp4_scale_bytes(rows, cols):
        raise ValueError(f"{name}: scales must be contiguous, mxfp4_scale_bytes(rows, cols) bytes")
    return data.data_ptr(), scales.data_ptr(), pitch


def _device(*tensors):
    """Index of the one CUDA device that all tensors are on."""
    first = tensors[0]
    if not first.is_cuda:
        raise ValueError("operands must be CUDA tensors")
    index = first.get_device()
    for t in tensors:
        if t.get_device() != index:
            raise ValueError("operands must be on one device")
    return index


def _run(where, index, stream, entry, *args):
    """The C call on device `index` and `stream`; raises on a status."""
    if stream is None:
        stream = _raw_stream(index)
    if index == torch.cuda.current_device():
        rc = entry(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = entry(*args, stream)
    if rc != MHR_OK:
        raise GemmError(rc, where)


def quantize_mxfp4(x, axis: int = 1, values: bool = False, stream=None):
    """Quantise a 2-D tensor (float32, bfloat16 or float16) to MXFP4.

    ``axis`` is the one that blocks of 32 run along: 1 packs ``x`` itself (the
    left operand of a product), 0 packs ``x.T`` (a K x N right operand, as
    ``matmul_mxfp4`` takes it). With ``values`` also returns a tensor like
    ``x`` holding what the codes stand for.
    """
    dtype = DTYPES.get(x.dtype)
    if dtype is None:
        raise TypeError("x must be float32, bfloat16 or float16")
    if axis not in (0, 1):
        raise ValueError("axis must be 0 or 1")
    rows, cols, ldx = _plain(x, "x")
    index = _device(x)
    device = x.device
    prows, pcols = (rows, cols) if axis else (cols, rows)
    ldd = -(-pcols // 32) * 16
    data = _empty((prows, ldd), dtype=_u8, device=device)
    scales = _empty(mxfp4_scale_bytes(prows, pcols), dtype=_u8, device=device)
    v = _empty((rows, cols), dtype=x.dtype, device=device) if values else None
    _run("gemm_mxfp4_quantize", index, stream, load().gemm_mxfp4_quantize, dtype, x.data_ptr(),
         rows, cols, ldx, 1 - axis, data.data_ptr(), ldd, scales.data_ptr(),
         v.data_ptr() if values else None, cols)
    q = MxFp4Matrix(data, scales, prows, pcols)
    return (q, v) if values else q


def matmul_mxfp4(a, b, out=None, out_dtype=torch.float32, stream=None):
    """C = a @ B for a 4-bit B, given as the packed N x K matrix ``b`` of its transpose.

    ``a``: an M x K ``MxFp4Matrix``, or a tensor (float32, bfloat16, float16) that is
    quantised along its rows on the way. ``out`` (M x N, float32, bfloat16 or float16; of
    ``out_dtype`` when omitted) is overwritten and returned.
    """
    packed = isinstance(a, MxFp4Matrix)
    if packed:
        M, K = a.rows, a.cols
        a_data, a_scales, lda = _packed(a, "a")
    else:
        a_type = DTYPES.get(a.dtype)
        if a_type is None:
            raise TypeError("a must be an MxFp4Matrix or float32, bfloat16 or float16")
        M, K, lda = _plain(a, "a")
    N = b.rows
    if b.cols != K:
        raise ValueError(f"inner dimensions differ: {K} vs {b.cols}")
    if out is None:
        out = _empty((M, N), dtype=out_dtype, device=b.data.device)
    c_type = DTYPES.get(out.dtype)
    if c_type is None:
        raise TypeError("out must be float32, bfloat16 or float16")
    rows, cols, ldc = _plain(out, "out")
    if rows != M or cols != N:
        raise TypeError("out must be of shape (M, N)")
    b_data, b_scales, ldb = _packed(b, "b")
    if packed:
        index = _device(b.data, b.scales, a.data, a.scales, out)
        _run("gemm_mxfp4", index, stream, load().gemm_mxfp4, c_type, a_data, a_scales, b_data,
             b_scales, out.data_ptr(), M, N, K, lda, ldb, ldc)
    else:
        index = _device(b.data, b.scales, a, out)
        _run("gemm_mxfp4_quantized", index, stream, load().gemm_mxfp4_quantized, a_type,
             a.data_ptr(), c_type, b_data, b_scales, out.data_ptr(), M, N, K, lda, ldb, ldc)
    return out


def moe_mxfp4(x, router, up, down, top: int, out=None, stream=None):
    """A mixture-of-experts layer over 4-bit experts for up to 64 tokens, in one kernel.

    ``x``: T x H bfloat16; ``router``: E x H bfloat16; ``up``: the packed 2 E I x H matrix of
    the experts' gate and up weights (expert e: I gate rows, then I up rows); ``down``: the
    packed E H x I matrix (expert e: H rows). Returns ``y`` (T x H bfloat16), the chosen
    experts (T x top int32, best first, ties to the lowest index) and their weights (T x top
    float32, a softmax over the chosen): y_t = sum of weight * down_e (silu(gate_e x_t) *
    (up_e x_t)).
    """
    if x.dtype is not _bf16 or router.dtype is not _bf16:
        raise TypeError("x and router must be bfloat16")
    T, H, ldx = _plain(x, "x")
    E, width, ldr = _plain(router, "router")
    I = down.cols
    if width != H or up.cols != H or up.rows != 2 * E * I or down.rows != E * H:
        raise ValueError("sizes differ: x is T x H, router E x H, up 2 E I x H, down E H x I")
    u_data, u_scales, ldu = _packed(up, "up")
    d_data, d_scales, ldd = _packed(down, "down")
    device = x.device
    if out is None:
        out = _empty((T, H), dtype=_bf16, device=device)
    rows, cols, ldy = _plain(out, "out")
    if out.dtype is not _bf16 or rows != T or cols != H:
        raise TypeError("out must be bfloat16 of x's shape")
    index = _device(x, router, up.data, up.scales, down.data, down.scales, out)
    experts = _empty((T, top), dtype=torch.int32, device=device)
    weights = _empty((T, top), dtype=torch.float32, device=device)
    _run("gemm_mxfp4_moe", index, stream, load().gemm_mxfp4_moe, x.data_ptr(), ldx,
         router.data_ptr(), ldr, u_data, u_scales, ldu, d_data, d_scales, ldd, out.data_ptr(), ldy,
         experts.data_ptr(), weights.data_ptr(), T, E, top, H, I)
    return out, experts, weights
