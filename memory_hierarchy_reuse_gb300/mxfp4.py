"""Microscaled 4-bit floats: the tensor-level calls over ``include/mhr_mxfp4.h``.

    quantize_mxfp4(x, axis=1, values=False, stream=None) -> MxFp4Matrix [, values]
    matmul_mxfp4(a, b, out=None, out_dtype=torch.float32, stream=None) -> C
    moe_mxfp4(x, router, up, down, top, out=None, stream=None) -> y, experts, weights

As in ``matmul``: argument checks and marshalling only, row-major CUDA tensors
(the last dimension contiguous), launches on ``stream`` (default: the current
torch stream) without synchronising, ``GemmError`` for a status other than
``MHR_OK``. On a stream other than the current one the caller orders the use
of the returned tensors itself.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import MHR_OK, GemmError, _rowmajor, load

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


def _check_packed(q, name):
    data, scales = q.data, q.scales
    if data.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise TypeError(f"{name}: data and scales must be uint8")
    if data.dim() != 2 or data.shape[0] != q.rows or data.shape[1] < -(-q.cols // 32) * 16:
        raise ValueError(f"{name}: data must be rows x 16 * ceil(cols / 32) bytes")
    if not scales.is_contiguous() or scales.numel() < mxfp4_scale_bytes(q.rows, q.cols):
        raise ValueError(f"{name}: scales must be contiguous, mxfp4_scale_bytes(rows, cols) bytes")
    return _rowmajor(data, f"{name}.data") if q.rows > 1 else -(-q.cols // 32) * 16


def _run(where, device, stream, entry, *args):
    """The C call on `device` and `stream`; raises on a status."""
    if stream is None:
        stream = torch.cuda.current_stream(device).cuda_stream
    if device.index == torch.cuda.current_device():
        rc = entry(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = entry(*args, stream)
    if rc != MHR_OK:
        raise GemmError(rc, where)


def _same_device(device, **tensors):
    if device.type != "cuda":
        raise ValueError("operands must be CUDA tensors")
    for name, t in tensors.items():
        if t.device != device:
            raise ValueError(f"{name} must be on {device}")


def quantize_mxfp4(x, axis: int = 1, values: bool = False, stream=None):
    """Quantise a 2-D tensor (float32, bfloat16 or float16) to MXFP4.

    ``axis`` is the one that blocks of 32 run along: 1 packs ``x`` itself (the
    left operand of a product), 0 packs ``x.T`` (a K x N right operand, as
    ``matmul_mxfp4`` takes it). With ``values`` also returns a tensor like
    ``x`` holding what the codes stand for.
    """
    if x.dtype not in DTYPES:
        raise TypeError("x must be float32, bfloat16 or float16")
    if axis not in (0, 1):
        raise ValueError("axis must be 0 or 1")
    ldx = _rowmajor(x, "x")
    _same_device(x.device)
    rows, cols = x.shape
    prows, pcols = (cols, rows) if axis == 0 else (rows, cols)
    ldd = -(-pcols // 32) * 16
    data = torch.empty((prows, ldd), dtype=torch.uint8, device=x.device)
    scales = torch.empty(mxfp4_scale_bytes(prows, pcols), dtype=torch.uint8, device=x.device)
    v = torch.empty((rows, cols), dtype=x.dtype, device=x.device) if values else None
    _run("gemm_mxfp4_quantize", x.device, stream, load().gemm_mxfp4_quantize, DTYPES[x.dtype],
         x.data_ptr(), rows, cols, ldx, 1 - axis, data.data_ptr(), ldd, scales.data_ptr(),
         None if v is None else v.data_ptr(), cols)
    q = MxFp4Matrix(data, scales, prows, pcols)
    return (q, v) if values else q


def matmul_mxfp4(a, b, out=None, out_dtype=torch.float32, stream=None):
    """C = a @ B for a 4-bit B, given as the packed N x K matrix ``b`` of its transpose.

    ``a``: an M x K ``MxFp4Matrix``, or a tensor (float32, bfloat16, float16) that is
    quantised along its rows on the way. ``out`` (M x N, float32, bfloat16 or float16; of
    ``out_dtype`` when omitted) is overwritten and returned.
    """
    packed = isinstance(a, MxFp4Matrix)
    M, K = (a.rows, a.cols) if packed else a.shape
    N = b.rows
    if b.cols != K:
        raise ValueError(f"inner dimensions differ: {K} vs {b.cols}")
    device = b.data.device
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=device)
    if out.dtype not in DTYPES or tuple(out.shape) != (M, N):
        raise TypeError("out must be float32, bfloat16 or float16 of shape (M, N)")
    ldb, ldc = _check_packed(b, "b"), _rowmajor(out, "out")
    c = DTYPES[out.dtype]
    if packed:
        lda = _check_packed(a, "a")
        _same_device(device, a=a.data, a_scales=a.scales, b_scales=b.scales, out=out)
        _run("gemm_mxfp4", device, stream, load().gemm_mxfp4, c, a.data.data_ptr(),
             a.scales.data_ptr(), b.data.data_ptr(), b.scales.data_ptr(), out.data_ptr(),
             M, N, K, lda, ldb, ldc)
    else:
        if a.dtype not in DTYPES:
            raise TypeError("a must be an MxFp4Matrix or float32, bfloat16 or float16")
        lda = _rowmajor(a, "a")
        _same_device(device, a=a, b_scales=b.scales, out=out)
        _run("gemm_mxfp4_quantized", device, stream, load().gemm_mxfp4_quantized, DTYPES[a.dtype],
             a.data_ptr(), c, b.data.data_ptr(), b.scales.data_ptr(), out.data_ptr(),
             M, N, K, lda, ldb, ldc)
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
    if x.dtype != torch.bfloat16 or router.dtype != torch.bfloat16:
        raise TypeError("x and router must be bfloat16")
    ldx, ldr = _rowmajor(x, "x"), _rowmajor(router, "router")
    (T, H), E, I = x.shape, router.shape[0], down.cols
    if router.shape[1] != H or up.cols != H or up.rows != 2 * E * I or down.rows != E * H:
        raise ValueError("sizes differ: x is T x H, router E x H, up 2 E I x H, down E H x I")
    ldu, ldd = _check_packed(up, "up"), _check_packed(down, "down")
    device = x.device
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=device)
    if out.dtype != torch.bfloat16 or out.shape != x.shape:
        raise TypeError("out must be bfloat16 of x's shape")
    ldy = _rowmajor(out, "out")
    _same_device(device, router=router, up=up.data, up_scales=up.scales, down=down.data,
                 down_scales=down.scales, out=out)
    experts = torch.empty((T, top), dtype=torch.int32, device=device)
    weights = torch.empty((T, top), dtype=torch.float32, device=device)
    _run("gemm_mxfp4_moe", device, stream, load().gemm_mxfp4_moe, x.data_ptr(), ldx,
         router.data_ptr(), ldr, up.data.data_ptr(), up.scales.data_ptr(), ldu,
         down.data.data_ptr(), down.scales.data_ptr(), ldd, out.data_ptr(), ldy,
         experts.data_ptr(), weights.data_ptr(), T, E, top, H, I)
    return out, experts, weights
