"""Products by an index per row: the tensor-level calls over ``include/mhr_routed.h``.

    choose_experts(logits, top, ...) -> experts, weights
    choose_experts_grad(logits, experts, grad_weights, ...) -> grad_logits
    sort_by_expert(experts, count) -> offsets, order
    matmul_experts(x, w, offsets, ...) -> out
    matmul_experts_grad(x, grad, offsets, ...) -> gradient of w
    add_adapters(y, x, down, up, which, ...) -> out

As in ``mxfp4.py``: argument checks and marshalling only (in the compiled
``csrc/torch_binding.cpp``), launches on ``stream`` (default: the current torch
stream) without synchronising, ``GemmError`` for a status other than ``MHR_OK``.
On a stream other than the current one the caller orders the use of the returned
tensors itself. All calls can be captured into a graph. Automatic differentiation
records none of them: a gradient is a call of its own (that of ``add_adapters``'
x is ``add_adapters`` with ``up`` and ``down`` in each other's place).
"""
from __future__ import annotations

import ctypes

from . import load
from .mxfp4 import DTYPES, _torch_binding

_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}

_lib = load()
_torch_binding.init_routed(*(ctypes.cast(f, ctypes.c_void_p).value
                             for f in (_lib.gemm_routed_choose, _lib.gemm_routed_choose_grad,
                                       _lib.gemm_routed_sort, _lib.gemm_routed_product_scratch,
                                       _lib.gemm_routed_product,
                                       _lib.gemm_routed_weight_grad_scratch,
                                       _lib.gemm_routed_weight_grad,
                                       _lib.gemm_routed_adapters_scratch,
                                       _lib.gemm_routed_adapters)))


def choose_experts(logits, top: int, score: str = "softmax", bias=None, groups: int = 1,
                   group_top: int = 1, group_score: str = "max", renormalize: bool = True,
                   scale: float = 1.0, stream=None):
    """The ``top`` experts of each token (T x top int32, best first) and their weights (float32).

    ``logits``: T x E float32, bfloat16 or float16. ``score``: "softmax" over all experts, or
    "sigmoid". ``bias`` (E float32) is added to the scores for the choice, not for the weights.
    With ``groups`` > 1, the ``group_top`` groups of neighbouring experts with the best
    ``group_score`` ("max", or "top2": the sum of the two best) stay in the choice. Ties go to the
    lowest index. Weights are the chosen scores, divided by their sum with ``renormalize``, times
    ``scale``. Limits: E <= 512, top <= 16, groups <= 32.
    """
    return _torch_binding.choose(logits, top, _SCORES.get(score, -1), bias, groups, group_top,
                                 _GROUP_SCORES.get(group_score, -1), renormalize, scale, stream)


def choose_experts_grad(logits, experts, grad_weights, score: str = "softmax",
                        renormalize: bool = True, scale: float = 1.0, out=None, stream=None):
    """The gradient of ``choose_experts``' logits (their type and shape) for one of its weights.

    ``experts``: as chosen (T x top int32); ``grad_weights``: T x top float32. The choice itself
    has no gradient, and so the bias and the groups have none.
    """
    return _torch_binding.choose_grad(logits, experts, grad_weights, _SCORES.get(score, -1),
                                      renormalize, scale, out, stream)


def sort_by_expert(experts, count: int, stream=None):
    """The (token, slot) pairs one expert after the other.

    ``experts``: int32 of any shape, contiguous. Returns ``offsets`` (count + 1 int32; expert e's
    pairs are at offsets[e] to offsets[e + 1]) and ``order`` (int32): the pairs' positions in
    ``experts`` (as a flat array), ascending within an expert; those of entries outside
    0 .. count-1 come last, from offsets[count] on. ``count`` <= 1024.
    """
    return _torch_binding.sort(experts, count, stream)


def _out_dtype(dtype):
    return None if dtype is None else DTYPES.get(dtype, -1)


def matmul_experts(x, w, offsets, gather=None, scatter=None, top: int = 1,
                   transposed: bool = False, out=None, out_dtype=None, stream=None):
    """out[q] = x[q] @ w[e] for the sorted rows q of each expert, offsets[e] <= q < offsets[e + 1].

    ``x``: rows x K and ``w``: experts x K x N (experts x N x K with ``transposed``, whose product
    is with ``w[e].T``: the gradient of x), both bfloat16 or both float16. ``gather`` and
    ``scatter`` (int32, one entry a sorted row: ``sort_by_expert``'s ``order``): row q is
    ``x[gather[q] // top]``, and is written to ``out[scatter[q]]`` -- with ``top`` the router's,
    ``x`` is the tokens, and ``out`` in (token, slot) order. ``out`` (of ``out_dtype``, x's when
    omitted; or given, float32, bfloat16 or float16, and of ``out_dtype`` where that is given too)
    is returned. Its rows that no expert has stay as they were: undefined when it is allocated here.
    """
    return _torch_binding.experts(x, w, offsets, gather, scatter, top, transposed, out,
                                  _out_dtype(out_dtype), stream)


def matmul_experts_grad(x, grad, offsets, gather=None, scatter=None, top: int = 1, out=None,
                        out_dtype=None, stream=None):
    """The gradient of ``matmul_experts``' weights (experts x K x N): the sum of
    ``x[row].T @ grad[row]`` over each expert's sorted rows, zeros for one without.

    ``grad``: the gradient of the product's output, of x's type, rows x N; the indices as there
    (``grad``'s rows are ``scatter``'s). ``out_dtype``: x's when omitted.
    """
    return _torch_binding.experts_grad(x, grad, offsets, gather, scatter, top, out,
                                       _out_dtype(out_dtype), stream)


def add_adapters(y, x, down, up, which, scales=None, out=None, stream=None):
    """out[t] = y[t] + scales[a] * (x[t] @ down[a].T) @ up[a] with a = which[t].

    ``y`` (T x N, float32, bfloat16 or float16): the shared projection's result. ``x``: T x K,
    ``down``: adapters x rank x K, ``up``: adapters x rank x N, all bfloat16 or all float16.
    ``which``: T int32; a row outside 0 .. adapters-1 has no adapter. ``scales``: one float32 an
    adapter (1 when omitted). ``out``: of y's type and shape, y itself for a sum in place, or
    allocated. Limits: 1024 adapters of rank 128.
    """
    return _torch_binding.adapters(y, x, down, up, which, scales, out, stream)
