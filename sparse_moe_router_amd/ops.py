"""The operators in ``include/moe_ops.h`` on torch tensors: products grouped by
expert with their gradients, 8-bit products, the norms around a block, and what a
training step needs beside them: gated products, the sum over a token's experts,
clipping and the loss.

Argument marshalling only, as in :mod:`.moe`: torch tensors provide device
memory and the stream, every step runs in the library's HIP kernels, and a
tensor that the kernels cannot take raises.  Activations (``x``, ``y``, ``dy``,
``residual``, ``gate`` ...) are matrices whose rows are contiguous; their rows
may be strided (a slice of columns), by a multiple of 16 bytes.  Weights,
offsets, permutations and per-token vectors are contiguous.  A call runs on the
current stream of its tensors' device, or on ``stream``; what the caller does
not pass is allocated there, workspaces among it, so that calls on different
streams and captured graphs never share one; tensors written on other streams
must be ready on it.  Nothing is recorded for automatic differentiation: the
gradients are calls of their own, and a tensor that requires a gradient where
torch records them gives a warning.  A tensor of the caller's that a call writes
(an ``out``, a list clipped in place) has a new version afterwards, so that a
graph which had saved it refuses its new values.

``offsets`` (int32 [E+1]) and ``perm`` (int32 [rows]) are the group offsets and
the permutation that :func:`sparse_moe_router_amd.route` reports.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import moe
from .moe import MoeError  # noqa: F401

try:
    from . import _ops
except ImportError as e:  # not built, or built against another torch
    raise ImportError(f"{e}; build it with `python -m sparse_moe_router_amd.build`") from e

EXPORTS = ("moe_grouped_matmul", "moe_grouped_matmul_grad_input", "moe_grouped_matmul_grad_weight",
           "moe_quantize_i8", "moe_matmul_i8_workspace_size", "moe_matmul_i8", "moe_block_norm",
           "moe_block_norm_grad", "moe_block_merge", "moe_block_merge_grad", "moe_norm_grad_workspace_size",
           "moe_gated_matmul", "moe_gated_matmul_grad", "moe_feed_forward_grad_workspace_size",
           "moe_feed_forward_grad", "moe_invert_permutation", "moe_combine", "moe_combine_grad",
           "moe_grad_norm_workspace_size", "moe_grad_norm", "moe_clip_grads", "moe_cross_entropy_workspace_size",
           "moe_cross_entropy", "moe_cross_entropy_grad_workspace_size", "moe_cross_entropy_grad")


class MoeGroups(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("x_rows", ctypes.c_int64), ("ldx", ctypes.c_int64),
                ("ldy", ctypes.c_int64), ("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("offsets", ctypes.c_void_p), ("perm", ctypes.c_void_p)]


class MoeNorm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("H", ctypes.c_int32), ("stream_type", ctypes.c_int),
                ("weight_type", ctypes.c_int), ("gate_mode", ctypes.c_int), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float)]


class MoeMat(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64)]


class MoeFeedForward(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("x_rows", ctypes.c_int64), ("ldx", ctypes.c_int64),
                ("ld_dy", ctypes.c_int64), ("E", ctypes.c_int32), ("I", ctypes.c_int32), ("K", ctypes.c_int32),
                ("H", ctypes.c_int32), ("top_k", ctypes.c_int32), ("offsets", ctypes.c_void_p), ("perm", ctypes.c_void_p)]


class MoeCombine(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("rows", ctypes.c_int64), ("H", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("E", ctypes.c_int32), ("out_type", ctypes.c_int), ("inverse", ctypes.c_void_p),
                ("perm", ctypes.c_void_p), ("offsets", ctypes.c_void_p)]


class MoeTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64), ("in_type", ctypes.c_int),
                ("out_type", ctypes.c_int)]


class MoeLoss(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("ldx", ctypes.c_int64), ("V", ctypes.c_int32), ("H", ctypes.c_int32),
                ("ignore_index", ctypes.c_int64)]



_bound = None


def lib() -> ctypes.CDLL:
    """The loaded library with this module's entry points declared (raises if it has not been built)."""
    global _bound
    if _bound is None:
        L = moe.lib()
        vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
        g, n, en, f32 = ctypes.POINTER(MoeGroups), ctypes.POINTER(MoeNorm), ctypes.c_int, ctypes.c_float
        ff = ctypes.POINTER(MoeFeedForward)
        c, t, l = ctypes.POINTER(MoeCombine), ctypes.POINTER(MoeTensor), ctypes.POINTER(MoeLoss)
        sig = {
            "moe_grouped_matmul": (en, [g, vp, vp, vp, en, vp]),
            "moe_grouped_matmul_grad_input": (en, [g, vp, vp, vp, en, vp]),
            "moe_grouped_matmul_grad_weight": (en, [g, vp, vp, vp, en, vp]),
            "moe_quantize_i8": (en, [i64, i32, i64, vp, vp, vp, vp]),
            "moe_matmul_i8_workspace_size": (sz, [g]),
            "moe_matmul_i8": (en, [g, vp, vp, vp, vp, vp, vp, en, vp, sz, vp]),
            "moe_block_norm": (en, [n, MoeMat, vp, MoeMat, vp]),
            "moe_block_norm_grad": (en, [n, MoeMat, MoeMat, vp, MoeMat, MoeMat, vp, vp, sz, vp]),
            "moe_block_merge": (en, [n, MoeMat, MoeMat, vp, MoeMat, vp, MoeMat, MoeMat, vp]),
            "moe_block_merge_grad": (en, [n, MoeMat, MoeMat, MoeMat, vp, MoeMat, MoeMat, vp, MoeMat, MoeMat, MoeMat,
                                          vp, vp, vp, sz, vp]),
            "moe_norm_grad_workspace_size": (sz, [n]),
            "moe_gated_matmul": (en, [g, vp, vp, vp, MoeMat, vp]),
            "moe_gated_matmul_grad": (en, [g, vp, vp, MoeMat, MoeMat, vp, vp]),
            "moe_feed_forward_grad_workspace_size": (sz, [ff]),
            "moe_feed_forward_grad": (en, [ff, vp, vp, vp, vp, MoeMat, MoeMat, vp, vp, en, vp, sz, vp]),
            "moe_invert_permutation": (en, [i64, vp, vp, i32, i64, vp, vp]),
            "moe_combine": (en, [c, MoeMat, vp, MoeMat, MoeMat, vp]),
            "moe_combine_grad": (en, [c, MoeMat, MoeMat, vp, MoeMat, vp, vp]),
            "moe_grad_norm_workspace_size": (sz, [t, i32]),
            "moe_grad_norm": (en, [t, i32, vp, vp, sz, vp]),
            "moe_clip_grads": (en, [t, i32, f32, f32, vp, i32, vp, sz, vp]),
            "moe_cross_entropy_workspace_size": (sz, [l]),
            "moe_cross_entropy": (en, [l, vp, vp, vp, vp, vp, vp, sz, vp]),
            "moe_cross_entropy_grad_workspace_size": (sz, [l]),
            "moe_cross_entropy_grad": (en, [l, vp, vp, vp, vp, vp, MoeMat, en, vp, en, vp, sz, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _bound = L
    return _bound


_FP32 = {torch.bfloat16: 0, torch.float32: 1}


def _fp32(dtype) -> int:
    try:
        return _FP32[dtype]
    except KeyError:
        raise TypeError(f"out_dtype must be torch.bfloat16 or torch.float32, got {dtype}") from None


def _same_device(stream, *args):
    for a in args:
        if isinstance(a, torch.Tensor) and a.is_cuda and a.device != stream.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {a.device}")


def _call(stream, f, *args):
    """f on `stream`: that stream and its device are current while it runs."""
    if stream is None:
        return f(*args)
    _same_device(stream, *args)
    with torch.cuda.stream(stream):
        return f(*args)


# ------------------------------------------------------------------ grouped products

def grouped_matmul(x: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor],
                   perm: Optional[torch.Tensor] = None, top_k: int = 1, out: Optional[torch.Tensor] = None,
                   out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """moe_grouped_matmul: ``out[p] = x[row(p)] @ w[e].T`` for the rows p of each expert's group.

    x bf16 [tokens, K]; w bf16 [E, N, K]; row(p) is ``perm[p] // top_k`` with a permutation, else p.
    Returns out [rows, N] (bf16 or fp32), rows = those of ``perm``, else of x; rows from
    ``offsets[E]`` on keep what ``out`` held (an allocated ``out`` is not cleared)."""
    return _call(stream, _ops.grouped_matmul, x, w, offsets, perm, top_k, out, _fp32(out_dtype))


def grouped_matmul_grad_input(dy: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor],
                              out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                              stream=None) -> torch.Tensor:
    """moe_grouped_matmul_grad_input: ``out[p] = dy[p] @ w[e]``, the gradient of each grouped row
    (with a permutation, of the row's own copy of its token)."""
    return _call(stream, _ops.grouped_matmul_grad_input, dy, w, offsets, out, _fp32(out_dtype))


def grouped_matmul_grad_weight(x: torch.Tensor, dy: torch.Tensor, offsets: Optional[torch.Tensor],
                               perm: Optional[torch.Tensor] = None, top_k: int = 1,
                               out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.float32,
                               stream=None) -> torch.Tensor:
    """moe_grouped_matmul_grad_weight: ``out[e] = sum_p dy[p].T x[row(p)]`` over each expert's rows,
    [E, N, K] in fp32 or bf16; zeros for an expert without rows."""
    return _call(stream, _ops.grouped_matmul_grad_weight, x, dy, offsets, perm, top_k, out, _fp32(out_dtype))


# ------------------------------------------------------------------ 8-bit products

def quantize_i8(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                stream=None):
    """moe_quantize_i8: (codes int8 [tokens, K], scale fp32 [tokens]) of bf16 rows,
    ``codes = rint(127 x / max|x|)``, ``scale = max|x| / 127``."""
    return _call(stream, _ops.quantize_i8, x, codes, scale)


def matmul_i8(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, x_scale: Optional[torch.Tensor] = None,
              bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              out_dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """moe_matmul_i8 with one weight matrix: ``out = (q @ w.T) * x_scale[:, None] * w_scale (+ bias)``.

    w int8 [N, K], w_scale fp32 [N], bias fp32 [N] or None.  x is bf16 [tokens, K] (quantised by the
    call as :func:`quantize_i8` does) or int8 codes with x_scale fp32 [tokens].  The integer sums are
    exact; out is bf16 or fp32."""
    if isinstance(w, torch.Tensor) and w.dim() != 2:
        raise ValueError(f"w must have 2 dimensions, got {tuple(w.shape)}")
    return _call(stream, _ops.matmul_i8, x, w, w_scale, None, None, 1, x_scale, bias, out, _fp32(out_dtype), workspace)


def grouped_matmul_i8(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, offsets: Optional[torch.Tensor],
                      perm: Optional[torch.Tensor] = None, top_k: int = 1, x_scale: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_matmul_i8 grouped by expert: :func:`grouped_matmul` on int8 weights w [E, N, K] with
    w_scale fp32 [E, N]; x as in :func:`matmul_i8`."""
    if isinstance(w, torch.Tensor) and w.dim() != 3:
        raise ValueError(f"w must have 3 dimensions, got {tuple(w.shape)}")
    return _call(stream, _ops.matmul_i8, x, w, w_scale, offsets, perm, top_k, x_scale, None, out, _fp32(out_dtype),
                 workspace)


# ------------------------------------------------------------------ block norms

def block_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """moe_block_norm: ``x * rsqrt(mean(x^2) + eps) * weight`` in bf16; x bf16 or fp32 [tokens, H],
    weight bf16 or fp32 [H]."""
    return _call(stream, _ops.block_norm, x, weight, eps, out)


def block_norm_grad(d_h: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, eps: float,
                    d_add: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> dict:
    """moe_block_norm_grad: the gradients of :func:`block_norm` as a dict: ``x`` (in x's type; d_add, the
    gradient that reaches x beside the norm, is added) and ``weight`` (fp32)."""
    return _call(stream, _ops.block_norm_grad, d_h, x, weight, eps, d_add, workspace)


def block_merge(residual: torch.Tensor, y: torch.Tensor, weight: torch.Tensor, eps: float,
                gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                next_weight: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                h: Optional[torch.Tensor] = None, stream=None):
    """moe_block_merge: ``out = residual + scale * sigmoid(gate) * rms_norm(y) * weight``; with
    next_weight returns (out, h), ``h = rms_norm(out) * next_weight`` in bf16, else out alone.

    residual and out are bf16 or fp32 [tokens, H], y bf16 [tokens, H]; gate is None, one logit a token
    (bf16 [tokens]) or one an element (bf16 [tokens, H]); the weights are both bf16 or both fp32 [H]."""
    return _call(stream, _ops.block_merge, residual, y, weight, eps, gate, scale, next_weight, out, h)


def block_merge_grad(d_out: Optional[torch.Tensor], y: torch.Tensor, weight: torch.Tensor, eps: float,
                     gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                     next_weight: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     d_h: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> dict:
    """moe_block_merge_grad: the gradients of :func:`block_merge` as a dict: ``residual`` (in the
    stream's type), ``y`` and ``gate`` (bf16; gate only with one), ``weight`` and ``next_weight``
    (fp32; next_weight only with one).

    d_out is the gradient of out (None = 0, with a next norm only).  With next_weight, d_h (bf16) is
    the gradient of h and out the forward call's result."""
    return _call(stream, _ops.block_merge_grad, d_out, y, weight, eps, gate, scale, next_weight, out, d_h, workspace)


def block_forward(x: torch.Tensor, router_w: torch.Tensor, expert_w: torch.Tensor, shared_w: Optional[torch.Tensor],
                  top_k: int, norm_weight: Optional[torch.Tensor], merge_weight: torch.Tensor, eps: float,
                  gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                  next_weight: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None, stream=None,
                  out: Optional[torch.Tensor] = None, **layer):
    """A whole MoE block around :func:`sparse_moe_router_amd.forward`: the norm before it, the layer, and
    the merge after it: ``block_merge(x, forward(h, ...), merge_weight, ...)`` with ``h =
    block_norm(x, norm_weight)``, or the h that the block before gave (norm_weight is then None).

    x is the residual stream (bf16 or fp32 [tokens, H]); gate, scale, next_weight and out as in
    :func:`block_merge`, whose result is returned; other keywords go to ``forward``."""
    if (h is None) == (norm_weight is None):
        raise ValueError("either norm_weight or h must be given")
    if stream is None and x.is_cuda:
        stream = torch.cuda.current_stream(x.device)
    elif stream is not None:
        _same_device(stream, x, h)
    with torch.cuda.stream(stream):  # and its device
        if h is None:
            h = block_norm(x, norm_weight, eps)
        (M, H), E = h.shape, router_w.shape[0]
        if layer.get("workspace") is None:
            # of the call's own, as every workspace here: captured graphs never share one
            sizes = expert_w.numel() // (3 * E * H), 0 if shared_w is None else shared_w.numel() // (3 * H)
            layer["workspace"] = torch.empty(moe.workspace_size(M, H, E, *sizes, top_k, layer.get("flags", 0)),
                                             dtype=torch.uint8, device=h.device)
        # without rows there is nothing to route; torch's empty tensors have no address, which the layer refuses
        y = moe.forward(h, router_w, expert_w, shared_w, top_k, **layer) if M > 0 else torch.empty_like(h)
        return block_merge(x, y, merge_weight, eps, gate=gate, scale=scale, next_weight=next_weight, out=out)


# ------------------------------------------------------------------ gated feed-forward blocks

def gated_matmul(x: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor],
                 perm: Optional[torch.Tensor] = None, top_k: int = 1, save: bool = False,
                 out: Optional[torch.Tensor] = None, gate_up: Optional[torch.Tensor] = None, stream=None):
    """moe_gated_matmul: ``out[p] = silu(x[row(p)] @ w[e, :I].T) * (x[row(p)] @ w[e, I:].T)``, both
    projections, the activation and the product in one kernel.

    w bf16 [E, 2 I, K] (the gate's rows, then the up projection's); x, offsets, perm and rows as in
    :func:`grouped_matmul`.  Returns bf16 [rows, I]; with save (out, gate_up), gate_up bf16
    [rows, 2 I] the two products for :func:`gated_matmul_grad`."""
    return _call(stream, _ops.gated_matmul, x, w, offsets, perm, top_k, save, out, gate_up)


def gated_matmul_grad(dy: torch.Tensor, w: torch.Tensor, gate_up: torch.Tensor, offsets: Optional[torch.Tensor],
                      stream=None) -> dict:
    """moe_gated_matmul_grad: the gradient dy of the projection behind a gated product, ``y = h @ w[e].T``
    with w bf16 [E, H, I], through that projection, the product and the activation, as a dict:
    ``gate_up`` (bf16 [rows, 2 I]) and ``h`` (bf16 [rows, I], which the gradient of w needs)."""
    return _call(stream, _ops.gated_matmul_grad, dy, w, gate_up, offsets)


def feed_forward(x: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor, offsets: Optional[torch.Tensor],
                 perm: Optional[torch.Tensor] = None, top_k: int = 1, save: bool = False,
                 out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16, stream=None):
    """A gated feed-forward block of every expert: :func:`gated_matmul` with w_gate_up [E, 2 I, K], then
    :func:`grouped_matmul` with w_down [E, H, I].  Returns y [rows, H]; with save (y, gate_up)."""
    h = gated_matmul(x, w_gate_up, offsets, perm, top_k, save, stream=stream)
    h, gate_up = h if save else (h, None)
    y = grouped_matmul(h, w_down, offsets, out=out, out_dtype=out_dtype, stream=stream)
    return (y, gate_up) if save else y


def feed_forward_grad(dy: torch.Tensor, x: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor,
                      gate_up: torch.Tensor, offsets: Optional[torch.Tensor], perm: Optional[torch.Tensor] = None,
                      top_k: int = 1, dw_dtype: torch.dtype = torch.float32,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """moe_feed_forward_grad: the gradients of :func:`feed_forward` from dy (bf16 [rows, H]) and the gate_up
    that it saved, as a dict: ``x`` (bf16, of each grouped row: :func:`combine` with top_k sums a
    token's), ``w_gate_up`` and ``w_down`` (in dw_dtype; zeros for an expert without rows).  The
    gradient of gate_up and h are rounded to bf16 between the kernels, except in calls of few rows
    (include/moe_ops.h has the sizes and the errors)."""
    return _call(stream, _ops.feed_forward_grad, dy, x, w_gate_up, w_down, gate_up, offsets, perm, top_k,
                 _fp32(dw_dtype), workspace)


# ------------------------------------------------------------------ combine

def invert_permutation(perm: torch.Tensor, assignments: Optional[int] = None, offsets: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_invert_permutation: int32 [assignments] (as many as perm has rows, if not given) with
    ``inverse[perm[p]] = p``, -1 where no row has the assignment; rows from ``offsets[-1]`` on do not count."""
    return _call(stream, _ops.invert_permutation, perm, assignments, offsets, out)


def combine(y: torch.Tensor, inverse: torch.Tensor, top_k: int, weight: Optional[torch.Tensor] = None,
            add: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """moe_combine: ``out[t] = add[t] + sum_s weight[t, s] * y[inverse[t * top_k + s]]``: a token's output
    from its experts' rows, and without weight a token's gradient from its copies'.

    y bf16 [rows, H]; inverse as :func:`invert_permutation` gives it; weight fp32 [tokens, top_k]; add
    and out bf16 or fp32 [tokens, H]."""
    return _call(stream, _ops.combine, y, inverse, top_k, weight, add, out, _fp32(out_dtype))


def combine_grad(d_out: torch.Tensor, y: Optional[torch.Tensor], perm: torch.Tensor, inverse: torch.Tensor,
                 weight: Optional[torch.Tensor] = None, top_k: Optional[int] = None,
                 offsets: Optional[torch.Tensor] = None, dy: Optional[torch.Tensor] = None, stream=None) -> dict:
    """moe_combine_grad: the gradients of :func:`combine` as a dict: ``y`` (bf16 [rows, H], into dy if
    given) and, with weight, ``weight`` (fp32 [tokens, top_k]).  d_out is also the gradient of add.

    Rows from ``offsets[-1]`` on (with offsets) keep what dy held.  y is needed with weight, top_k
    without."""
    return _call(stream, _ops.combine_grad, d_out, y, perm, inverse, weight, top_k, offsets, dy)


# ------------------------------------------------------------------ clipping

def grad_norm(grads, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_grad_norm: the 2-norm of all elements of a list of gradients (bf16 or fp32, contiguous, any
    shapes), an fp32 tensor of no dimensions."""
    return _call_list(stream, grads, None, _ops.grad_norm, grads, workspace)


def clip_grads(grads, max_norm: float, norm: Optional[torch.Tensor] = None, eps: float = 1e-6, out=None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_clip_grads: every gradient times ``min(1, max_norm / (norm + eps))``, in place or into the list
    out (of the same shapes, bf16 or fp32).  Returns the norm: that of grads, computed by the call, or
    the given one (fp32, one element on the GPU), which holds the share of other devices, say."""
    return _call_list(stream, grads, out, _ops.clip_grads, grads, max_norm, norm, eps, out, workspace)


def _call_list(stream, grads, out, f, *args):
    if stream is not None:
        _same_device(stream, *(grads if isinstance(grads, (list, tuple)) else ()),
                     *(out if isinstance(out, (list, tuple)) else ()))
    return _call(stream, f, *args)


# ------------------------------------------------------------------ cross entropy

def cross_entropy(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """moe_cross_entropy: (loss, lse), fp32 [tokens] each, of the logits ``x @ w.T`` against targets (int64
    [tokens]), without keeping the logits: ``lse = logsumexp(logits)``, ``loss = lse - logits[target]``.

    x bf16 [tokens, H], w bf16 [V, H].  A token whose target is ignore_index or lies outside the
    vocabulary has loss 0 and no gradient."""
    return _call(stream, _ops.cross_entropy, x, w, targets, ignore_index, workspace)


def cross_entropy_grad(d_loss: torch.Tensor, x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor,
                       lse: torch.Tensor, ignore_index: int = -100, dx_dtype: Optional[torch.dtype] = torch.bfloat16,
                       dw_dtype: Optional[torch.dtype] = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                       stream=None) -> dict:
    """moe_cross_entropy_grad: the gradients of the loss of :func:`cross_entropy` as a dict ``x`` and ``w``
    (each in its dtype, left out where that is None), from d_loss (fp32 [tokens]) and the lse that the
    forward call gave.  The gradient of a logit is rounded to bf16 before the products, without d_loss;
    where the tokens' d_loss differ, so are the rows of x times their share of the largest one."""
    return _call(stream, _ops.cross_entropy_grad, d_loss, x, w, targets, lse, ignore_index,
                 None if dx_dtype is None else _fp32(dx_dtype), None if dw_dtype is None else _fp32(dw_dtype), workspace)
