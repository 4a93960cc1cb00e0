"""Python binding of the operators in ``include/moe_ops.h``: products grouped by
expert with their gradients, 8-bit products, and the norms around a block.

Argument marshalling only, as in :mod:`.moe`: torch tensors provide device
memory and the stream, every step runs in the library's HIP kernels, and a
tensor that the kernels cannot take raises.  Activations (``x``, ``y``, ``dy``,
``residual``, ``gate`` ...) are matrices whose rows are contiguous; their rows
may be strided (a slice of columns), by a multiple of 16 bytes.  Weights,
offsets, permutations and per-token vectors are contiguous.  Results are
allocated on the call's stream unless the caller passes them.

``offsets`` (int32 [E+1]) and ``perm`` (int32 [rows]) are the group offsets and
the permutation that :func:`sparse_moe_router_amd.route` reports.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import moe
from .moe import MoeError

EXPORTS = ("moe_grouped_matmul", "moe_grouped_matmul_grad_input", "moe_grouped_matmul_grad_weight",
           "moe_quantize_i8", "moe_matmul_i8_workspace_size", "moe_matmul_i8", "moe_block_norm",
           "moe_block_norm_grad", "moe_block_merge", "moe_block_merge_grad", "moe_norm_grad_workspace_size")

_BF16, _F32, _I8, _I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32
_DTYPE = {_BF16: 0, _F32: 1}  # moe_dtype_t


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


_NONE = MoeMat(None, 0)


_bound = None


def lib() -> ctypes.CDLL:
    """The loaded library with this module's entry points declared (raises if it has not been built)."""
    global _bound
    if _bound is None:
        L = moe.lib()
        vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
        g, n, en = ctypes.POINTER(MoeGroups), ctypes.POINTER(MoeNorm), ctypes.c_int
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
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _bound = L
    return _bound


# ------------------------------------------------------------------ argument checks

def _tensor(t, dtypes, dims, name, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call on {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimension(s), got {tuple(t.shape)}")
    return t


def _flat(t, dtypes, shape, name, device):
    """A contiguous tensor of exactly this shape."""
    _tensor(t, dtypes, len(shape), name, device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _rows(t, dtypes, cols, name, device, rows=None):
    """A matrix with contiguous rows; returns its row stride in elements."""
    _tensor(t, dtypes, 2, name, device)
    if t.shape[1] != cols or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} must have shape ({'rows' if rows is None else rows}, {cols}), got {tuple(t.shape)}")
    if t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    # a matrix of one row (or none) has no row stride of its own
    ld = t.stride(0) if t.shape[0] > 1 else cols
    if ld < cols:
        raise ValueError(f"{name} must not have overlapping rows")
    return ld


class _Call:
    """The device and stream of one call: the tensors' device is current while it lasts, and what it
    allocates belongs to its stream."""

    __slots__ = ("device", "stream", "_outer", "_ctx")

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        self.device, self._ctx = device, None
        self._outer = stream
        self.stream = None

    def __enter__(self):
        if self._outer is not None:
            self._ctx = torch.cuda.stream(self._outer)  # sets the device too
            self._ctx.__enter__()
            self.stream = self._outer.cuda_stream
        else:
            if torch.cuda.current_device() != self.device.index:
                self._ctx = torch.cuda.device(self.device)
                self._ctx.__enter__()
            self.stream = torch.cuda.current_stream(self.device).cuda_stream
        return self

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)
        return False

    def empty(self, *shape, dtype):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def workspace(self, given, nbytes):
        # a buffer of the call's own: calls on different streams, and captured graphs, never share one
        if given is None:
            return torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        _flat(given, (torch.uint8,), (given.numel(),), "workspace", self.device)
        return given


def _check(st, what):
    if st != 0:
        moe._check(st, what)


def _p(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ grouped products

def _groups(w_shape, offsets, perm, top_k, rows, x_rows, ldx, ldy, dev) -> MoeGroups:
    E, N, K = w_shape
    if offsets is None:
        if E != 1:
            raise ValueError("offsets may be left out with one expert only")
    else:
        _flat(offsets, (_I32,), (E + 1,), "offsets", dev)
    if perm is not None:
        _flat(perm, (_I32,), (rows,), "perm", dev)
    return MoeGroups(rows, x_rows, ldx, ldy, E, N, K, int(top_k), _p(offsets), _p(perm))


def _forward_rows(x, perm, out):
    return out.shape[0] if out is not None else perm.shape[0] if perm is not None else x.shape[0]


def grouped_matmul(x: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor],
                   perm: Optional[torch.Tensor] = None, top_k: int = 1, out: Optional[torch.Tensor] = None,
                   out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """moe_grouped_matmul: ``out[p] = x[row(p)] @ w[e].T`` for the rows p of each expert's group.

    x bf16 [tokens, K]; w bf16 [E, N, K]; row(p) is ``perm[p] // top_k`` with a permutation, else p.
    Returns out [rows, N] (bf16 or fp32), rows = those of ``perm``, else of x; rows from
    ``offsets[E]`` on keep what ``out`` held (an allocated ``out`` is not cleared)."""
    dev = _tensor(x, (_BF16,), 2, "x", None).device
    _tensor(w, (_BF16,), 3, "w", dev)
    E, N, K = w.shape
    _flat(w, (_BF16,), (E, N, K), "w", dev)
    ldx = _rows(x, (_BF16,), K, "x", dev)
    with _Call(dev, stream) as c:
        if out is None:
            out = c.empty(_forward_rows(x, perm, None), N, dtype=out_dtype)
        ldy = _rows(out, (_BF16, _F32), N, "out", dev)
        g = _groups((E, N, K), offsets, perm, top_k, out.shape[0], x.shape[0], ldx, ldy, dev)
        _check(lib().moe_grouped_matmul(ctypes.byref(g), x.data_ptr(), w.data_ptr(), out.data_ptr(),
                                        _DTYPE[out.dtype], c.stream), "moe_grouped_matmul")
    return out


def grouped_matmul_grad_input(dy: torch.Tensor, w: torch.Tensor, offsets: Optional[torch.Tensor],
                              out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                              stream=None) -> torch.Tensor:
    """moe_grouped_matmul_grad_input: ``out[p] = dy[p] @ w[e]``, the gradient of each grouped row
    (with a permutation, of the row's own copy of its token)."""
    dev = _tensor(dy, (_BF16,), 2, "dy", None).device
    _tensor(w, (_BF16,), 3, "w", dev)
    E, N, K = w.shape
    _flat(w, (_BF16,), (E, N, K), "w", dev)
    ldy = _rows(dy, (_BF16,), N, "dy", dev)
    rows = dy.shape[0]
    with _Call(dev, stream) as c:
        if out is None:
            out = c.empty(rows, K, dtype=out_dtype)
        ldx = _rows(out, (_BF16, _F32), K, "out", dev, rows)
        g = _groups((E, N, K), offsets, None, 1, rows, rows, ldx, ldy, dev)
        _check(lib().moe_grouped_matmul_grad_input(ctypes.byref(g), dy.data_ptr(), w.data_ptr(), out.data_ptr(),
                                                   _DTYPE[out.dtype], c.stream), "moe_grouped_matmul_grad_input")
    return out


def grouped_matmul_grad_weight(x: torch.Tensor, dy: torch.Tensor, offsets: Optional[torch.Tensor],
                               perm: Optional[torch.Tensor] = None, top_k: int = 1,
                               out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.float32,
                               stream=None) -> torch.Tensor:
    """moe_grouped_matmul_grad_weight: ``out[e] = sum_p dy[p].T x[row(p)]`` over each expert's rows,
    [E, N, K] in fp32 or bf16; zeros for an expert without rows."""
    dev = _tensor(x, (_BF16,), 2, "x", None).device
    _tensor(dy, (_BF16,), 2, "dy", dev)
    E = 1 if offsets is None else _tensor(offsets, (_I32,), 1, "offsets", dev).shape[0] - 1
    K, N = x.shape[1], dy.shape[1]
    ldx, ldy = _rows(x, (_BF16,), K, "x", dev), _rows(dy, (_BF16,), N, "dy", dev)
    with _Call(dev, stream) as c:
        if out is None:
            out = c.empty(E, N, K, dtype=out_dtype)
        _flat(out, (_BF16, _F32), (E, N, K), "out", dev)
        g = _groups((E, N, K), offsets, perm, top_k, dy.shape[0], x.shape[0], ldx, ldy, dev)
        _check(lib().moe_grouped_matmul_grad_weight(ctypes.byref(g), x.data_ptr(), dy.data_ptr(), out.data_ptr(),
                                                    _DTYPE[out.dtype], c.stream), "moe_grouped_matmul_grad_weight")
    return out


# ------------------------------------------------------------------ 8-bit products

def quantize_i8(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                stream=None):
    """moe_quantize_i8: (codes int8 [tokens, K], scale fp32 [tokens]) of bf16 rows,
    ``codes = rint(127 x / max|x|)``, ``scale = max|x| / 127``."""
    dev = _tensor(x, (_BF16,), 2, "x", None).device
    M, K = x.shape
    ldx = _rows(x, (_BF16,), K, "x", dev)
    with _Call(dev, stream) as c:
        codes = c.empty(M, K, dtype=_I8) if codes is None else _flat(codes, (_I8,), (M, K), "codes", dev)
        scale = c.empty(M, dtype=_F32) if scale is None else _flat(scale, (_F32,), (M,), "scale", dev)
        _check(lib().moe_quantize_i8(M, K, ldx, x.data_ptr(), codes.data_ptr(), scale.data_ptr(), c.stream),
               "moe_quantize_i8")
    return codes, scale


def _matmul_i8(x, w, w_scale, offsets, perm, top_k, x_scale, bias, out, out_dtype, workspace, stream):
    dev = _tensor(x, (_BF16, _I8), 2, "x", None).device
    if (x.dtype == _I8) != (x_scale is not None):
        raise ValueError("x is either bf16, quantised by the call, or int8 codes with x_scale")
    E, N, K = w.shape
    _flat(w, (_I8,), (E, N, K), "w", dev)
    ldx = _rows(x, (x.dtype,), K, "x", dev)
    if x_scale is not None:
        _flat(x_scale, (_F32,), (x.shape[0],), "x_scale", dev)
    if bias is not None:
        _flat(bias, (_F32,), (N,), "bias", dev)
    with _Call(dev, stream) as c:
        if out is None:
            out = c.empty(_forward_rows(x, perm, None), N, dtype=out_dtype)
        ldy = _rows(out, (_BF16, _F32), N, "out", dev)
        g = _groups((E, N, K), offsets, perm, top_k, out.shape[0], x.shape[0], ldx, ldy, dev)
        ws, nbytes = None, 0
        if x_scale is None:
            ws = c.workspace(workspace, lib().moe_matmul_i8_workspace_size(ctypes.byref(g)))
            nbytes = ws.numel()
        _check(lib().moe_matmul_i8(ctypes.byref(g), x.data_ptr(), _p(x_scale), w.data_ptr(), w_scale.data_ptr(),
                                   _p(bias), out.data_ptr(), _DTYPE[out.dtype], _p(ws), nbytes, c.stream),
               "moe_matmul_i8")
    return out


def matmul_i8(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, x_scale: Optional[torch.Tensor] = None,
              bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              out_dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """moe_matmul_i8 with one weight matrix: ``out = (q @ w.T) * x_scale[:, None] * w_scale (+ bias)``.

    w int8 [N, K], w_scale fp32 [N], bias fp32 [N] or None.  x is bf16 [tokens, K] (quantised by the
    call as :func:`quantize_i8` does) or int8 codes with x_scale fp32 [tokens].  The integer sums are
    exact; out is bf16 or fp32."""
    dev = _tensor(x, (_BF16, _I8), 2, "x", None).device
    _tensor(w, (_I8,), 2, "w", dev)
    _flat(w_scale, (_F32,), (w.shape[0],), "w_scale", dev)
    if out is not None:
        _rows(out, (_BF16, _F32), w.shape[0], "out", dev, x.shape[0])
    return _matmul_i8(x, w.unsqueeze(0), w_scale, None, None, 1, x_scale, bias, out, out_dtype, workspace, stream)


def grouped_matmul_i8(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, offsets: Optional[torch.Tensor],
                      perm: Optional[torch.Tensor] = None, top_k: int = 1, x_scale: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_matmul_i8 grouped by expert: :func:`grouped_matmul` on int8 weights w [E, N, K] with
    w_scale fp32 [E, N]; x as in :func:`matmul_i8`."""
    dev = _tensor(x, (_BF16, _I8), 2, "x", None).device
    _tensor(w, (_I8,), 3, "w", dev)
    _flat(w_scale, (_F32,), tuple(w.shape[:2]), "w_scale", dev)
    return _matmul_i8(x, w, w_scale, offsets, perm, top_k, x_scale, None, out, out_dtype, workspace, stream)


# ------------------------------------------------------------------ block norms

def _mat(t, dtypes, rows, H, name, dev) -> MoeMat:
    return _NONE if t is None else MoeMat(t.data_ptr(), _rows(t, dtypes, H, name, dev, rows))


def _gate(gate, rows, H, name, dev):
    """(moe_gate_t, matrix) of a gate tensor or its gradient."""
    if gate is None:
        return 0, _NONE
    if isinstance(gate, torch.Tensor) and gate.dim() == 1:
        return 1, MoeMat(_flat(gate, (_BF16,), (rows,), name, dev).data_ptr(), 0)
    return 2, _mat(gate, (_BF16,), rows, H, name, dev)


def _weight(w, H, name, dev, dtypes=(_BF16, _F32)):
    return None if w is None else _flat(w, dtypes, (H,), name, dev).data_ptr()


def block_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """moe_block_norm: ``x * rsqrt(mean(x^2) + eps) * weight`` in bf16; x bf16 or fp32 [tokens, H],
    weight bf16 or fp32 [H]."""
    dev = _tensor(x, (_BF16, _F32), 2, "x", None).device
    M, H = x.shape
    wp = _weight(weight, H, "weight", dev)
    with _Call(dev, stream) as c:
        if out is None:
            out = c.empty(M, H, dtype=_BF16)
        d = MoeNorm(M, H, _DTYPE[x.dtype], _DTYPE[weight.dtype], 0, eps, 1.0)
        _check(lib().moe_block_norm(ctypes.byref(d), _mat(x, (x.dtype,), M, H, "x", dev), wp,
                                    _mat(out, (_BF16,), M, H, "out", dev), c.stream), "moe_block_norm")
    return out


def block_norm_grad(d_h: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, eps: float,
                    d_add: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> dict:
    """moe_block_norm_grad: the gradients of :func:`block_norm` as a dict: ``x`` (in x's type; d_add, the
    gradient that reaches x beside the norm, is added) and ``weight`` (fp32)."""
    dev = _tensor(x, (_BF16, _F32), 2, "x", None).device
    M, H = x.shape
    wp = _weight(weight, H, "weight", dev)
    with _Call(dev, stream) as c:
        dx, dw = c.empty(M, H, dtype=x.dtype), c.empty(H, dtype=_F32)
        d = MoeNorm(M, H, _DTYPE[x.dtype], _DTYPE[weight.dtype], 0, eps, 1.0)
        ws = c.workspace(workspace, lib().moe_norm_grad_workspace_size(ctypes.byref(d)))
        _check(lib().moe_block_norm_grad(ctypes.byref(d), _mat(d_h, (_BF16,), M, H, "d_h", dev),
                                         _mat(x, (x.dtype,), M, H, "x", dev), wp,
                                         _mat(d_add, (x.dtype,), M, H, "d_add", dev), MoeMat(dx.data_ptr(), H),
                                         dw.data_ptr(), ws.data_ptr(), ws.numel(), c.stream), "moe_block_norm_grad")
    return dict(x=dx, weight=dw)


def block_merge(residual: torch.Tensor, y: torch.Tensor, weight: torch.Tensor, eps: float,
                gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                next_weight: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                h: Optional[torch.Tensor] = None, stream=None):
    """moe_block_merge: ``out = residual + scale * sigmoid(gate) * rms_norm(y) * weight``; with
    next_weight returns (out, h), ``h = rms_norm(out) * next_weight`` in bf16, else out alone.

    residual and out are bf16 or fp32 [tokens, H], y bf16 [tokens, H]; gate is None, one logit a token
    (bf16 [tokens]) or one an element (bf16 [tokens, H]); the weights are both bf16 or both fp32 [H]."""
    dev = _tensor(residual, (_BF16, _F32), 2, "residual", None).device
    M, H = residual.shape
    st = (residual.dtype,)
    wp = _weight(weight, H, "weight", dev)
    wn = _weight(next_weight, H, "next_weight", dev, (weight.dtype,))
    mode, gm = _gate(gate, M, H, "gate", dev)
    if next_weight is None and h is not None:
        raise ValueError("h needs next_weight")
    with _Call(dev, stream) as c:
        if out is None:
            out = c.empty(M, H, dtype=residual.dtype)
        if next_weight is not None and h is None:
            h = c.empty(M, H, dtype=_BF16)
        d = MoeNorm(M, H, _DTYPE[residual.dtype], _DTYPE[weight.dtype], mode, eps, scale)
        _check(lib().moe_block_merge(ctypes.byref(d), _mat(residual, st, M, H, "residual", dev),
                                     _mat(y, (_BF16,), M, H, "y", dev), wp, gm, wn, _mat(out, st, M, H, "out", dev),
                                     _mat(h, (_BF16,), M, H, "h", dev), c.stream), "moe_block_merge")
    return out if next_weight is None else (out, h)


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
    dev = _tensor(y, (_BF16,), 2, "y", None).device
    M, H = y.shape
    if (next_weight is None) != (d_h is None) or (next_weight is None) != (out is None):
        raise ValueError("next_weight, out and d_h are given together")
    ref = d_out if d_out is not None else out
    if ref is None:
        raise ValueError("d_out or d_h must be given")
    st = (_tensor(ref, (_BF16, _F32), 2, "d_out" if d_out is not None else "out", dev).dtype,)
    wp = _weight(weight, H, "weight", dev)
    wn = _weight(next_weight, H, "next_weight", dev, (weight.dtype,))
    mode, gm = _gate(gate, M, H, "gate", dev)
    with _Call(dev, stream) as c:
        res = dict(residual=c.empty(M, H, dtype=st[0]), y=c.empty(M, H, dtype=_BF16), weight=c.empty(H, dtype=_F32))
        if mode:
            res["gate"] = c.empty(*gate.shape, dtype=_BF16)
        if next_weight is not None:
            res["next_weight"] = c.empty(H, dtype=_F32)
        d = MoeNorm(M, H, _DTYPE[st[0]], _DTYPE[weight.dtype], mode, eps, scale)
        ws = c.workspace(workspace, lib().moe_norm_grad_workspace_size(ctypes.byref(d)))
        _check(lib().moe_block_merge_grad(
            ctypes.byref(d), _mat(d_out, st, M, H, "d_out", dev), _mat(d_h, (_BF16,), M, H, "d_h", dev),
            _mat(y, (_BF16,), M, H, "y", dev), wp, gm, _mat(out, st, M, H, "out", dev), wn,
            MoeMat(res["residual"].data_ptr(), H), MoeMat(res["y"].data_ptr(), H),
            MoeMat(_p(res.get("gate")), H), res["weight"].data_ptr(), _p(res.get("next_weight")), ws.data_ptr(),
            ws.numel(), c.stream), "moe_block_merge_grad")
    return res
