"""Low-rank adapters of many requests at once beside a shared projection (bf16 / fp16):

    y[m] = base[m] + scales[l] b[l] (a[l] x[m]),  l = ids[m]

base [M, N] is the shared projection's output (grouped_matmul with one group, an expert projection,
any other), a [L, R, K] and b [L, N, R] the adapters, ids int32 [M] each row's adapter on the device
(outside [0, L): none).  Rows need not be sorted.  lora is differentiable in base, x, a and b;
lora_forward and lora_backward are the same calls without autograd.  Argument marshalling only.
"""
import ctypes
import functools
from dataclasses import dataclass

import torch

from . import _SIGS, _check, _dev_ptr, lib
from .matmul import (_DTYPES, _check_rows_out, _dtype16, _gs, _ld, _no_overlap, _packer, _row_major, _run, _same, _written,
                     once_differentiable)


class LoraWeights(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("lda", ctypes.c_int64), ("a_stride", ctypes.c_int64),
                ("b", ctypes.c_void_p), ("ldb", ctypes.c_int64), ("b_stride", ctypes.c_int64), ("scales", ctypes.c_void_p)]


class LoraSizes(ctypes.Structure):
    _fields_ = [("ctx_bytes", ctypes.c_size_t), ("fwd_ws_bytes", ctypes.c_size_t), ("bwd_ws_bytes", ctypes.c_size_t)]


class LoraFwdArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("R", ctypes.c_int32), ("L", ctypes.c_int32), ("M", ctypes.c_int64),
                ("K", ctypes.c_int64), ("N", ctypes.c_int64), ("base", ctypes.c_void_p), ("ldbase", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("w", LoraWeights), ("ids", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("ctx", ctypes.c_void_p), ("ctx_bytes", ctypes.c_size_t),
                ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t)]


class LoraBwdArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("R", ctypes.c_int32), ("L", ctypes.c_int32), ("M", ctypes.c_int64),
                ("K", ctypes.c_int64), ("N", ctypes.c_int64), ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("w", LoraWeights), ("dx_add", ctypes.c_void_p),
                ("lddx_add", ctypes.c_int64), ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64), ("da", ctypes.c_void_p),
                ("db", ctypes.c_void_p), ("ctx", ctypes.c_void_p), ("ctx_bytes", ctypes.c_size_t), ("ws", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_size_t)]


_SIGS.update({
    "gmlp_lora_query_sizes": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                             ctypes.c_int32, ctypes.POINTER(LoraSizes)]),
    "gmlp_lora_forward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),          # LoraFwdArgs*
    "gmlp_lora_backward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),         # LoraBwdArgs*
})
_pack_fwd, _pack_bwd = _packer(LoraFwdArgs), _packer(LoraBwdArgs)


@functools.lru_cache(maxsize=4096)
def _sizes(M, K, N, R, L):
    s = LoraSizes()
    _check(lib().gmlp_lora_query_sizes(M, K, N, R, L, ctypes.byref(s)))
    return s.ctx_bytes, s.fwd_ws_bytes, s.bwd_ws_bytes


def lora_query_sizes(M, K, N, R, L):
    return dict(zip(("ctx_bytes", "fwd_ws_bytes", "bwd_ws_bytes"), _sizes(M, K, N, R, L)))


@dataclass
class LoraContext:
    """What a forward leaves for the backward: the rows' order by adapter and u = a x (the sum of two
    16-bit values; fp16: in fp32 as well), opaque, and the call's sizes and scales."""
    buf: torch.Tensor
    M: int
    K: int
    N: int
    R: int
    L: int
    dtype: torch.dtype
    scales: torch.Tensor


def _check_weights(x, a, b, scales, what):
    _dtype16(x, what)
    if x.dim() != 2:
        raise ValueError(f"{what}: 2 dimensions expected, got {x.dim()}")
    _same(a, x, 3, "a")
    _same(b, x, 3, "b")
    L, R, K = a.shape
    N = b.shape[1]
    if tuple(b.shape) != (L, N, R):
        raise ValueError(f"b: [{L}, N, {R}] expected (a is {tuple(a.shape)}), got {tuple(b.shape)}")
    if scales is not None and (not isinstance(scales, torch.Tensor) or scales.dtype != torch.float32 or scales.numel() != L
                               or scales.device != x.device):
        raise TypeError(f"scales: an fp32 tensor of {L} elements on {x.device} is required")
    return L, R, K, N


def _ptr(t):
    return t.data_ptr() if t is not None else 0


def _weights(a, b, scales):
    return a.data_ptr(), _ld(a), _gs(a), b.data_ptr(), _ld(b), _gs(b), _ptr(scales)


def lora_forward(base, x, a, b, ids, scales=None, out=None):
    """(y, ctx): y [M, N] in x's dtype; ctx for lora_backward.  base may be None (zeros); out may be
    base itself (in place)."""
    L, R, K, N = _check_weights(x, a, b, scales, "x")
    M, dev = x.shape[0], x.device
    if x.shape[1] != K:
        raise ValueError(f"x: rows of {K} elements expected (a is {tuple(a.shape)}), got {x.shape[1]}")
    if not isinstance(ids, torch.Tensor) or ids.dtype != torch.int32 or tuple(ids.shape) != (M,):
        raise TypeError(f"ids: an int32 tensor of {M} elements is required")
    if ids.device != dev:
        raise ValueError(f"ids: on {ids.device}, the other tensors are on {dev}")
    if out is not None:
        _check_rows_out(out, (M, N), x, "out")
    if base is not None:
        _same(base, x, 2, "base")
        if tuple(base.shape) != (M, N):
            raise ValueError(f"base: shape {(M, N)} expected, got {tuple(base.shape)}")
        base = _row_major(base)
    if out is not None:
        _no_overlap(out, "out", x=x, a=a, b=b, ids=ids, scales=scales)
        if base is not None and (out.data_ptr() != base.data_ptr() or _ld(out) != _ld(base)):
            _no_overlap(out, "out", base=base)
    _dev_ptr(x, "x")
    x, a, b, ids = _row_major(x), _row_major(a), _row_major(b), ids.contiguous()
    scales = scales.contiguous() if scales is not None else None
    ctx_bytes, ws_bytes, _ = _sizes(M, K, N, R, L)
    y = out if out is not None else torch.empty((M, N), dtype=x.dtype, device=dev)
    # one allocation: the workspace lies behind the context
    at = (ctx_bytes + 255) // 256 * 256
    buf = torch.empty(at + ws_bytes, dtype=torch.uint8, device=dev)
    p = buf.data_ptr()
    args = _pack_fwd(_DTYPES[x.dtype], R, L, M, K, N, _ptr(base), _ld(base) if base is not None else 0, x.data_ptr(), _ld(x),
                     *_weights(a, b, scales), ids.data_ptr(), y.data_ptr(), _ld(y), p, ctx_bytes, p + at, ws_bytes)
    _run(lib().gmlp_lora_forward, args, dev)
    if out is not None:
        _written(out)
    return y, LoraContext(buf, M, K, N, R, L, x.dtype, scales)


def lora_backward(dy, x, a, b, ctx, dx_add=None, need_dx=True, need_da=True, need_db=True):
    """{"dx" [M, K], "da" [L, R, K], "db" [L, N, R]} (None where not needed) from the gradient of y and
    the forward's x, a, b and ctx.  dx_add: added to dx in the same pass (the shared projection's dx).
    The gradient for base is dy itself."""
    if not isinstance(ctx, LoraContext):
        raise TypeError("ctx: the LoraContext of a lora_forward is required")
    L, R, K, N = _check_weights(dy, a, b, ctx.scales, "dy")
    M, dev = ctx.M, dy.device
    if (L, R, K, N, dy.dtype) != (ctx.L, ctx.R, ctx.K, ctx.N, ctx.dtype):
        raise ValueError("ctx: written by a forward of other sizes or another dtype")
    if tuple(dy.shape) != (M, N):
        raise ValueError(f"dy: shape {(M, N)} expected, got {tuple(dy.shape)}")
    _same(x, dy, 2, "x")
    if tuple(x.shape) != (M, K):
        raise ValueError(f"x: shape {(M, K)} expected, got {tuple(x.shape)}")
    ctx_bytes, _, ws_bytes = _sizes(M, K, N, R, L)
    if ctx.buf.device != dev:
        raise ValueError(f"ctx: on {ctx.buf.device}, the other tensors are on {dev}")
    if not ctx.buf.is_contiguous() or ctx.buf.numel() * ctx.buf.element_size() < ctx_bytes:
        raise ValueError(f"ctx: a contiguous buffer of at least {ctx_bytes} bytes is required, got {ctx.buf.numel() * ctx.buf.element_size()}")
    if dx_add is not None:
        _same(dx_add, dy, 2, "dx_add")
        if tuple(dx_add.shape) != (M, K):
            raise ValueError(f"dx_add: shape {(M, K)} expected, got {tuple(dx_add.shape)}")
        dx_add = _row_major(dx_add)
    _dev_ptr(dy, "dy")
    dy, x, a, b = _row_major(dy), _row_major(x), _row_major(a), _row_major(b)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    dx = torch.empty((M, K), dtype=dy.dtype, device=dev) if need_dx else None
    da = torch.empty((L, R, K), dtype=dy.dtype, device=dev) if need_da else None
    db = torch.empty((L, N, R), dtype=dy.dtype, device=dev) if need_db else None
    args = _pack_bwd(_DTYPES[dy.dtype], R, L, M, K, N, dy.data_ptr(), _ld(dy), x.data_ptr(), _ld(x),
                     *_weights(a, b, ctx.scales), _ptr(dx_add), _ld(dx_add) if dx_add is not None else 0, _ptr(dx), K,
                     _ptr(da), _ptr(db), ctx.buf.data_ptr(), ctx_bytes, ws.data_ptr(), ws_bytes)
    _run(lib().gmlp_lora_backward, args, dev)
    return {"dx": dx, "da": da, "db": db}


class LoraFunction(torch.autograd.Function):
    @staticmethod
    def forward(fctx, base, x, a, b, ids, scales):
        y, c = lora_forward(base, x, a, b, ids, scales)
        fctx.lora = (c.M, c.K, c.N, c.R, c.L, c.dtype)
        fctx.save_for_backward(x, a, b, scales, c.buf)
        return y

    @staticmethod
    @once_differentiable
    def backward(fctx, dy):
        x, a, b, scales, buf = fctx.saved_tensors
        need = fctx.needs_input_grad
        dyt = dy.to(x.dtype)
        g = {"dx": None, "da": None, "db": None}
        if need[1] or need[2] or need[3]:
            ctx = LoraContext(buf, *fctx.lora, scales.contiguous() if scales is not None else None)
            g = lora_backward(dyt, x, a, b, ctx, need_dx=need[1], need_da=need[2], need_db=need[3])
        return dyt if need[0] else None, g["dx"], g["da"], g["db"], None, None


def lora(base, x, a, b, ids, scales=None):
    """lora_forward under torch.autograd: gradients for base, x, a and b (scales are constants)."""
    if scales is not None and isinstance(scales, torch.Tensor) and scales.requires_grad:
        raise ValueError("scales: no gradient is computed for the scales")
    return LoraFunction.apply(base, x, a, b, ids, scales)
