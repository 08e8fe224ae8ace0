"""Grouped products on bf16 / fp16 tensors whose rows are grouped by expert (no quantization):

    grouped_matmul_forward  y[r, :]  = x[r, :] w[g]^T         x [M, K], w [G, N, K]
    grouped_matmul_dgrad    dx[r, :] = dy[r, :] w[g]
    grouped_matmul_wgrad    dw[g]    = dy_g^T x_g             w's dtype, fp32, or added to an fp32 main_grad
    grouped_matmul          the three under torch.autograd

g is the group of row r by m_splits (int32 [G] on the device), products are accumulated in fp32
and rounded once.  Argument marshalling only; the kernels are the library's.
"""
import ctypes
import functools
import struct

import torch
from torch.autograd.function import once_differentiable

from . import (_SIGS, _check, _check_out, _dev_ptr, _splits, GEMM_DGRAD, GEMM_FPROP, GEMM_WGRAD, OUT_FP32,
               OUT_FP32_ACCUMULATE, lib)

OUT_SAME = 0                   # the operands' type
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class GroupedMatmulArgs(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("zero_rest", ctypes.c_int32), ("a", ctypes.c_void_p), ("lda", ctypes.c_int64),
                ("b", ctypes.c_void_p), ("ldb", ctypes.c_int64), ("b_stride", ctypes.c_int64),
                ("c", ctypes.c_void_p), ("ldc", ctypes.c_int64), ("c_stride", ctypes.c_int64),
                ("m_splits", ctypes.c_void_p), ("G", ctypes.c_int32), ("M", ctypes.c_int64), ("n", ctypes.c_int64),
                ("k", ctypes.c_int64), ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t)]


_CODES = {ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_void_p: "P", ctypes.c_size_t: "N"}


def _packer(cls):
    """pack(field values in order) -> the bytes of a ctypes structure (nested ones flattened): a
    decode step's calls spend most of their host time in filling ctypes fields one by one."""
    def codes(c):
        return "".join(codes(t) if issubclass(t, ctypes.Structure) else _CODES[t] for _, t in c._fields_)
    pk = struct.Struct("@" + codes(cls) + "0P")
    assert pk.size == ctypes.sizeof(cls), cls
    return pk.pack


_SIGS.update({
    "gmlp_grouped_matmul_ws_bytes": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64,
                                                    ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)]),
    "gmlp_grouped_matmul": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),       # GroupedMatmulArgs*
})
_pack_mm = _packer(GroupedMatmulArgs)


def _run(fn, args, device):
    """One library call with packed arguments on the device's current stream."""
    i = device.index
    if i == torch._C._cuda_getDevice():
        _check(fn(args, torch._C._cuda_getCurrentRawStream(i)))
    else:
        with torch.cuda.device(i):
            _check(fn(args, torch._C._cuda_getCurrentRawStream(i)))


def _dtype16(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise TypeError(f"{name}: a bf16 or fp16 tensor is required, got {getattr(t, 'dtype', type(t).__name__)}")
    return _DTYPES[t.dtype]


def _same(t, ref, dim, name):
    """t: a tensor of ref's dtype, on ref's device, of `dim` dimensions."""
    if not isinstance(t, torch.Tensor) or t.dtype != ref.dtype:
        raise TypeError(f"{name}: a {ref.dtype} tensor is required, got {getattr(t, 'dtype', type(t).__name__)}")
    if t.device != ref.device:
        raise ValueError(f"{name}: on {t.device}, the other tensors are on {ref.device}")
    if t.dim() != dim:
        raise ValueError(f"{name}: {dim} dimensions expected, got {t.dim()}")


def _row_major(t):
    """t with its last dimension contiguous and rows that do not overlap (a copy if it is not so)."""
    if t.is_contiguous():
        return t
    ok = t.shape[-1] <= 1 or t.stride(-1) == 1
    need = t.shape[-1]
    for d in range(t.dim() - 2, -1, -1):
        if t.shape[d] > 1 and t.stride(d) < need:
            ok = False
        if t.shape[d] > 1:
            need = t.stride(d) * (t.shape[d] - 1) + need
    if ok and t.dim() >= 2 and t.shape[-2] > 1 and t.stride(-2) >= 1 << 20:
        ok = False
    return t if ok else t.contiguous()


def _ld(t):
    """Row stride of a _row_major tensor (the row's length where there is at most one row)."""
    return t.stride(-2) if t.shape[-2] > 1 else t.shape[-1]


def _gs(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * _ld(t)


def _extent(t):
    """(first byte, byte behind the last) of a tensor's elements."""
    n = sum((t.shape[d] - 1) * t.stride(d) for d in range(t.dim())) + 1
    return t.data_ptr(), t.data_ptr() + n * t.element_size()


def _no_overlap(out, name, /, **inputs):
    """An output must not share elements with what the call reads while it is written (columns of one
    wide tensor beside each other are fine)."""
    if out.numel() == 0:
        return
    o0, o1 = _extent(out)
    for k, t in inputs.items():
        if t is None or t.numel() == 0:
            continue
        i0, i1 = _extent(t)
        if o0 >= i1 or i0 >= o1:
            continue
        if out.dim() == 2 == t.dim() and out.element_size() == t.element_size() and _ld(out) == _ld(t):
            es, ld = t.element_size(), _ld(t)
            if (o0 - i0) % es == 0:
                d = (o0 - i0) // es % ld
                if d >= t.shape[1] and d + out.shape[1] <= ld:
                    continue
        raise ValueError(f"{name}: overlaps {k}")


def _check_rows_out(t, shape, like, name):
    """A given output: like's dtype and device, the shape, last dimension contiguous, rows apart."""
    if not isinstance(t, torch.Tensor) or tuple(t.shape) != tuple(shape) or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name}: a {like.dtype} tensor of shape {tuple(shape)} on {like.device} is required")
    if _row_major(t) is not t:
        raise ValueError(f"{name}: the last dimension must be contiguous and rows must not overlap")


def _written(t):
    """A tensor of the caller's was written by its address: its version is raised, as an in-place torch
    operation would, so that the backward of a node that saved it raises.  Returns t."""
    torch.autograd.graph.increment_version(t)
    return t


@functools.lru_cache(maxsize=4096)
def grouped_matmul_ws_bytes(layout, G, M, n, k):
    v = ctypes.c_size_t(0)
    _check(lib().gmlp_grouped_matmul_ws_bytes(layout, G, M, n, k, ctypes.byref(v)))
    return v.value


def _call(layout, a, b, c, m_splits, M, n, k, out_dtype, zero_rest, ws):
    dev = a.device
    G = m_splits.numel()
    if m_splits.device != dev:
        raise ValueError(f"m_splits: on {m_splits.device}, the other tensors are on {dev}")
    if ws is not None:
        if not isinstance(ws, torch.Tensor) or ws.device != dev or not ws.is_contiguous():
            raise ValueError(f"ws: a contiguous tensor on {dev} is required")
        # the kernels address what the tables in it say
        _no_overlap(ws, "ws", out=c, m_splits=m_splits, **{"x" if layout == GEMM_FPROP else "dy": a,
                                                           "x" if layout == GEMM_WGRAD else "w": b})
    if dev.type != "cuda":
        _dev_ptr(a, "dy" if layout != GEMM_FPROP else "x")          # refuses host tensors
    if ws is None:
        ws = torch.empty(grouped_matmul_ws_bytes(layout, G, M, n, k), dtype=torch.uint8, device=dev)
    wgrad = layout == GEMM_WGRAD
    args = _pack_mm(layout, _DTYPES[a.dtype], out_dtype, zero_rest, a.data_ptr(), _ld(a), b.data_ptr(), _ld(b),
                    0 if wgrad else _gs(b), c.data_ptr(), _ld(c), _gs(c) if wgrad else 0, m_splits.data_ptr(), G, M, n, k,
                    ws.data_ptr(), ws.numel() * ws.element_size())
    _run(lib().gmlp_grouped_matmul, args, dev)


def grouped_matmul_forward(x, w, m_splits, out=None, ws=None):
    """y [M, N] = x [M, K] times each group's w[g] [N, K] transposed, in x's dtype.  Rows behind the
    last group (splits that sum short of M) are zero in a new output and left as they are in `out`."""
    _dtype16(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x: 2 dimensions expected, got {x.dim()}")
    _same(w, x, 3, "w")
    G, N, K = w.shape
    if x.shape[1] != K:
        raise ValueError(f"x: rows of {K} elements expected (w is {tuple(w.shape)}), got {x.shape[1]}")
    m_splits = _splits(m_splits, G)
    if out is not None:
        _check_rows_out(out, (x.shape[0], N), x, "out")
        _no_overlap(out, "out", x=x, w=w, m_splits=m_splits)
    y = out if out is not None else torch.empty((x.shape[0], N), dtype=x.dtype, device=x.device)
    _call(GEMM_FPROP, _row_major(x), _row_major(w), y, m_splits, x.shape[0], N, K, OUT_SAME, out is None, ws)
    return y if out is None else _written(out)


def grouped_matmul_dgrad(dy, w, m_splits, out=None, ws=None):
    """dx [M, K] = dy [M, N] times each group's w[g] [N, K], in dy's dtype (rows as in the forward)."""
    _dtype16(dy, "dy")
    if dy.dim() != 2:
        raise ValueError(f"dy: 2 dimensions expected, got {dy.dim()}")
    _same(w, dy, 3, "w")
    G, N, K = w.shape
    if dy.shape[1] != N:
        raise ValueError(f"dy: rows of {N} elements expected (w is {tuple(w.shape)}), got {dy.shape[1]}")
    m_splits = _splits(m_splits, G)
    if out is not None:
        _check_rows_out(out, (dy.shape[0], K), dy, "out")
        _no_overlap(out, "out", dy=dy, w=w, m_splits=m_splits)
    dx = out if out is not None else torch.empty((dy.shape[0], K), dtype=dy.dtype, device=dy.device)
    _call(GEMM_DGRAD, _row_major(dy), _row_major(w), dx, m_splits, dy.shape[0], K, N, OUT_SAME, out is None, ws)
    return dx if out is None else _written(out)


def grouped_matmul_wgrad(dy, x, m_splits, out_dtype=OUT_SAME, out=None, ws=None):
    """dw [G, N, K]: dy_g^T x_g of every group, in dy's dtype, fp32 (OUT_FP32), or added in fp32 to
    `out` (OUT_FP32_ACCUMULATE).  An empty group's slice is zero, or left as it is when accumulating."""
    _dtype16(dy, "dy")
    if dy.dim() != 2:
        raise ValueError(f"dy: 2 dimensions expected, got {dy.dim()}")
    _same(x, dy, 2, "x")
    if x.shape[0] != dy.shape[0]:
        raise ValueError(f"x: {dy.shape[0]} rows expected, got {x.shape[0]}")
    m_splits = _splits(m_splits)
    if out_dtype not in (OUT_SAME, OUT_FP32, OUT_FP32_ACCUMULATE):
        raise ValueError(f"out_dtype: unknown value {out_dtype}")
    shape = (m_splits.numel(), dy.shape[1], x.shape[1])
    dt = dy.dtype if out_dtype == OUT_SAME else torch.float32
    if out is not None or out_dtype == OUT_FP32_ACCUMULATE:
        _check_out(out, shape, dt, "out")
        if out.device != dy.device:
            raise ValueError(f"out: on {out.device}, the other tensors are on {dy.device}")
        _no_overlap(out, "out", dy=dy, x=x, m_splits=m_splits)
    dw = out if out is not None else torch.empty(shape, dtype=dt, device=dy.device)
    _call(GEMM_WGRAD, _row_major(dy), _row_major(x), dw, m_splits, dy.shape[0], dy.shape[1], x.shape[1], out_dtype, False, ws)
    return dw if out is None else _written(out)


class GroupedMatmulFunction(torch.autograd.Function):
    """torch.autograd over the three products: the backward computes dx only when x requires grad
    and dw (w's dtype, or added to w.main_grad in fp32) only when w does."""

    @staticmethod
    def forward(fctx, x, w, m_splits, accumulate_main_grad=False):
        fctx.main_grad = w.main_grad if accumulate_main_grad else None
        fctx.save_for_backward(x, w, m_splits)
        return grouped_matmul_forward(x, w, m_splits)

    @staticmethod
    @once_differentiable
    def backward(fctx, dy):
        x, w, m_splits = fctx.saved_tensors
        need = fctx.needs_input_grad
        dy = dy.to(x.dtype)
        dx = grouped_matmul_dgrad(dy, w, m_splits) if need[0] else None
        dw = None
        if need[1] and fctx.main_grad is not None:
            grouped_matmul_wgrad(dy, x, m_splits, OUT_FP32_ACCUMULATE, out=fctx.main_grad)
        elif need[1]:
            dw = grouped_matmul_wgrad(dy, x, m_splits)
        return dx, dw, None, None


def grouped_matmul(x, w, m_splits, accumulate_main_grad=False):
    """y [M, N] = the grouped product of x [M, K] and w [G, N, K], differentiable in x and w.
    accumulate_main_grad: the weight gradient is added to the fp32 w.main_grad and autograd
    receives none for w."""
    if accumulate_main_grad:
        _check_out(getattr(w, "main_grad", None), tuple(w.shape), torch.float32, "w.main_grad")
    return GroupedMatmulFunction.apply(x, w, m_splits, accumulate_main_grad)
