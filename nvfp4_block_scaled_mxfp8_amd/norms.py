"""The norms on both sides of a block, with its gate and the residual sum (bf16 / fp16):

    y, h = residual_norm(x, branch, weight, branch_weight, gate, scale)

    n = branch / sqrt(mean(branch^2) + eps) branch_weight     # branch_weight None: n = branch
    y = x + scale gate n                                      # the residual stream [T, H]
    h = y / sqrt(mean(y^2) + eps) weight                      # the next block's input; weight None: no h

gate: [H] by channel, [T, 1] by token, [T, H], or None (1).  weight, branch_weight and gate are of x's type or
fp32.  Sums and y are fp32, each result is rounded once (h from the unrounded y).  rms_norm(x, weight) is h
of x alone.  residual_norm and rms_norm are differentiable in all tensors; the *_forward and *_backward
functions are the same calls without autograd.  Argument marshalling only.
"""
import ctypes
import functools

import torch

from . import _SIGS, _check, _dev_ptr, lib
from .matmul import _CODES, _check_rows_out, _dtype16, _ld, _no_overlap, _packer, _row_major, _run, _written, once_differentiable

_CODES.setdefault(ctypes.c_float, "f")
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3


class NormInputs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("gate_kind", ctypes.c_int32), ("weight_fp32", ctypes.c_int32),
                ("branch_weight_fp32", ctypes.c_int32), ("gate_fp32", ctypes.c_int32), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float), ("T", ctypes.c_int64), ("H", ctypes.c_int64), ("x", ctypes.c_void_p),
                ("ldx", ctypes.c_int64), ("branch", ctypes.c_void_p), ("ldbranch", ctypes.c_int64), ("weight", ctypes.c_void_p),
                ("branch_weight", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("ld_gate", ctypes.c_int64)]


class NormArgs(ctypes.Structure):
    _fields_ = [("inputs", NormInputs), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("h", ctypes.c_void_p),
                ("ldh", ctypes.c_int64), ("stats", ctypes.c_void_p)]


class NormBwdArgs(ctypes.Structure):
    _fields_ = [("inputs", NormInputs), ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64), ("dh", ctypes.c_void_p),
                ("lddh", ctypes.c_int64), ("stats", ctypes.c_void_p), ("dx", ctypes.c_void_p), ("lddx", ctypes.c_int64),
                ("dbranch", ctypes.c_void_p), ("lddbranch", ctypes.c_int64), ("dgate", ctypes.c_void_p),
                ("dweight", ctypes.c_void_p), ("dbranch_weight", ctypes.c_void_p), ("ws", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_size_t)]


_SIGS.update({
    "gmlp_residual_norm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),            # NormArgs*
    "gmlp_residual_norm_bwd_ws_bytes": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)]),
    "gmlp_residual_norm_backward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),   # NormBwdArgs*
})
_pack_fwd, _pack_bwd = _packer(NormArgs), _packer(NormBwdArgs)


@functools.lru_cache(maxsize=4096)
def _ws_bytes(T, H):
    need = ctypes.c_size_t(0)
    _check(lib().gmlp_residual_norm_bwd_ws_bytes(T, H, ctypes.byref(need)))
    return need.value


# A decode step's norm takes 4.5 us on the device, so the checks below ask each tensor for each property once.
def _param(t, H, dt, dev, name):
    """A vector of H parameters, of the rows' type or fp32: (the tensor to keep, its address, fp32 or not)."""
    if t is None:
        return None, 0, 0
    if not isinstance(t, torch.Tensor) or (t.dtype is not dt and t.dtype is not torch.float32):
        raise TypeError(f"{name}: a {dt} or fp32 tensor is required, got {getattr(t, 'dtype', type(t).__name__)}")
    if tuple(t.shape) != (H,):
        raise ValueError(f"{name}: {H} elements expected (rows of x), got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name}: on {t.device}, the other tensors are on {dev}")
    if not t.is_contiguous():
        t = t.contiguous()
    return t, t.data_ptr(), t.dtype is torch.float32


def _gate(gate, T, H, dt, dev):
    """(kind, the gate as the kernels address it, its address, fp32 or not, its row stride)."""
    if gate is None:
        return GATE_NONE, None, 0, 0, 0
    if isinstance(gate, torch.Tensor) and gate.dim() == 1:
        return (GATE_CHANNEL, *_param(gate, H, dt, dev, "gate"), 0)
    if not isinstance(gate, torch.Tensor) or gate.dtype not in (dt, torch.float32):
        raise TypeError(f"gate: a {dt} or fp32 tensor is required, got {getattr(gate, 'dtype', type(gate).__name__)}")
    if gate.device != dev:
        raise ValueError(f"gate: on {gate.device}, the other tensors are on {dev}")
    if tuple(gate.shape) == (T, 1):
        if T > 1 and gate.stride(0) < 1:
            gate = gate.contiguous()
        return GATE_TOKEN, gate, gate.data_ptr(), gate.dtype is torch.float32, gate.stride(0) if T > 1 else 1
    if tuple(gate.shape) != (T, H):
        raise ValueError(f"gate: shape [{H}], [{T}, 1] or [{T}, {H}] expected, got {tuple(gate.shape)}")
    gate = _row_major(gate)
    return GATE_FULL, gate, gate.data_ptr(), gate.dtype is torch.float32, _ld(gate)


def _rows(t, shape, dt, dev, name):
    """Rows beside x's, of its type, device and shape: (the tensor to keep, its address, its row stride)."""
    if t is None:
        return None, 0, 0
    if not isinstance(t, torch.Tensor) or t.dtype is not dt:
        raise TypeError(f"{name}: a {dt} tensor is required, got {getattr(t, 'dtype', type(t).__name__)}")
    if t.device != dev:
        raise ValueError(f"{name}: on {t.device}, the other tensors are on {dev}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t, t.data_ptr(), shape[1]
    t = _row_major(t)
    return t, t.data_ptr(), _ld(t)


def _inputs(x, branch, weight, branch_weight, gate, scale, eps):
    """(the fields of NormInputs, the tensors that they address: x, branch, weight, branch_weight, gate, x's device and shape)."""
    code = _dtype16(x, "x")
    dt, dev, shape = x.dtype, x.device, x.shape
    if len(shape) != 2:
        raise ValueError(f"x: 2 dimensions expected, got {len(shape)}")
    T, H = shape
    branch, pb, ldb = _rows(branch, shape, dt, dev, "branch")
    weight, pw, w32 = _param(weight, H, dt, dev, "weight")
    branch_weight, pbw, bw32 = _param(branch_weight, H, dt, dev, "branch_weight")
    kind, gate, pg, g32, ldg = _gate(gate, T, H, dt, dev)
    if dev.type != "cuda":
        _dev_ptr(x, "x")                                             # refuses host tensors
    x, px, ldx = _rows(x, shape, dt, dev, "x")
    return ((code, kind, w32, bw32, g32, eps, scale, T, H, px, ldx, pb, ldb, pw, pbw, pg, ldg),
            (x, branch, weight, branch_weight, gate), dev, shape)


def residual_norm_forward(x, branch, weight=None, branch_weight=None, gate=None, scale=1.0, eps=1e-6, out=None):
    """(y, h, stats): y and h [T, H] in x's dtype (h None without weight; y is x without branch), stats for
    residual_norm_backward.  out: y is written there; it may be x or branch itself (in place)."""
    fields, kept, dev, shape = _inputs(x, branch, weight, branch_weight, gate, scale, eps)
    T, H = shape
    y, py, ldy = x, 0, H
    if out is not None:
        _check_rows_out(out, shape, x, "out")
        if branch is None:
            raise ValueError("out: without a branch, y is x")
        _no_overlap(out, "out", weight=weight, branch_weight=branch_weight, gate=gate,
                    **{n: t for n, t in (("x", kept[0]), ("branch", kept[1]))
                       if t.data_ptr() != out.data_ptr() or _ld(t) != _ld(out)})
        y, py, ldy = out, out.data_ptr(), _ld(out)
    elif branch is not None:
        y = torch.empty(shape, dtype=x.dtype, device=dev)
        py = y.data_ptr()
    h = torch.empty(shape, dtype=x.dtype, device=dev) if weight is not None else None
    stats = torch.empty((2, T), dtype=torch.float32, device=dev)
    if T > 0:
        _run(lib().gmlp_residual_norm, _pack_fwd(*fields, py, ldy, h.data_ptr() if h is not None else 0, H, stats.data_ptr()), dev)
    return y if out is None else _written(out), h, stats


def residual_norm_backward(dy, dh, x, branch, stats, weight=None, branch_weight=None, gate=None, scale=1.0, eps=1e-6,
                           need_dx=True, need_dbranch=True, need_dweight=True, need_dbranch_weight=True, need_dgate=True):
    """{"dx", "dbranch", "dweight", "dbranch_weight", "dgate"} (None where there is no such input or it is
    not needed) from the gradients of y (None: zeros) and h (None without weight) and a forward's inputs and
    stats.  The inputs, scale and eps must be as the forward had them: not after an in-place forward."""
    fields, kept, dev, shape = _inputs(x, branch, weight, branch_weight, gate, scale, eps)
    T, H = shape
    dy, pdy, lddy = _rows(dy, shape, x.dtype, dev, "dy")
    dh, pdh, lddh = _rows(dh, shape, x.dtype, dev, "dh")
    if (dh is None) != (weight is None):
        raise ValueError("dh: goes with a weight")
    if not isinstance(stats, torch.Tensor) or stats.dtype is not torch.float32 or tuple(stats.shape) != (2, T) \
            or not stats.is_contiguous() or stats.device != dev:
        raise ValueError(f"stats: the fp32 tensor [2, {T}] of a residual_norm_forward is required")
    res, ptrs = {}, {}
    for name, t, wanted in (("dx", x, need_dx), ("dbranch", branch, need_dbranch), ("dweight", weight, need_dweight),
                            ("dbranch_weight", branch_weight, need_dbranch_weight), ("dgate", gate, need_dgate)):
        r = torch.empty(t.shape, dtype=t.dtype, device=dev) if wanted and t is not None else None
        res[name], ptrs[name] = r, r.data_ptr() if r is not None else 0
    if T == 0:                                                       # sums over no rows
        return {k: r.zero_() if r is not None else None for k, r in res.items()}
    need = _ws_bytes(T, H)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    args = _pack_bwd(*fields, pdy, lddy, pdh, lddh, stats.data_ptr(), ptrs["dx"], H, ptrs["dbranch"], H, ptrs["dgate"], ptrs["dweight"],
                     ptrs["dbranch_weight"], ws.data_ptr(), need)
    _run(lib().gmlp_residual_norm_backward, args, dev)
    return res


def rms_norm_forward(x, weight, eps=1e-6):
    """(h, stats): h [T, H] = x / sqrt(mean(x^2) + eps) weight in x's dtype."""
    if weight is None:
        raise TypeError("weight: a tensor is required")
    return residual_norm_forward(x, None, weight, eps=eps)[1:]


def rms_norm_backward(dh, x, weight, stats, eps=1e-6):
    """(dx, dweight) of rms_norm_forward."""
    g = residual_norm_backward(None, dh, x, None, stats, weight, eps=eps)
    return g["dx"], g["dweight"]


class ResidualNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(fctx, x, branch, weight, branch_weight, gate, scale, eps):
        fctx.how = (scale, eps)
        fctx.set_materialize_grads(False)
        y, h, stats = residual_norm_forward(x, branch, weight, branch_weight, gate, scale, eps)
        fctx.save_for_backward(x, branch, weight, branch_weight, gate, stats)
        fctx.with_y, fctx.with_h = branch is not None, weight is not None
        return (y, h) if fctx.with_y and fctx.with_h else y if fctx.with_y else h

    @staticmethod
    @once_differentiable
    def backward(fctx, *grads):
        x, branch, weight, branch_weight, gate, stats = fctx.saved_tensors
        grads = list(grads)
        dy = grads.pop(0) if fctx.with_y else None
        dh = grads.pop(0) if fctx.with_h else None
        if dy is None and dh is None:
            return (None,) * 7
        if dh is None:                                               # h went nowhere
            weight = None
        need = fctx.needs_input_grad
        g = residual_norm_backward(dy.to(x.dtype) if dy is not None else None, dh.to(x.dtype) if dh is not None else None, x,
                                   branch, stats, weight, branch_weight, gate, *fctx.how, *need[:5])
        return g["dx"], g["dbranch"], g["dweight"], g["dbranch_weight"], g["dgate"], None, None


def residual_norm(x, branch, weight=None, branch_weight=None, gate=None, scale=1.0, eps=1e-6):
    """residual_norm_forward under torch.autograd: (y, h), or y where weight is None."""
    if branch is None:
        raise TypeError("branch: a tensor is required (rms_norm is the norm alone)")
    return ResidualNormFunction.apply(x, branch, weight, branch_weight, gate, scale, eps)


def rms_norm(x, weight, eps=1e-6):
    """rms_norm_forward under torch.autograd."""
    if weight is None:
        raise TypeError("weight: a tensor is required")
    return ResidualNormFunction.apply(x, None, weight, None, None, 1.0, eps)
