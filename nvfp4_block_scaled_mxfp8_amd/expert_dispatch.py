"""Tokens brought into expert order and back, around grouped_mlp or grouped_matmul:

    plan = dispatch_plan(experts, E)        # the order, from each token's experts [T, k]
    xg = dispatch(x, plan)                  # [T k, H], rows grouped by expert; plan.m_splits the group sizes
    y = combine(expert_output, plan, probs) # y[t] = sum_j probs[t, j] expert_output[row of (t, j)]

dispatch and combine are differentiable (x; expert_output and probs); the *_forward and *_backward
functions are the same calls without autograd.  Argument marshalling only.
"""
import ctypes
import functools
from dataclasses import dataclass

import torch

from . import _SIGS, _check, _dev_ptr, lib
from .matmul import _DTYPES, _check_rows_out, _dtype16, _ld, _no_overlap, _packer, _row_major, _run, _written, once_differentiable


class MoveArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("zero_rest", ctypes.c_int32), ("src", ctypes.c_void_p),
                ("ld_src", ctypes.c_int64), ("src2", ctypes.c_void_p), ("ld_src2", ctypes.c_int64),
                ("dst", ctypes.c_void_p), ("ld_dst", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
                ("k", ctypes.c_int32), ("E", ctypes.c_int32), ("rows", ctypes.c_void_p),
                ("m_splits", ctypes.c_void_p), ("probs", ctypes.c_void_p), ("dprobs", ctypes.c_void_p)]


_SIGS.update({
    "gmlp_dispatch_plan_ws_bytes": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
    "gmlp_dispatch_plan": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                          ctypes.c_void_p]),
    "gmlp_dispatch": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),              # MoveArgs*
    "gmlp_combine": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "gmlp_combine_dprobs": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
})
_pack_move = _packer(MoveArgs)


@dataclass
class DispatchPlan:
    """m_splits int32 [E]: rows per expert; rows int32 [T, k]: the row of each slot in expert order, -1
    for a dropped one (an expert outside [0, E)); rows behind the sum of m_splits belong to no expert."""
    m_splits: torch.Tensor
    rows: torch.Tensor

    def __post_init__(self):
        for t, name, dim in ((self.m_splits, "m_splits", 1), (self.rows, "rows", 2)):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != dim or not t.is_contiguous():
                raise TypeError(f"{name}: a contiguous int32 tensor of {dim} dimensions is required")
        if self.m_splits.device != self.rows.device or self.m_splits.numel() < 1 or self.rows.shape[1] < 1:
            raise ValueError("plan: m_splits [E] and rows [T, k] on one device are required")

    @property
    def tokens(self):
        return self.rows.shape[0]

    @property
    def k(self):
        return self.rows.shape[1]


@functools.lru_cache(maxsize=4096)
def _plan_ws_bytes(n, E):
    need = ctypes.c_size_t(0)
    _check(lib().gmlp_dispatch_plan_ws_bytes(n, E, ctypes.byref(need)))
    return need.value


def dispatch_plan(experts, E):
    """The stable order by expert of the slots of `experts` (int32 [T, k] on the device)."""
    if not isinstance(experts, torch.Tensor) or experts.dtype != torch.int32 or experts.dim() != 2 or experts.shape[1] < 1:
        raise TypeError("experts: an int32 tensor [T, k] is required")
    experts = experts.contiguous()
    dev, n = experts.device, experts.numel()
    need = _plan_ws_bytes(n, E)
    _dev_ptr(experts, "experts")
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    plan = DispatchPlan(torch.empty(E, dtype=torch.int32, device=dev), torch.empty_like(experts))
    L = lib()
    _run(lambda _, stream: L.gmlp_dispatch_plan(experts.data_ptr(), n, E, plan.m_splits.data_ptr(), plan.rows.data_ptr(),
                                                None, ws.data_ptr() if need else None, need, stream), None, dev)
    return plan


def _check_plan(plan, t, name, per_slot):
    if not isinstance(plan, DispatchPlan):
        raise TypeError("plan: a DispatchPlan is required")
    _dtype16(t, name)
    n = plan.rows.numel() if per_slot else plan.tokens
    if t.dim() != 2 or t.shape[0] != n:
        raise ValueError(f"{name}: {n} rows expected (T = {plan.tokens}, k = {plan.k}), got {tuple(t.shape)}")
    if t.device != plan.rows.device:
        raise ValueError(f"{name}: on {t.device}, the plan is on {plan.rows.device}")


def _check_probs(probs, plan):
    if probs is None:
        return None
    if not isinstance(probs, torch.Tensor) or probs.dtype != torch.float32 or probs.shape != plan.rows.shape:
        raise TypeError(f"probs: an fp32 tensor of shape {tuple(plan.rows.shape)} is required")
    if probs.device != plan.rows.device:
        raise ValueError(f"probs: on {probs.device}, the plan is on {plan.rows.device}")
    return probs.contiguous()


def _ptr(t):
    return t.data_ptr() if t is not None else 0


def _move(fn, plan, src, dst, probs=None, zero_rest=False, src2=None, dprobs=None):
    _dev_ptr(src, "src")                                             # refuses host tensors
    src = _row_major(src)
    if src2 is not None:
        src2 = _row_major(src2)
    T, k = plan.rows.shape
    args = _pack_move(_DTYPES[src.dtype], zero_rest, src.data_ptr(), _ld(src), _ptr(src2),
                      _ld(src2) if src2 is not None else 0, _ptr(dst), _ld(dst) if dst is not None else 0, T, src.shape[1],
                      k, plan.m_splits.numel(), plan.rows.data_ptr(), plan.m_splits.data_ptr(), _ptr(probs), _ptr(dprobs))
    _run(getattr(lib(), fn), args, src.device)


def _to_rows(src, plan, probs, out):
    shape = (plan.rows.numel(), src.shape[1])
    if out is not None:
        _check_rows_out(out, shape, src, "out")
        _no_overlap(out, "out", input=src, probs=probs, rows=plan.rows, m_splits=plan.m_splits)
    dst = out if out is not None else torch.empty(shape, dtype=src.dtype, device=src.device)
    _move("gmlp_dispatch", plan, src, dst, probs, zero_rest=out is None)
    return dst if out is None else _written(out)


def _to_tokens(src, plan, probs, out):
    shape = (plan.tokens, src.shape[1])
    if out is not None:
        _check_rows_out(out, shape, src, "out")
        _no_overlap(out, "out", input=src, probs=probs, rows=plan.rows, m_splits=plan.m_splits)
    dst = out if out is not None else torch.empty(shape, dtype=src.dtype, device=src.device)
    _move("gmlp_combine", plan, src, dst, probs)
    return dst if out is None else _written(out)


def dispatch_forward(x, plan, out=None):
    """xg [T k, H]: x[t] at the row of each of its slots.  Rows of no expert are zero in a new output
    and left as they are in `out`."""
    _check_plan(plan, x, "x", False)
    return _to_rows(x, plan, None, out)


def dispatch_backward(dxg, plan, out=None):
    """dx [T, H]: the sum over a token's slots of dxg's rows (fp32, rounded once)."""
    _check_plan(plan, dxg, "dxg", True)
    return _to_tokens(dxg, plan, None, out)


def combine_forward(v, plan, probs=None, out=None):
    """y [T, H]: sum over j of probs[t, j] v[row of (t, j)] (probs fp32 [T, k]; None: 1)."""
    _check_plan(plan, v, "v", True)
    return _to_tokens(v, plan, _check_probs(probs, plan), out)


def combine_backward(dy, v, plan, probs=None, need_dv=True, need_dprobs=True):
    """(dv [T k, H], dprobs fp32 [T, k]) of combine_forward; v is read for dprobs only."""
    _check_plan(plan, dy, "dy", False)
    probs = _check_probs(probs, plan)
    dv = _to_rows(dy, plan, probs, None) if need_dv else None
    dp = None
    if need_dprobs and probs is not None:
        _check_plan(plan, v, "v", True)
        if v.dtype != dy.dtype or v.shape[1] != dy.shape[1]:
            raise ValueError(f"v: {dy.dtype} rows of {dy.shape[1]} elements expected, got {v.dtype} {tuple(v.shape)}")
        dp = torch.empty_like(probs)
        _move("gmlp_combine_dprobs", plan, dy, None, src2=v, dprobs=dp)
    return dv, dp


class DispatchFunction(torch.autograd.Function):
    @staticmethod
    def forward(fctx, x, plan):
        fctx.dtype = x.dtype
        xg = dispatch_forward(x, plan)
        fctx.save_for_backward(plan.m_splits, plan.rows)
        return xg

    @staticmethod
    @once_differentiable
    def backward(fctx, dxg):
        return dispatch_backward(dxg.to(fctx.dtype), DispatchPlan(*fctx.saved_tensors)), None


class CombineFunction(torch.autograd.Function):
    @staticmethod
    def forward(fctx, v, probs, plan):
        y = combine_forward(v, plan, probs)
        fctx.save_for_backward(plan.m_splits, plan.rows, v, probs)
        return y

    @staticmethod
    @once_differentiable
    def backward(fctx, dy):
        m_splits, rows, v, probs = fctx.saved_tensors
        need = fctx.needs_input_grad
        dv, dp = combine_backward(dy.to(v.dtype), v, DispatchPlan(m_splits, rows), probs, need[0], need[1])
        return dv, dp, None


def dispatch(x, plan):
    """dispatch_forward under torch.autograd (gradient for x)."""
    return DispatchFunction.apply(x, plan)


def combine(v, plan, probs=None):
    """combine_forward under torch.autograd (gradients for v and probs)."""
    return CombineFunction.apply(v, probs, plan)
