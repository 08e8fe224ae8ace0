"""The experts of each token from the router's logits, as dispatch_plan takes them:

    experts, probs = route(logits, k)            # logits [T, E] -> int32 [T, k], fp32 [T, k]

    score        s = "softmax" or "sigmoid" of the logits
    bias         fp32 [E], added to s for the choice only (compared as in 64 bits); None: the choice is by the logits
    groups       experts in groups of E / groups; those of the top_groups groups take part whose group_best
                 (1 or 2) largest s + bias have the largest sum (1 without a bias: the largest logit)
    renormalize  probs = scale s / sum of the row's chosen s, else scale s

A logit of -inf masks its expert; a slot that finds none has expert -1 (dispatch_plan drops it) and
probability 0.  Ties go to the lowest index.  route is differentiable in the logits (through probs);
route_forward and route_backward are the same calls without autograd.  Argument marshalling only.
"""
import ctypes

import torch

from . import _SIGS, _dev_ptr, lib
from .matmul import _CODES, _ld, _packer, _row_major, _run, once_differentiable

_CODES.setdefault(ctypes.c_float, "f")
_SCORES = {"softmax": 0, "sigmoid": 1}
_LOGITS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class RouteArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("score", ctypes.c_int32), ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("T", ctypes.c_int64), ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("bias", ctypes.c_void_p),
                ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32), ("group_best", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float), ("experts", ctypes.c_void_p),
                ("probs", ctypes.c_void_p)]


class RouteBwdArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("score", ctypes.c_int32), ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("T", ctypes.c_int64), ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("experts", ctypes.c_void_p),
                ("dprobs", ctypes.c_void_p), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float),
                ("dlogits", ctypes.c_void_p), ("ld_dlogits", ctypes.c_int64)]


_SIGS.update({
    "gmlp_route": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),                # RouteArgs*
    "gmlp_route_backward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),       # RouteBwdArgs*
})
_pack_fwd, _pack_bwd = _packer(RouteArgs), _packer(RouteBwdArgs)


def _check_logits(logits, score):
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _LOGITS:
        raise TypeError(f"logits: a bf16, fp16 or fp32 tensor is required, got {getattr(logits, 'dtype', type(logits).__name__)}")
    if logits.dim() != 2 or logits.shape[1] < 1:
        raise ValueError(f"logits: [T, E] expected, got {tuple(logits.shape)}")
    if score not in _SCORES:
        raise ValueError(f"score: one of {', '.join(_SCORES)} expected, got {score!r}")
    return _LOGITS[logits.dtype], _SCORES[score]


def route_forward(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0):
    """(experts int32 [T, k], probs fp32 [T, k]) of logits [T, E]."""
    dtype, sc = _check_logits(logits, score)
    T, E = logits.shape
    dev = logits.device
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or bias.dtype != torch.float32 or tuple(bias.shape) != (E,):
            raise TypeError(f"bias: an fp32 tensor of {E} elements is required")
        if bias.device != dev:
            raise ValueError(f"bias: on {bias.device}, the logits are on {dev}")
        bias = bias.contiguous()
    if not isinstance(k, int) or k < 1:
        raise ValueError(f"k: a number of experts >= 1 is required, got {k!r}")
    _dev_ptr(logits, "logits")
    logits = _row_major(logits)
    experts = torch.empty((T, k), dtype=torch.int32, device=dev)
    probs = torch.empty((T, k), dtype=torch.float32, device=dev)
    args = _pack_fwd(dtype, sc, logits.data_ptr(), _ld(logits), T, E, k, bias.data_ptr() if bias is not None else 0, groups,
                     top_groups, group_best, renormalize, scale, experts.data_ptr(), probs.data_ptr())
    _run(lib().gmlp_route, args, dev)
    return experts, probs


def route_backward(dprobs, logits, experts, score="softmax", renormalize=True, scale=1.0):
    """dlogits [T, E], in the logits' type, from the gradient of probs and a forward's experts (its score,
    renormalize and scale)."""
    dtype, sc = _check_logits(logits, score)
    T, E = logits.shape
    dev = logits.device
    if not isinstance(experts, torch.Tensor) or experts.dtype != torch.int32 or experts.dim() != 2 or experts.shape[0] != T \
            or experts.shape[1] < 1:
        raise TypeError(f"experts: an int32 tensor [{T}, k] is required")
    if not isinstance(dprobs, torch.Tensor) or dprobs.dtype != torch.float32 or dprobs.shape != experts.shape:
        raise TypeError(f"dprobs: an fp32 tensor of shape {tuple(experts.shape)} is required")
    if experts.device != dev or dprobs.device != dev:
        raise ValueError(f"experts, dprobs: on {experts.device} and {dprobs.device}, the logits are on {dev}")
    _dev_ptr(logits, "logits")
    logits, experts, dprobs = _row_major(logits), experts.contiguous(), dprobs.contiguous()
    dlogits = torch.empty((T, E), dtype=logits.dtype, device=dev)
    args = _pack_bwd(dtype, sc, logits.data_ptr(), _ld(logits), T, E, experts.shape[1], experts.data_ptr(), dprobs.data_ptr(),
                     renormalize, scale, dlogits.data_ptr(), E)
    _run(lib().gmlp_route_backward, args, dev)
    return dlogits


class RouteFunction(torch.autograd.Function):
    @staticmethod
    def forward(fctx, logits, k, score, bias, groups, top_groups, group_best, renormalize, scale):
        experts, probs = route_forward(logits, k, score, bias, groups, top_groups, group_best, renormalize, scale)
        fctx.how = (score, renormalize, scale)
        fctx.save_for_backward(logits, experts)
        fctx.mark_non_differentiable(experts)
        return experts, probs

    @staticmethod
    @once_differentiable
    def backward(fctx, _, dprobs):
        logits, experts = fctx.saved_tensors
        return (route_backward(dprobs.float(), logits, experts, *fctx.how),) + (None,) * 8


def route(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0):
    """route_forward under torch.autograd (gradient for the logits; the bias is a constant)."""
    if isinstance(bias, torch.Tensor) and bias.requires_grad:
        raise ValueError("bias: no gradient is computed for the bias")
    return RouteFunction.apply(logits, k, score, bias, groups, top_groups, group_best, renormalize, scale)
