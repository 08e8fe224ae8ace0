"""Grouped products of few rows with weights of 4 bits, as decoding has them (bf16 / fp16 rows):

    y = grouped_matmul_w4(x, w, m_splits)       # y[r] = x[r] w[g]^T, g the group of row r by m_splits

w is an Int4Weights (integers with a scale, and a zero if given, by group of 32, 64 or 128 along K) or what
weight_quantize made with the NVFP4 recipe (a QTensor put together by hand says how long its rows are by its shape
or by a row_data or row_scale [G, N, ..]: where all are flat, rows are taken to be as long as x's).  One group is a
dense layer.  Sums are fp32 over exact products, each result is rounded once; scales of integers are 0 or 2^-100 to
2^96 in magnitude.  The weights are constants: no gradient is computed.  Argument marshalling only.
"""
import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _SIGS, NVFP4_RHT, QTensor, _dev_ptr, _splits, lib
from .matmul import _DTYPES, _check_rows_out, _dtype16, _ld, _no_overlap, _packer, _row_major, _run, _written

W4_INT, W4_NVFP4 = 0, 1


class W4Args(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("kind", ctypes.c_int32), ("group", ctypes.c_int32), ("zero_rest", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p), ("amax", ctypes.c_void_p), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
                ("m_splits", ctypes.c_void_p), ("G", ctypes.c_int32), ("M", ctypes.c_int64), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64)]


_SIGS.update({"gmlp_grouped_matmul_four_bit": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p])})      # W4Args*
_pack = _packer(W4Args)


@dataclass(frozen=True, eq=False)
class Int4Weights:
    """w[g, n, k] = (q - zero) scale.  codes uint8 [G, N, K / 2]: q of k even in the low four bits, odd in the
    high; scales bf16 or fp16 [G, N, K / group] (the rows' type), zeros uint8 of that shape with values 0 to 15 or
    None (8).  Checked once, so its tensors are not replaced afterwards."""
    codes: torch.Tensor
    scales: torch.Tensor
    zeros: Optional[torch.Tensor] = None

    def __post_init__(self):
        c, s, z = self.codes, self.scales, self.zeros
        if not isinstance(c, torch.Tensor) or c.dtype != torch.uint8 or c.dim() != 3 or not c.is_contiguous():
            raise TypeError("codes: a contiguous uint8 tensor [G, N, K / 2] is required")
        _dtype16(s, "scales")
        if s.dim() != 3 or not s.is_contiguous() or s.shape[:2] != c.shape[:2]:
            raise ValueError(f"scales: a contiguous tensor [{c.shape[0]}, {c.shape[1]}, K / group] is required, got {tuple(s.shape)}")
        if self.group not in (32, 64, 128) or self.group * s.shape[2] != self.K:
            raise ValueError(f"scales: groups of 32, 64 or 128 are required, got {s.shape[2]} scales for K = {self.K}")
        if z is not None and (not isinstance(z, torch.Tensor) or z.dtype != torch.uint8 or z.shape != s.shape or not z.is_contiguous()):
            raise TypeError(f"zeros: a contiguous uint8 tensor of shape {tuple(s.shape)} is required")
        if s.device != c.device or (z is not None and z.device != c.device):
            raise ValueError("codes, scales and zeros on one device are required")

    @property
    def K(self):
        return 2 * self.codes.shape[2]

    @property
    def group(self):
        return self.K // max(self.scales.shape[2], 1)


def _nvfp4(w, G, K):
    """(codes, scales, amax, N) of a weight quantized with the NVFP4 recipe."""
    if w.kind != NVFP4_RHT:
        raise ValueError("w: 4-bit weights are required (the NVFP4 recipe's)")
    c, s, a = (w.bufs.get(n) for n in ("row_data", "row_scale", "amax_pre"))
    if any(not isinstance(t, torch.Tensor) or not t.is_contiguous() for t in (c, s, a)):
        raise ValueError("w: contiguous row_data, row_scale and amax_pre are required")
    if c.dtype != torch.uint8 or s.dtype != torch.uint8 or a.dtype != torch.float32:
        raise TypeError("w: uint8 row_data and row_scale and fp32 amax_pre are required")
    if w.shape is not None and (len(w.shape) != 3 or w.shape[0] != G or w.shape[2] != K):
        raise ValueError(f"w: [{G}, N, {K}] expected, got {list(w.shape)}")
    for t, n in ((c, K // 2), (s, K // 16)):                         # flatter ones do not say how long a row is
        if t.dim() > 2 and t.shape[-1] != n:
            raise ValueError(f"w: rows of {K} elements expected, got row_data {tuple(c.shape)} and row_scale {tuple(s.shape)}")
    N = w.shape[1] if w.shape is not None else 2 * c.numel() // max(G * K, 1)
    if N < 1 or 2 * c.numel() != G * N * K or s.numel() * 16 != G * N * K or a.numel() != G:
        raise ValueError(f"w: sizes do not fit {G} groups of rows of {K} elements")
    return c, s, a, N


def grouped_matmul_w4(x, w, m_splits, out=None):
    """y [M, N] in x's dtype.  Rows behind the last group are zero in a new output and left as they are in
    `out`."""
    _dtype16(x, "x")
    if x.dim() != 2 or x.shape[1] < 1:
        raise ValueError(f"x: [M, K] expected, got {tuple(x.shape)}")
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError("x: no gradient is computed through 4-bit weights")
    M, K = x.shape
    dev = x.device
    m_splits = _splits(m_splits)
    G = m_splits.numel()
    zeros = amax = None
    if isinstance(w, Int4Weights):
        codes, scales, zeros, group = w.codes, w.scales, w.zeros, w.group
        if codes.shape[0] != G or w.K != K:
            raise ValueError(f"w: [{G}, N, {K}] expected, got [{codes.shape[0]}, {codes.shape[1]}, {w.K}]")
        if scales.dtype != x.dtype:
            raise TypeError(f"w: scales of x's type {x.dtype} are required, got {scales.dtype}")
        N, kind = codes.shape[1], W4_INT
    elif isinstance(w, QTensor):
        codes, scales, amax, N = _nvfp4(w, G, K)
        kind, group = W4_NVFP4, 16
    else:
        raise TypeError("w: an Int4Weights or a QTensor is required")
    if (scales.requires_grad or (amax is not None and amax.requires_grad)) and torch.is_grad_enabled():
        raise ValueError("w: no gradient is computed for the weights' scales")
    for t, name in ((codes, "w"), (scales, "w"), (zeros, "w"), (amax, "w"), (m_splits, "m_splits")):
        if t is not None and t.device != dev:
            raise ValueError(f"{name}: on {t.device}, the other tensors are on {dev}")
    if out is not None:
        _check_rows_out(out, (M, N), x, "out")
        _no_overlap(out, "out", x=x, codes=codes, scales=scales, zeros=zeros, amax=amax, m_splits=m_splits)
    _dev_ptr(x, "x")
    x = _row_major(x)
    y = out if out is not None else torch.empty((M, N), dtype=x.dtype, device=dev)
    args = _pack(_DTYPES[x.dtype], kind, group, out is None, x.data_ptr(), _ld(x), codes.data_ptr(), scales.data_ptr(),
                 zeros.data_ptr() if zeros is not None else 0, amax.data_ptr() if amax is not None else 0, y.data_ptr(), _ld(y),
                 m_splits.data_ptr(), G, M, N, K)
    _run(lib().gmlp_grouped_matmul_four_bit, args, dev)
    return y if out is None else _written(out)
