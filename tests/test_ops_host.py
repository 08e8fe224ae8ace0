"""Refusals of the bf16 / fp16 operators (CPU): bad arguments are errors before anything is launched,
in the binding and in the C ABI."""
import ctypes

import pytest
import torch

import nvfp4_block_scaled_mxfp8_amd as g


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_host_tensors_and_wrong_types():
    x, w, m = _t(4, 16), _t(2, 8, 16), torch.tensor([2, 2], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.grouped_matmul_forward(x, w, m)
    with pytest.raises(TypeError, match="bf16 or fp16"):
        g.grouped_matmul_forward(x.float(), w.float(), m)
    with pytest.raises(TypeError, match="w:"):
        g.grouped_matmul_forward(x, w.half(), m)
    with pytest.raises(TypeError, match="m_splits"):
        g.grouped_matmul_forward(x, w, m.long())
    with pytest.raises(ValueError, match="groups expected"):
        g.grouped_matmul_forward(x, w, m[:1])
    with pytest.raises(ValueError, match="16 elements"):
        g.grouped_matmul_forward(_t(4, 8), w, m)
    with pytest.raises(ValueError, match="8 elements"):
        g.grouped_matmul_dgrad(_t(4, 16), w, m)
    with pytest.raises(ValueError, match="4 rows"):
        g.grouped_matmul_wgrad(_t(4, 8), _t(5, 16), m)
    with pytest.raises(ValueError, match="dimensions"):
        g.grouped_matmul_forward(_t(2, 2, 16), w, m)
    with pytest.raises(ValueError, match="out"):
        g.grouped_matmul_forward(x, w, m, out=_t(4, 9))
    with pytest.raises(ValueError, match="out"):
        g.grouped_matmul_wgrad(_t(4, 8), x, m, g.OUT_FP32_ACCUMULATE)
    with pytest.raises(ValueError, match="main_grad"):
        g.grouped_matmul(x, w, m, accumulate_main_grad=True)


def _mm(**kw):
    a = g.GroupedMatmulArgs()
    vals = dict(layout=0, dtype=0, out_dtype=0, zero_rest=0, a=256, lda=16, b=256, ldb=16, b_stride=128, c=256, ldc=8,
                c_stride=0, m_splits=256, G=2, M=4, n=8, k=16, ws=256, ws_bytes=256)
    vals.update(kw)
    for k, v in vals.items():
        setattr(a, k, v)
    return g.lib().gmlp_grouped_matmul(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status,why", [
    (dict(layout=3), 1, "layout"), (dict(dtype=2), 2, "dtype"), (dict(out_dtype=1), 2, "weight gradients"),
    (dict(out_dtype=9), 1, "out_dtype"), (dict(G=0), 1, "groups"), (dict(M=-1), 2, "rows"),
    (dict(M=(1 << 30) + 1), 2, "rows"), (dict(n=0), 2, "n and k"), (dict(k=1 << 20), 2, "n and k"), (dict(a=None), 1, "null"),
    (dict(b=None), 1, "null"), (dict(c=None), 1, "null"), (dict(m_splits=None), 1, "null"), (dict(a=257), 1, "aligned"),
    (dict(lda=15), 1, "strides"), (dict(ldc=7), 1, "strides"), (dict(ldb=1 << 20), 1, "strides"),
    (dict(b_stride=127), 1, "overlap"), (dict(ws=None), 3, "workspace"), (dict(ws_bytes=8), 3, "workspace"),
    (dict(ws=264), 3, "workspace"), (dict(layout=1, lda=8, ldb=16, ldc=16, c_stride=127), 1, "overlap"),
    (dict(layout=1, lda=8, ldb=16, ldc=16, c_stride=128, c=None, M=0), 1, "null"),
    (dict(layout=1, lda=8, ldb=16, ldc=16, c_stride=128, out_dtype=1, c=258), 1, "aligned"),
    (dict(M=1 << 30, n=(1 << 20) - 8, ldc=(1 << 20) - 8, b_stride=1 << 30), 2, "one launch"),
])
def test_grouped_matmul_abi_refusals(kw, status, why):
    assert _mm(**kw) == status and why in g.last_error(), g.last_error()


def test_grouped_matmul_null_arguments():
    assert g.lib().gmlp_grouped_matmul(None, None) == 1
    assert g.lib().gmlp_grouped_matmul_ws_bytes(0, 1, 1, 1, 1, None) == 1
    assert g.grouped_matmul_ws_bytes(g.GEMM_WGRAD, 128, 65536, 4096, 7168) >= 256
