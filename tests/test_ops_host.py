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


def test_a_plan_of_other_tensors_is_refused():
    m, rows = torch.zeros(4, dtype=torch.int32), torch.zeros((8, 2), dtype=torch.int32)
    assert g.DispatchPlan(m, rows).tokens == 8
    for bad in ((m.long(), rows), (m, rows.long()), (m, rows[:, :1]), (m, rows.view(-1)), (m.view(2, 2), rows),
                (None, rows)):
        with pytest.raises(TypeError, match="int32"):
            g.DispatchPlan(*bad)
    for bad in ((m[:0], rows), (m, torch.zeros((8, 0), dtype=torch.int32))):
        with pytest.raises(ValueError, match="plan"):
            g.DispatchPlan(*bad)


def test_outputs_that_overlap_inputs_are_refused():
    """Shared elements are an error; columns of one wide tensor beside each other are not."""
    m = torch.tensor([2, 2], dtype=torch.int32)
    x, w = _t(4, 16), _t(2, 16, 16)
    with pytest.raises(ValueError, match="overlaps x"):
        g.grouped_matmul_forward(x, w, m, out=x)
    with pytest.raises(ValueError, match="overlaps dy"):
        g.grouped_matmul_dgrad(x, w, m, out=x)
    buf = _t(5, 16)
    with pytest.raises(ValueError, match="overlaps x"):
        g.grouped_matmul_forward(buf[:4], w, m, out=buf[1:])
    wide = _t(4, 40)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.grouped_matmul_forward(wide[:, :16], w, m, out=wide[:, 16:32])
    with pytest.raises(ValueError, match="overlaps x"):
        g.grouped_matmul_forward(wide[:, :16], w, m, out=wide[:, 8:24])
    plan = g.DispatchPlan(m, torch.zeros((4, 1), dtype=torch.int32))
    with pytest.raises(ValueError, match="overlaps input"):
        g.dispatch_forward(x, plan, out=x)
    a, b = _t(2, 4, 16), _t(2, 16, 4)
    ids = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="overlaps x"):
        g.lora_forward(_t(4, 16), x, a, b, ids, out=x)
    with pytest.raises(ValueError, match="overlaps base"):
        g.lora_forward(buf[:4], x, a, b, ids, out=buf[1:])
    with pytest.raises(ValueError, match="GPU tensor"):
        g.lora_forward(buf[:4], x, a, b, ids, out=buf[:4])


def test_outputs_over_splits_orders_and_scales_are_refused():
    """What a call reads besides its 16-bit tensors must not lie in its output either."""
    def beside(out, n, dtype):
        return out.view(-1).view(torch.uint8)[-n * dtype.itemsize:].view(dtype)
    x, w, dy = _t(4, 16), _t(2, 8, 16), _t(4, 8)
    y, dx, dw = _t(4, 8), _t(4, 16), _t(2, 8, 16)
    with pytest.raises(ValueError, match="out: overlaps m_splits"):
        g.grouped_matmul_forward(x, w, beside(y, 2, torch.int32), out=y)
    with pytest.raises(ValueError, match="out: overlaps m_splits"):
        g.grouped_matmul_dgrad(dy, w, beside(dx, 2, torch.int32), out=dx)
    with pytest.raises(ValueError, match="out: overlaps m_splits"):
        g.grouped_matmul_wgrad(dy, x, beside(dw, 2, torch.int32), out=dw)
    m, rows, xg = torch.zeros(3, dtype=torch.int32), torch.zeros((4, 2), dtype=torch.int32), _t(8, 16)
    with pytest.raises(ValueError, match="out: overlaps rows"):
        g.dispatch_forward(x, g.DispatchPlan(m, beside(xg, 8, torch.int32).view(4, 2)), out=xg)
    with pytest.raises(ValueError, match="out: overlaps m_splits"):
        g.dispatch_forward(x, g.DispatchPlan(beside(xg, 3, torch.int32), rows), out=xg)
    with pytest.raises(ValueError, match="out: overlaps probs"):
        g.combine_forward(xg, g.DispatchPlan(m, rows), beside(x, 8, torch.float32).view(4, 2), out=x)
    a, b = _t(2, 4, 16), _t(2, 8, 4)
    with pytest.raises(ValueError, match="out: overlaps ids"):
        g.lora_forward(None, x, a, b, beside(y, 4, torch.int32), out=y)
    with pytest.raises(ValueError, match="out: overlaps scales"):
        g.lora_forward(None, x, a, b, torch.zeros(4, dtype=torch.int32), beside(y, 2, torch.float32), out=y)


def test_a_workspace_inside_a_tensor_of_the_call_is_refused():
    """The kernels address what the tables in the workspace say, so nothing else may be written there."""
    m = torch.tensor([2, 2], dtype=torch.int32)
    x, w, dy = _t(4, 16), _t(2, 8, 16), _t(4, 8)
    y, dx, dw = _t(4, 8), _t(4, 16), _t(2, 8, 16)
    fwd = lambda ws: g.grouped_matmul_forward(x, w, m, out=y, ws=ws)
    dgrad = lambda ws: g.grouped_matmul_dgrad(dy, w, m, out=dx, ws=ws)
    wgrad = lambda ws: g.grouped_matmul_wgrad(dy, x, m, out=dw, ws=ws)
    for call, names in ((fwd, dict(x=x, w=w, out=y, m_splits=m)), (dgrad, dict(dy=dy, w=w, out=dx, m_splits=m)),
                        (wgrad, dict(dy=dy, x=x, out=dw, m_splits=m))):
        for name, t in names.items():
            with pytest.raises(ValueError, match=f"ws: overlaps {name}"):
                call(t.view(torch.uint8)[-1:])
        with pytest.raises(ValueError, match="GPU tensor"):
            call(_t(4096))
        with pytest.raises(ValueError, match="ws: a contiguous"):
            call(_t(64, 64)[:, :32])


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


def test_grouped_matmul_group_limit():
    """Each workgroup walks the groups: more than 2^16 would take minutes to hours."""
    assert _mm(G=(1 << 16) + 1, b_stride=128) == 2 and "at most 65536 groups" in g.last_error()
    assert _mm(G=1 << 24, M=1 << 24, n=1, k=1, lda=1, ldb=1, ldc=1, b_stride=1) == 2 and "65536 groups" in g.last_error()
    with pytest.raises(g.GmlpError, match="65536 groups"):
        g.grouped_matmul_ws_bytes(g.GEMM_WGRAD, (1 << 16) + 1, 4, 8, 8)
    assert g.grouped_matmul_ws_bytes(g.GEMM_WGRAD, 1 << 16, 4, 8, 8) > 0


def test_dispatch_binding_refusals():
    with pytest.raises(TypeError, match="experts"):
        g.dispatch_plan(torch.zeros((4, 2), dtype=torch.int64), 8)
    with pytest.raises(TypeError, match="experts"):
        g.dispatch_plan(torch.zeros(4, dtype=torch.int32), 8)
    with pytest.raises(g.GmlpError, match="1 to 1024 experts"):
        g.dispatch_plan(torch.zeros((4, 2), dtype=torch.int32), 1025)
    with pytest.raises(g.GmlpError, match="1 to 1024 experts"):
        g.dispatch_plan(torch.zeros((4, 2), dtype=torch.int32), 0)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.dispatch_plan(torch.zeros((4, 2), dtype=torch.int32), 8)
    plan = g.DispatchPlan(torch.zeros(3, dtype=torch.int32), torch.zeros((4, 2), dtype=torch.int32))
    with pytest.raises(ValueError, match="x: 4 rows"):
        g.dispatch_forward(_t(5, 8), plan)
    with pytest.raises(ValueError, match="v: 8 rows"):
        g.combine_forward(_t(4, 8), plan)
    with pytest.raises(TypeError, match="probs"):
        g.combine_forward(_t(8, 8), plan, torch.zeros(4, 2, dtype=torch.float64))
    with pytest.raises(TypeError, match="probs"):
        g.combine_forward(_t(8, 8), plan, torch.zeros(8))
    with pytest.raises(TypeError, match="bf16 or fp16"):
        g.dispatch_forward(torch.zeros(4, 8), plan)
    with pytest.raises(ValueError, match="out"):
        g.dispatch_forward(_t(4, 8), plan, out=_t(8, 9))
    with pytest.raises(ValueError, match="GPU tensor"):
        g.dispatch_forward(_t(4, 8), plan)
    with pytest.raises(TypeError, match="plan"):
        g.dispatch_forward(_t(4, 8), None)


def _mv(fn="gmlp_dispatch", **kw):
    a = g.MoveArgs()
    vals = dict(dtype=0, zero_rest=0, src=256, ld_src=8, src2=256, ld_src2=8, dst=256, ld_dst=8, T=4, H=8, k=2, E=3, rows=256,
                m_splits=256, probs=256, dprobs=256)
    vals.update(kw)
    for k, v in vals.items():
        setattr(a, k, v)
    return getattr(g.lib(), fn)(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status,why", [
    (dict(dtype=5), 2, "dtype"), (dict(T=-1), 2, "tokens"), (dict(k=0), 2, "tokens"), (dict(T=1 << 30, k=1), 2, "tokens"),
    (dict(H=0), 2, "H"), (dict(src=None), 1, "null"), (dict(dst=None), 1, "null"), (dict(rows=None), 1, "null"),
    (dict(zero_rest=1, m_splits=None), 1, "null"), (dict(zero_rest=1, E=0), 1, "experts"), (dict(src=257), 1, "aligned"),
    (dict(probs=258), 1, "aligned"), (dict(ld_src=7), 1, "strides"), (dict(ld_dst=7), 1, "strides"),
    (dict(fn="gmlp_combine", dst=None), 1, "null"), (dict(fn="gmlp_combine_dprobs", dprobs=None), 1, "null"),
    (dict(fn="gmlp_combine_dprobs", src2=None), 1, "null"), (dict(fn="gmlp_combine_dprobs", ld_src2=7), 1, "strides"),
])
def test_move_abi_refusals(kw, status, why):
    assert _mv(**kw) == status and why in g.last_error(), g.last_error()


def test_plan_abi_refusals():
    L = g.lib()
    p = ctypes.c_void_p(256)
    n = ctypes.c_size_t(0)
    assert L.gmlp_dispatch(None, None) == 1
    assert L.gmlp_dispatch_plan_ws_bytes(8, 3, None) == 1
    assert L.gmlp_dispatch_plan_ws_bytes(1 << 30, 3, ctypes.byref(n)) == 2
    assert L.gmlp_dispatch_plan_ws_bytes(65536, 128, ctypes.byref(n)) == 0 and n.value == 64 * 128 * 4
    assert L.gmlp_dispatch_plan(p, 65536, 128, p, p, None, None, 0, None) == 3
    assert L.gmlp_dispatch_plan(p, 8, 3, None, p, None, None, 0, None) == 1
    assert L.gmlp_dispatch_plan(None, 8, 3, p, p, None, None, 0, None) == 1
    assert L.gmlp_dispatch_plan(ctypes.c_void_p(255), 8, 3, p, p, None, None, 0, None) == 1


def _lora_args():
    return dict(base=_t(4, 8), x=_t(4, 16), a=_t(2, 4, 16), b=_t(2, 8, 4), ids=torch.zeros(4, dtype=torch.int32),
                scales=torch.ones(2))


@pytest.mark.parametrize("kw,exc,why", [
    (dict(), ValueError, "GPU tensor"), (dict(x=torch.zeros(4, 16)), TypeError, "bf16 or fp16"),
    (dict(a=_t(2, 4, 16, dtype=torch.float16)), TypeError, "a:"), (dict(x=_t(4, 15)), ValueError, "16 elements"),
    (dict(b=_t(2, 8, 5)), ValueError, "b:"), (dict(b=_t(3, 8, 4)), ValueError, "b:"),
    (dict(ids=torch.zeros(4, dtype=torch.int64)), TypeError, "ids"), (dict(ids=torch.zeros(5, dtype=torch.int32)), TypeError, "ids"),
    (dict(scales=torch.ones(3)), TypeError, "scales"), (dict(scales=torch.ones(2).half()), TypeError, "scales"),
    (dict(base=_t(4, 9)), ValueError, "base"), (dict(out=_t(4, 9)), ValueError, "out"),
    (dict(a=_t(2, 129, 16), b=_t(2, 8, 129)), ValueError, "GPU tensor"),
])
def test_lora_binding_refusals(kw, exc, why):
    args = _lora_args()
    args.update(kw)
    with pytest.raises(exc, match=why):
        g.lora_forward(**args)


def test_lora_sizes_and_scale_gradient_refused():
    with pytest.raises(g.GmlpError, match="ranks 1 to 128"):
        g.lora_query_sizes(4, 16, 8, 129, 2)
    with pytest.raises(g.GmlpError, match="1 to 1023 adapters"):
        g.lora_query_sizes(4, 16, 8, 4, 1024)
    with pytest.raises(g.GmlpError, match="K and N"):
        g.lora_query_sizes(4, 0, 8, 4, 2)
    a = _lora_args()
    a["scales"].requires_grad_()
    with pytest.raises(ValueError, match="scales"):
        g.lora(**a)
    with pytest.raises(TypeError, match="ctx"):
        g.lora_backward(_t(4, 8), _t(4, 16), _t(2, 4, 16), _t(2, 8, 4), None)


def test_lora_context_of_another_size_is_refused():
    """The kernels address the context by the call's sizes, not by the buffer's."""
    need = g.lora_query_sizes(4, 16, 8, 4, 2)["ctx_bytes"]
    args = (_t(4, 8), _t(4, 16), _t(2, 4, 16), _t(2, 8, 4))

    def ctx(buf):
        return g.LoraContext(buf, 4, 16, 8, 4, 2, torch.bfloat16, None)
    u8 = dict(dtype=torch.uint8)
    for buf in (torch.zeros(need - 1, **u8), torch.zeros(0, **u8), torch.zeros((need, 2), **u8)[:, 0]):
        with pytest.raises(ValueError, match="ctx: a contiguous buffer"):
            g.lora_backward(*args, ctx(buf))
    with pytest.raises(ValueError, match="GPU tensor"):
        g.lora_backward(*args, ctx(torch.zeros(need, **u8)))


def _lf(**kw):
    a = g.LoraFwdArgs()
    w = dict(a=256, lda=16, a_stride=64, b=256, ldb=4, b_stride=32, scales=256)
    vals = dict(dtype=0, R=4, L=2, M=4, K=16, N=8, base=256, ldbase=8, x=256, ldx=16, ids=256, y=256, ldy=8, ctx=256,
                ctx_bytes=1 << 20, ws=256, ws_bytes=1 << 20)
    for k, v in kw.items():
        (w if k in w else vals)[k] = v
    for k, v in vals.items():
        setattr(a, k, v)
    a.w = g.LoraWeights(*[w[k] for k in ("a", "lda", "a_stride", "b", "ldb", "b_stride", "scales")])
    return g.lib().gmlp_lora_forward(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status,why", [
    (dict(dtype=3), 2, "dtype"), (dict(R=0), 2, "ranks"), (dict(L=0), 2, "adapters"), (dict(M=-1), 2, "rows"),
    (dict(x=None), 1, "null"), (dict(ids=None), 1, "null"), (dict(y=None), 1, "null"), (dict(a=None), 1, "null"),
    (dict(b=None), 1, "null"), (dict(x=257), 1, "aligned"), (dict(scales=258), 1, "aligned"), (dict(lda=15), 1, "strides"),
    (dict(ldb=3), 1, "strides"), (dict(a_stride=63), 1, "overlap"), (dict(ldx=15), 1, "strides"), (dict(ldy=7), 1, "strides"),
    (dict(ldbase=16), 1, "two row strides"), (dict(ctx=None), 3, "ctx"), (dict(ctx_bytes=16), 3, "ctx"), (dict(ctx=264), 3, "ctx"),
    (dict(M=20000, ctx_bytes=1 << 30, ws=None), 3, "workspace"), (dict(M=0, x=None, y=None, ids=None, ctx=None), 0, ""),
])
def test_lora_abi_refusals(kw, status, why):
    assert _lf(**kw) == status and why in g.last_error(), g.last_error()


def _lb(**kw):
    a = g.LoraBwdArgs()
    w = dict(a=256, lda=16, a_stride=64, b=256, ldb=4, b_stride=32, scales=256)
    vals = dict(dtype=0, R=4, L=2, M=4, K=16, N=8, dy=256, lddy=8, x=256, ldx=16, dx_add=None, lddx_add=0, dx=256, lddx=16,
                da=256, db=256, ctx=256, ctx_bytes=1 << 20, ws=256, ws_bytes=1 << 24)
    for k, v in kw.items():
        (w if k in w else vals)[k] = v
    for k, v in vals.items():
        setattr(a, k, v)
    a.w = g.LoraWeights(*[w[k] for k in ("a", "lda", "a_stride", "b", "ldb", "b_stride", "scales")])
    return g.lib().gmlp_lora_backward(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status,why", [
    (dict(dy=None), 1, "null"), (dict(x=None), 1, "null"), (dict(ctx=None), 1, "null"), (dict(da=257), 1, "aligned"),
    (dict(lddx=15), 1, "strides"), (dict(lddy=7), 1, "strides"), (dict(dx_add=256, lddx_add=24), 1, "two row strides"),
    (dict(ctx_bytes=8), 3, "ctx"), (dict(ws=None), 3, "workspace"), (dict(ws_bytes=64), 3, "workspace"),
])
def test_lora_backward_abi_refusals(kw, status, why):
    assert _lb(**kw) == status and why in g.last_error(), g.last_error()
