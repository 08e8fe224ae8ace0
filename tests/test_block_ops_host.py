"""Refusals of the operators around the experts (CPU): bad arguments are errors before anything is launched, in the
binding and in the C ABI; and the C ABI's host code under the sanitizers."""
import dataclasses
import ctypes
import os
import shutil

import pytest
import torch

import nvfp4_block_scaled_mxfp8_amd as g
from test_host_sanitizers import CSRC, FLAGS, ROCM, SAN, _run


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32)


# ----------------------------------------------------------------------------- binding
def test_route_refuses():
    l = _t(4, 8, dtype=torch.float32)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.route_forward(l, 2)
    with pytest.raises(TypeError, match="logits"):
        g.route_forward(l.double(), 2)
    with pytest.raises(ValueError, match="T, E"):
        g.route_forward(l[0], 2)
    with pytest.raises(ValueError, match="T, E"):
        g.route_forward(l[:, :0], 1)
    with pytest.raises(ValueError, match="score"):
        g.route_forward(l, 2, "tanh")
    with pytest.raises(TypeError, match="bias"):
        g.route_forward(l, 2, bias=_t(8))
    with pytest.raises(TypeError, match="bias"):
        g.route_forward(l, 2, bias=_t(7, dtype=torch.float32))
    with pytest.raises(ValueError, match="bias"):
        g.route_forward(l, 2, bias=_t(8, dtype=torch.float32).to("meta"))
    for k in (0, -1, 2.0):
        with pytest.raises(ValueError, match="k:"):
            g.route_forward(l, k)
    with pytest.raises(ValueError, match="no gradient"):
        g.route(l, 2, bias=_t(8, dtype=torch.float32).requires_grad_())
    d, e = _t(4, 2, dtype=torch.float32), torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(TypeError, match="experts"):
        g.route_backward(d, l, e.long())
    with pytest.raises(TypeError, match="experts"):
        g.route_backward(d, l, e[:3])
    with pytest.raises(TypeError, match="dprobs"):
        g.route_backward(d.half(), l, e)
    with pytest.raises(TypeError, match="dprobs"):
        g.route_backward(d[:, :1], l, e)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.route_backward(d, l, e)


def test_norms_refuse():
    x, w = _t(4, 16), _t(16)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.residual_norm_forward(x, x, w)
    with pytest.raises(TypeError, match="bf16 or fp16"):
        g.residual_norm_forward(x.float(), x.float(), w)
    with pytest.raises(ValueError, match="dimensions"):
        g.residual_norm_forward(x[0], x[0], w)
    with pytest.raises(TypeError, match="branch"):
        g.residual_norm_forward(x, x.half(), w)
    with pytest.raises(ValueError, match="branch"):
        g.residual_norm_forward(x, x[:, :8], w)
    for name in ("weight", "branch_weight"):
        with pytest.raises(TypeError, match=name):
            g.residual_norm_forward(x, x, **{name: w.half()})
        with pytest.raises(ValueError, match=name):
            g.residual_norm_forward(x, x, **{name: _t(15)})
    with pytest.raises(TypeError, match="gate"):
        g.residual_norm_forward(x, x, w, gate=_t(4, 1, dtype=torch.float16))
    for shape in ((15,), (3, 1), (4, 15), (1, 16), (4, 16, 1)):
        with pytest.raises(ValueError, match="gate"):
            g.residual_norm_forward(x, x, w, gate=_t(*shape))
    with pytest.raises(TypeError, match="branch"):
        g.residual_norm(x, None, w)
    with pytest.raises(TypeError, match="weight"):
        g.rms_norm(x, None)
    with pytest.raises(TypeError, match="weight"):
        g.rms_norm_forward(x, None)


def test_w4_refuses():
    x, m = _t(4, 64), _i32(2, 2)
    codes, scales = _t(2, 8, 32, dtype=torch.uint8), _t(2, 8, 2)
    w = g.Int4Weights(codes, scales)
    assert (w.K, w.group) == (64, 32)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.grouped_matmul_w4(x, w, m)
    with pytest.raises(TypeError, match="bf16 or fp16"):
        g.grouped_matmul_w4(x.float(), w, m)
    with pytest.raises(TypeError, match="scales"):
        g.grouped_matmul_w4(x.half(), w, m)
    with pytest.raises(ValueError, match="no gradient"):
        g.grouped_matmul_w4(x.clone().requires_grad_(), w, m)
    with pytest.raises(ValueError, match="w:"):
        g.grouped_matmul_w4(_t(4, 128), w, m)
    with pytest.raises(ValueError, match="w:"):
        g.grouped_matmul_w4(x, w, _i32(4))
    with pytest.raises(TypeError, match="m_splits"):
        g.grouped_matmul_w4(x, w, m.long())
    with pytest.raises(TypeError, match="w:"):
        g.grouped_matmul_w4(x, codes, m)
    with pytest.raises(ValueError, match="out"):
        g.grouped_matmul_w4(x, w, m, out=_t(4, 9))
    for bad in ((codes.int(), scales), (codes[0], scales[0]), (codes[:, ::2], scales[:, ::2])):
        with pytest.raises(TypeError, match="codes"):
            g.Int4Weights(*bad)
    for bad in (_t(2, 8, 4), _t(2, 8, 3), _t(2, 7, 2), _t(2, 8, 0), _t(2, 16, 2)[:, ::2]):
        with pytest.raises(ValueError, match="scales"):
            g.Int4Weights(codes, bad)
    with pytest.raises(TypeError, match="scales"):
        g.Int4Weights(codes, scales.float())
    for bad in (_t(2, 8, 2), _t(2, 8, 1, dtype=torch.uint8)):
        with pytest.raises(TypeError, match="zeros"):
            g.Int4Weights(codes, scales, bad)
    for name, bad in (("codes", codes[:1]), ("scales", scales[:1]), ("zeros", _t(1, 8, 2, dtype=torch.uint8))):
        with pytest.raises(dataclasses.FrozenInstanceError):           # would be read past its end
            setattr(w, name, bad)
    q = {"row_data": codes.reshape(-1), "row_scale": _t(2 * 8 * 4, dtype=torch.uint8), "amax_pre": _t(2, dtype=torch.float32)}
    with pytest.raises(ValueError, match="GPU tensor"):
        g.grouped_matmul_w4(x, g.QTensor(g.NVFP4_RHT, q), m)
    with pytest.raises(ValueError, match="4-bit"):
        g.grouped_matmul_w4(x, g.QTensor(g.MXFP8, q), m)
    for name, bad in (("row_data", codes.reshape(-1)[:500]), ("row_scale", q["row_scale"][:-1]), ("amax_pre", q["amax_pre"][:1]), ("amax_pre", None),
                      ("row_data", codes.reshape(-1)[::2])):
        with pytest.raises(ValueError, match="w:"):
            g.grouped_matmul_w4(x, g.QTensor(g.NVFP4_RHT, {**q, name: bad}), m)
    with pytest.raises(TypeError, match="w:"):
        g.grouped_matmul_w4(x, g.QTensor(g.NVFP4_RHT, {**q, "row_scale": _t(64)}), m)


def test_w4_refuses_an_nvfp4_weight_of_another_width():
    """The weight's own K is held against x's, not inferred from it: rows of 64 read as twice as many of 32 would be other
    weights."""
    codes, scales, amax = _t(2, 8, 32, dtype=torch.uint8), _t(2, 8, 4, dtype=torch.uint8), _t(2, dtype=torch.float32)
    flat = {"row_data": codes.reshape(-1), "row_scale": scales.reshape(-1), "amax_pre": amax}
    m = _i32(2, 2)
    for bufs, shape in (({**flat, "row_data": codes}, None), ({**flat, "row_scale": scales}, None), (flat, (2, 8, 64))):
        w = g.QTensor(g.NVFP4_RHT, bufs, shape)
        with pytest.raises(ValueError, match="GPU tensor"):                   # the width that it has
            g.grouped_matmul_w4(_t(4, 64), w, m)
        for K in (32, 128):
            with pytest.raises(ValueError, match="^w:"):
                g.grouped_matmul_w4(_t(4, K), w, m)
    with pytest.raises(ValueError, match="^w:"):                              # the number of weights too
        g.grouped_matmul_w4(_t(4, 64), g.QTensor(g.NVFP4_RHT, flat, (1, 16, 64)), m)
    with pytest.raises(ValueError, match="^w:"):
        g.grouped_matmul_w4(_t(4, 64), g.QTensor(g.NVFP4_RHT, flat), _i32())
    # what the library makes says what it is
    rec = g.recipe("nvfp4", 0x1234)
    w = g.alloc_weight_q(rec, 2, 128, 256, device="cpu")
    assert w.shape == (2, 128, 256)
    with pytest.raises(ValueError, match="GPU tensor"):
        g.grouped_matmul_w4(_t(4, 256), w, m)
    with pytest.raises(ValueError, match="^w:"):
        g.grouped_matmul_w4(_t(4, 128), w, m)
    assert g.alloc_grouped_q(rec, 128, 256, 2, device="cpu").shape is None


def test_w4_refuses_scales_that_wait_for_a_gradient():
    """They would get none; without autograd they are numbers like others."""
    x, m = _t(4, 64), _i32(2, 2)
    scales = _t(2, 8, 2).requires_grad_()
    amax = _t(2, dtype=torch.float32).requires_grad_()
    flat = {"row_data": _t(512, dtype=torch.uint8), "row_scale": _t(64, dtype=torch.uint8), "amax_pre": amax}
    for w in (g.Int4Weights(_t(2, 8, 32, dtype=torch.uint8), scales), g.QTensor(g.NVFP4_RHT, flat)):
        with pytest.raises(ValueError, match="^w: no gradient"):
            g.grouped_matmul_w4(x, w, m)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU tensor"):
            g.grouped_matmul_w4(x, w, m)


# ----------------------------------------------------------------------------- C ABI
P = 1 << 20          # an address that is aligned to everything and never read: each call is refused, or has no rows


def _call(name, args):
    return g.lib()[name](ctypes.byref(args), None) if args is not None else g.lib()[name](None, None)


def _refused(name, make, status, text, **change):
    a = make()
    for k, v in change.items():
        s = a.inputs if hasattr(a, "inputs") and hasattr(a.inputs, k) else a
        assert hasattr(s, k), k
        setattr(s, k, v)
    assert _call(name, a) == status, (name, change, g.last_error())
    assert text in g.last_error(), (name, change, g.last_error())


def _route():
    return g.RouteArgs(2, 0, P, 16, 4, 16, 4, None, 1, 1, 1, 1, 1.0, P, P)


def _route_bwd():
    return g.RouteBwdArgs(2, 0, P, 16, 4, 16, 4, P, P, 1, 1.0, P, 16)


@pytest.mark.parametrize("name,make", [("gmlp_route", _route), ("gmlp_route_backward", _route_bwd)])
def test_route_abi(name, make):
    assert _call(name, None) == 1
    for change, status, text in (({"dtype": 3}, 2, "dtype"), ({"dtype": -1}, 2, "dtype"), ({"score": 2}, 1, "score"), ({"T": -1}, 2, "T = "),
                                 ({"T": (1 << 30) + 1}, 2, "T = "), ({"E": 0}, 2, "experts"), ({"E": 1025, "ld": 2000}, 2, "experts"),
                                 ({"k": 0}, 2, "k must"), ({"k": 65}, 2, "k must"), ({"scale": float("inf")}, 1, "scale"),
                                 ({"scale": float("nan")}, 1, "scale"), ({"logits": None}, 1, "null"), ({"experts": None}, 1, "null"),
                                 ({"logits": P + 2}, 1, "aligned"), ({"experts": P + 2}, 1, "aligned"), ({"ld": 15}, 1, "strides")):
        _refused(name, make, status, text, **change)
    empty = make()
    empty.T = 0
    empty.logits = empty.experts = None
    assert _call(name, empty) == 0


def test_route_abi_groups_and_outputs():
    for change, status, text in (({"groups": 0}, 2, "groups"), ({"groups": 3}, 2, "groups"), ({"groups": 65, "E": 650, "ld": 650}, 2, "groups"),
                                 ({"top_groups": 2}, 1, "top_groups"), ({"groups": 4, "top_groups": 0}, 1, "top_groups"),
                                 ({"group_best": 3}, 2, "group_best"), ({"group_best": 0}, 2, "group_best"), ({"k": 17}, 1, "k = 17"),
                                 ({"groups": 4, "k": 5}, 1, "k = 5"), ({"probs": None}, 1, "null"), ({"probs": P + 2}, 1, "aligned"),
                                 ({"bias": P + 2}, 1, "aligned")):
        _refused("gmlp_route", _route, status, text, **change)
    for change, status, text in (({"dprobs": None}, 1, "null"), ({"dlogits": None}, 1, "null"), ({"dprobs": P + 1}, 1, "aligned"),
                                 ({"dlogits": P + 2}, 1, "aligned"), ({"ld_dlogits": 15}, 1, "strides")):
        _refused("gmlp_route_backward", _route_bwd, status, text, **change)


def _inputs():
    return g.NormInputs(0, 1, 0, 0, 0, 1e-6, 0.5, 4, 16, P, 16, P, 16, P, P, P, 16)


def _norm():
    return g.NormArgs(_inputs(), P, 16, P, 16, P)


def _norm_bwd():
    return g.NormBwdArgs(_inputs(), P, 16, P, 16, P, P, 16, P, 16, P, P, P, P, 1 << 20)


@pytest.mark.parametrize("name,make", [("gmlp_residual_norm", _norm), ("gmlp_residual_norm_backward", _norm_bwd)])
def test_norm_abi(name, make):
    assert _call(name, None) == 1
    inf, nan = float("inf"), float("nan")
    for change, status, text in (({"dtype": 2}, 2, "dtype"), ({"T": -1}, 2, "T = "), ({"T": (1 << 30) + 1}, 2, "T = "), ({"H": 0}, 2, "H must"),
                                 ({"H": 32769}, 2, "H must"), ({"gate_kind": 4}, 1, "gate_kind"), ({"gate_kind": -1}, 1, "gate_kind"),
                                 ({"eps": -1.0}, 1, "eps"), ({"eps": nan}, 1, "eps"), ({"eps": inf}, 1, "eps"), ({"scale": nan}, 1, "scale"),
                                 ({"scale": inf}, 1, "scale"), ({"branch": None}, 1, "branch"), ({"x": None}, 1, "null"), ({"gate": None}, 1, "null"),
                                 ({"x": P + 1}, 1, "aligned"), ({"branch": P + 1}, 1, "aligned"), ({"weight": P + 1}, 1, "aligned"),
                                 ({"weight": P + 2, "weight_fp32": 1}, 1, "aligned"), ({"branch_weight": P + 2, "branch_weight_fp32": 1}, 1, "aligned"),
                                 ({"gate": P + 2, "gate_fp32": 1}, 1, "aligned"), ({"ldx": 15}, 1, "strides"), ({"ldbranch": 15}, 1, "strides"),
                                 ({"gate_kind": 3, "ld_gate": 15}, 1, "strides"), ({"gate_kind": 2, "ld_gate": 0}, 1, "strides")):
        _refused(name, make, status, text, **change)
    nothing = dict(branch=None, branch_weight=None, gate=None, gate_kind=0, scale=1.0, weight=None)
    _refused(name, make, 1, "nothing", **nothing)


def test_norm_abi_outputs():
    for change, status, text in (({"y": None}, 1, "null"), ({"h": None}, 1, "null"), ({"y": P + 1}, 1, "aligned"), ({"h": P + 1}, 1, "aligned"),
                                 ({"stats": P + 2}, 1, "aligned"), ({"ldy": 15}, 1, "strides"), ({"ldh": 15}, 1, "strides"),
                                 ({"ldy": 17}, 1, "two row strides")):
        _refused("gmlp_residual_norm", _norm, status, text, **change)
    need = ctypes.c_size_t(0)
    assert g.lib().gmlp_residual_norm_bwd_ws_bytes(4, 16, ctypes.byref(need)) == 0 and need.value > 0
    for T, H in ((-1, 16), ((1 << 30) + 1, 16), (4, 0), (4, 32769)):
        assert g.lib().gmlp_residual_norm_bwd_ws_bytes(T, H, ctypes.byref(need)) == 2
    assert g.lib().gmlp_residual_norm_bwd_ws_bytes(4, 16, None) == 1
    for change, status, text in (({"dh": None}, 1, "dh"), ({"weight": None, "dweight": None}, 1, "dh"), ({"stats": None}, 1, "null"),
                                 ({"branch_weight": None}, 1, "not there"), ({"gate_kind": 0}, 1, "not there"),
                                 ({"dy": P + 1}, 1, "aligned"), ({"dx": P + 1}, 1, "aligned"), ({"dbranch": P + 1}, 1, "aligned"),
                                 ({"dgate": P + 2, "gate_fp32": 1}, 1, "aligned"), ({"lddy": 15}, 1, "strides"), ({"lddh": 15}, 1, "strides"),
                                 ({"lddx": 15}, 1, "strides"), ({"lddbranch": 15}, 1, "strides"), ({"ws": None}, 3, "workspace"),
                                 ({"ws": P + 8}, 3, "workspace"), ({"ws_bytes": 16}, 3, "workspace")):
        _refused("gmlp_residual_norm_backward", _norm_bwd, status, text, **change)


def _w4():
    return g.W4Args(0, 0, 32, 1, P, 64, P, P, None, None, P, 8, P, 2, 4, 8, 64)


def test_w4_abi():
    name = "gmlp_grouped_matmul_four_bit"
    assert _call(name, None) == 1
    for change, status, text in (({"dtype": 2}, 2, "dtype"), ({"kind": 2}, 1, "kind"), ({"group": 16}, 2, "group"), ({"group": 256}, 2, "group"),
                                 ({"kind": 1}, 2, "group"), ({"M": -1}, 2, "M = "), ({"M": (1 << 30) + 1}, 2, "M = "), ({"G": 0}, 2, "groups"),
                                 ({"G": 65537}, 2, "groups"), ({"N": 0}, 2, "N and K"), ({"N": 1 << 20}, 2, "N and K"), ({"K": 0}, 2, "N and K"),
                                 ({"K": 48}, 2, "multiple"), ({"K": 96, "ldx": 96, "group": 64}, 2, "multiple"),
                                 ({"K": 48, "kind": 1, "group": 16}, 2, "multiple"), ({"x": None}, 1, "null"), ({"codes": None}, 1, "null"),
                                 ({"scales": None}, 1, "null"), ({"y": None}, 1, "null"), ({"m_splits": None}, 1, "null"),
                                 ({"kind": 1, "group": 16}, 1, "null"), ({"kind": 1, "group": 16, "amax": P, "zeros": P}, 1, "zeros"),
                                 ({"x": P + 1}, 1, "aligned"), ({"codes": P + 8}, 1, "aligned"), ({"scales": P + 1}, 1, "aligned"),
                                 ({"y": P + 1}, 1, "aligned"), ({"m_splits": P + 2}, 1, "aligned"), ({"ldx": 63}, 1, "strides"),
                                 ({"ldy": 7}, 1, "strides"), ({"ldx": 1 << 20}, 1, "strides"),
                                 ({"M": 1 << 30, "N": (1 << 20) - 1, "ldy": (1 << 20) - 1}, 2, "one launch")):
        _refused(name, _w4, status, text, **change)
    empty = _w4()
    empty.M = 0
    empty.x = empty.y = None
    assert _call(name, empty) == 0


# ----------------------------------------------------------------------------- sanitizers
@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "lib", "libamdhip64.so")),
                    reason="needs g++ and the HIP runtime library")
def test_host_code_under_asan_and_ubsan(tmp_path):
    hip = ["-L" + os.path.join(ROCM, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(ROCM, "lib")]
    drv = str(tmp_path / "block_ops_driver")
    src = [os.path.join(CSRC, "api.cpp"), os.path.join(CSRC, "block_ops.cpp")] + \
        [os.path.join(SAN, f) for f in ("launch_stubs.cpp", "block_ops_driver.cpp")]
    _run(["g++"] + FLAGS + src + ["-o", drv] + hip)
    out = _run([drv], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
                               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1"))
    text = out.stdout + out.stderr
    assert "AddressSanitizer" not in text and "runtime error" not in text, text
    assert "all statuses as expected" in text
