"""The operators around the experts together, as a layer uses them: norm, router, dispatch, experts, combine, residual
sum and the next norm; in training with 16-bit experts under autograd, in decoding with 4-bit experts captured
into a graph, and around the quantized grouped MLP."""
import pytest
import torch

import nvfp4_block_scaled_mxfp8_amd as g
from block_util import int4_values, nvfp4_values
from mm_util import randn

pytestmark = pytest.mark.gpu

T, E, k, H, F = 96, 8, 3, 256, 128
SCALE = 0.5


def _err(a, b):
    return float((a.detach().cpu().double() - b).norm() / b.norm())


def _inputs(dtype):
    return {"x": randn((T, H), dtype, 1), "wn": 1 + randn((H,), torch.float32, 2, 0.1), "wr": randn((E, H), torch.float32, 3, H ** -0.5),
            "w1": randn((E, 2 * F, H), dtype, 4, H ** -0.5), "w2": randn((E, H, F), dtype, 5, F ** -0.5),
            "wp": 1 + randn((H,), torch.float32, 6, 0.1), "gate": 1 + randn((H,), torch.float32, 7, 0.1),
            "wl": 1 + randn((H,), torch.float32, 8, 0.1)}


def _swiglu(h):
    return (torch.nn.functional.silu(h[:, :F].float()) * h[:, F:].float()).to(h.dtype)


def _layer(v):
    h = g.rms_norm(v["x"], v["wn"])
    experts, probs = g.route(h.float() @ v["wr"].t(), k, "sigmoid", scale=1.5)
    plan = g.dispatch_plan(experts, E)
    rows = g.grouped_matmul(_swiglu(g.grouped_matmul(g.dispatch(h, plan), v["w1"], plan.m_splits)), v["w2"], plan.m_splits)
    y, last = g.residual_norm(v["x"], g.combine(rows, plan, probs), v["wl"], v["wp"], v["gate"], SCALE)
    return y, last, experts


def _norm(x, w):
    return x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6) * w


def _plain(v, experts, w1, w2, norm=True):
    """The same in 64 bits on the CPU, with the experts given."""
    h = _norm(v["x"], v["wn"])
    s = torch.sigmoid(h @ v["wr"].t()).gather(1, experts)
    probs = 1.5 * s / s.sum(1, keepdim=True)
    out = torch.zeros_like(h)
    for e in range(E):
        t, j = (experts == e).nonzero(as_tuple=True)
        if t.numel():
            a = h[t] @ w1[e].t()
            out = out.index_add(0, t, probs[t, j][:, None] * ((torch.nn.functional.silu(a[:, :F]) * a[:, F:]) @ w2[e].t()))
    y = v["x"] + SCALE * v["gate"] * _norm(out, v["wp"])
    return y, _norm(y, v["wl"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_training_layer_forward_and_gradients(dtype):
    """Relative Frobenius errors: a value passes about twelve roundings of the type on its way (norm, product, activation,
    product, combine, sum, norm and their gradients), independent ones, so sqrt(12) half steps; held to four times that."""
    d = _inputs(dtype)
    dev = {n: t.cuda().requires_grad_() for n, t in d.items()}
    y, last, experts = _layer(dev)
    dy, dl = randn((T, H), dtype, 11), randn((T, H), dtype, 12)
    torch.autograd.backward([y, last], [dy.cuda(), dl.cuda()])
    ref = {n: t.double().requires_grad_() for n, t in d.items()}
    want = _plain(ref, experts.cpu().long(), ref["w1"], ref["w2"])
    torch.autograd.backward(want, [dy.double(), dl.double()])
    tol = 4 * 12 ** 0.5 * torch.finfo(dtype).eps / 2
    assert _err(y, want[0].detach()) <= tol and _err(last, want[1].detach()) <= tol
    for n in d:
        assert _err(dev[n].grad, ref[n].grad) <= tol, (n, _err(dev[n].grad, ref[n].grad), tol)


def _quantized(d, seed):
    """w1 as integers by groups of 64, w2 as the library's NVFP4, and what both stand for."""
    gen = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (E, 2 * F, H // 2), dtype=torch.uint8, generator=gen)
    scales = (torch.rand((E, 2 * F, H // 64), generator=gen) / (4 * H ** 0.5)).to(d["x"].dtype)
    zeros = torch.randint(6, 10, (E, 2 * F, H // 64), dtype=torch.uint8, generator=gen)
    q2 = g.weight_quantize(d["w2"].to(torch.bfloat16).cuda(), g.recipe("nvfp4", 0x1111))
    v2 = nvfp4_values(q2.bufs["row_data"].cpu().view(E, H, F // 2), q2.bufs["row_scale"].cpu().view(E, H, F // 16), q2.bufs["amax_pre"].cpu())
    return g.Int4Weights(codes.cuda(), scales.cuda(), zeros.cuda()), q2, int4_values(codes, scales, zeros), v2


def _decode(v, w1, w2, out=None):
    h, _ = g.rms_norm_forward(v["x"], v["wn"])
    experts, probs = g.route_forward((h.float()[:, None, :] * v["wr"][None]).sum(2), k, "sigmoid", scale=1.5)
    plan = g.dispatch_plan(experts, E)
    rows = g.grouped_matmul_w4(_swiglu(g.grouped_matmul_w4(g.dispatch_forward(h, plan), w1, plan.m_splits)), w2, plan.m_splits)
    y, last, _ = g.residual_norm_forward(v["x"], g.combine_forward(rows, plan, probs), v["wl"], v["wp"], v["gate"], SCALE, out=out)
    return y, last, experts


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_decode_layer(dtype):
    """As above without gradients: about seven roundings."""
    d = _inputs(dtype)
    w1, w2, v1, v2 = _quantized(d, 5)
    y, last, experts = _decode({n: t.cuda() for n, t in d.items()}, w1, w2)
    want = _plain({n: t.double() for n, t in d.items()}, experts.cpu().long(), v1, v2)
    tol = 4 * 7 ** 0.5 * torch.finfo(dtype).eps / 2
    assert _err(y, want[0]) <= tol and _err(last, want[1]) <= tol


def test_decode_layer_captured_and_replayed():
    """The residual stream updated in place; eager work of the same layer between the replays."""
    d = _inputs(torch.bfloat16)
    w1, w2, _, _ = _quantized(d, 6)
    v = {n: t.cuda() for n, t in d.items()}
    first, second = v["x"].clone(), v["x"].flip(0).contiguous()
    refs = []
    for x in (first, second):
        v["x"].copy_(x)
        refs.append([t.clone() for t in _decode(v, w1, w2, out=v["x"])])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _decode(v, w1, w2)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _decode(v, w1, w2, out=v["x"])
    for r in range(4):
        other = dict(v, x=second.clone())
        _decode(other, w1, w2)
        v["x"].copy_(first if r % 2 == 0 else second)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert out[0].data_ptr() == v["x"].data_ptr()
        assert all(torch.equal(a, b) for a, b in zip(refs[r % 2], out)), r
    del graph


def test_routed_tokens_through_the_quantized_mlp():
    """route and the norms around dispatch and grouped_mlp: the sum of the rows it gives, by hand."""
    d = _inputs(torch.bfloat16)
    v = {n: t.cuda() for n, t in d.items()}
    rec = g.recipe("mxfp8")
    h, _ = g.rms_norm_forward(v["x"], v["wn"])
    experts, probs = g.route_forward(h.float() @ v["wr"].t(), k)
    plan = g.dispatch_plan(experts, E)
    by_row = torch.empty(T * k, device="cuda")
    by_row[plan.rows.flatten().long()] = probs.flatten()
    rows = g.grouped_mlp(g.dispatch(h, plan), by_row, v["w1"], v["w2"], plan.m_splits, "swiglu", rec)
    out = g.combine_forward(rows, plan)
    y, _, _ = g.residual_norm_forward(v["x"], out)
    want = v["x"].double() + out.double()
    # one rounding of the sum (the addition itself is exact to 2^-24)
    assert bool(((y.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs() + 2.0 ** -23 * out.double().abs()).all())


def test_other_stream_and_two_calls_at_once():
    """The same inputs on two streams at once, backward and forward: each call's scratch is its own."""
    d = _inputs(torch.bfloat16)
    v = {n: t.cuda() for n, t in d.items()}
    big = {"x": randn((3000, 2048), torch.bfloat16, 21).cuda(), "b": randn((3000, 2048), torch.bfloat16, 22).cuda()}
    w = (1 + randn((2048,), torch.float32, 23, 0.1)).cuda()
    gate = (1 + randn((2048,), torch.float32, 24, 0.1)).cuda()
    logits = randn((3000, 64), torch.float32, 25).cuda()

    def step():
        y, h, st = g.residual_norm_forward(big["x"], big["b"], w, w, gate)
        r = g.residual_norm_backward(big["b"], big["x"], big["x"], big["b"], st, w, w, gate)
        e, p = g.route_forward(logits, 4, "sigmoid", bias=w[:64].contiguous())
        return [y, h, *r.values(), e, p, g.route_backward(p, logits, e, "sigmoid")]
    ref = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[i].append(step())
    torch.cuda.synchronize()
    for outs in got:
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(ref, o))
    del v
