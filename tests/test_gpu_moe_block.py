"""The 16-bit operators together, as a layer uses them: tokens routed to experts, a gated MLP of two
grouped products with low-rank adapters of the requests on each expert projection, combined back;
forward and gradients under autograd, beside the quantized grouped MLP on the same order."""
import pytest
import torch

import nvfp4_block_scaled_mxfp8_amd as g
from mm_util import randn

pytestmark = pytest.mark.gpu

T, k, E, H, F, R, L = 96, 3, 5, 128, 256, 8, 4          # L requests' adapters, one per expert each


def _inputs(dtype):
    gen = torch.Generator().manual_seed(3)
    score = torch.rand((T, E), generator=gen)
    score[:, 2] = -1.0                                    # an expert without tokens
    top, experts = score.topk(k, dim=1)
    d = {"x": randn((T, H), dtype, 1), "w1": randn((E, 2 * F, H), dtype, 2, H ** -0.5), "w2": randn((E, H, F), dtype, 3, F ** -0.5),
         "a": randn((L * E, R, H), dtype, 4, H ** -0.5), "b": randn((L * E, 2 * F, R), dtype, 5, 0.5),
         "probs": torch.softmax(top, 1), "dy": randn((T, H), dtype, 6)}
    experts[5, 1] = -1                                    # a dropped slot
    request = torch.arange(T) * L // T
    request[-7:] = -1                                     # rows of no request
    return d, experts.to(torch.int32), request.to(torch.int32)


def _layer(v, experts, request):
    plan = g.dispatch_plan(experts, E)
    xg = g.dispatch(v["x"], plan)
    # the adapter of a row: its token's request, at its expert
    rows = plan.rows.flatten()
    ids = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    per_slot = torch.where((request[:, None] >= 0), request[:, None] * E + experts, -1).flatten().to(torch.int32)
    live = rows >= 0
    ids.index_copy_(0, torch.where(live, rows, T * k - 1).long(), torch.where(live, per_slot, -1))
    h = g.lora(g.grouped_matmul(xg, v["w1"], plan.m_splits), xg, v["a"], v["b"], ids)
    act = (torch.nn.functional.silu(h[:, :F].float()) * h[:, F:].float()).to(h.dtype)
    return g.combine(g.grouped_matmul(act, v["w2"], plan.m_splits), plan, v["probs"])


def _plain(v, experts, request):
    """The same in 64 bits, token by token and expert by expert, on the CPU."""
    y = torch.zeros((T, H), dtype=torch.float64)
    for e in range(E):
        t, j = (experts == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        h = v["x"][t] @ v["w1"][e].t()
        for r in range(L):
            m = (request[t] == r).nonzero().flatten()
            if m.numel():
                i = r * E + e
                h = h.index_add(0, m, v["x"][t[m]] @ v["a"][i].t() @ v["b"][i].t())
        out = (torch.nn.functional.silu(h[:, :F]) * h[:, F:]) @ v["w2"][e].t()
        y = y.index_add(0, t, v["probs"][t, j][:, None] * out)
    return y


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_layer_forward_and_gradients(dtype):
    """Relative Frobenius errors: each value passes about eight roundings of the type on its way (the
    product, the adapter's sum, the activation, the second product, the combine and their gradients),
    independent ones, so sqrt(8) half steps; held to four times that."""
    d, experts, request = _inputs(dtype)
    names = ("x", "w1", "w2", "a", "b", "probs")
    dev = {n: d[n].cuda().requires_grad_() for n in names}
    y = _layer(dev, experts.cuda(), request.cuda())
    y.backward(d["dy"].cuda())
    ref = {n: d[n].double().requires_grad_() for n in names}
    want = _plain(ref, experts, request)
    want.backward(d["dy"].double())
    tol = 4 * 8 ** 0.5 * torch.finfo(dtype).eps / 2

    def err(a, b):
        return float((a.detach().cpu().double() - b).norm() / b.norm())
    assert err(y, want.detach()) <= tol
    for n in names:
        assert err(dev[n].grad, ref[n].grad) <= tol, (n, err(dev[n].grad, ref[n].grad), tol)
    used = torch.bincount(experts[experts >= 0].long(), minlength=E)
    assert not dev["w1"].grad[used == 0].any() and not dev["w2"].grad[used == 0].any()


def test_dispatch_feeds_the_quantized_mlp():
    """grouped_mlp on dispatched rows and combined back equals its rows combined by hand."""
    d, experts, _ = _inputs(torch.bfloat16)
    experts = experts.clamp(min=0).cuda()
    plan = g.dispatch_plan(experts, E)
    rec = g.recipe("mxfp8")
    xg = g.dispatch(d["x"].cuda(), plan)
    probs = torch.empty(T * k, device="cuda")
    probs[plan.rows.flatten().long()] = d["probs"].cuda().flatten()
    rows = g.grouped_mlp(xg, probs, d["w1"].cuda(), d["w2"].cuda(), plan.m_splits, "swiglu", rec)
    y = g.combine(rows, plan)
    want = rows.double()[plan.rows.long()].sum(1)
    assert torch.equal(y.double(), want.float().to(torch.bfloat16).double()) or \
        float((y.double() - want).abs().max()) <= float(want.abs().max()) * 2 ** -8


def test_layer_captured_and_replayed():
    """The forward captured (inputs' addresses kept, routing changed in place) replays its eager bits."""
    d, experts, request = _inputs(torch.bfloat16)
    v = {n: d[n].cuda() for n in ("x", "w1", "w2", "a", "b", "probs")}
    ex, rq = experts.cuda(), request.cuda()
    other = ex.roll(1, 0).contiguous()
    first = ex.clone()
    refs = []
    with torch.no_grad():
        for e in (first, other):
            ex.copy_(e)
            refs.append(_layer(v, ex, rq).clone())
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _layer(v, ex, rq)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = _layer(v, ex, rq)
        for r in range(4):
            ex.copy_(first if r % 2 == 0 else other)
            out.fill_(3)
            _layer(v, first, rq)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, refs[r % 2]), r
    del graph


def test_ids_and_probabilities_by_row():
    """A token's adapter and a slot's probability brought to the slot's row with one indexed write each, dropped
    slots to a spare entry: as an explicit loop over the slots."""
    d, experts, request = _inputs(torch.bfloat16)
    experts[7] = torch.tensor([-1, E, 9])
    plan = g.dispatch_plan(experts.cuda(), E)
    ids = torch.full((T * k + 1,), -1, dtype=torch.int32, device="cuda")
    ids[plan.rows.long()] = request.cuda()[:, None].expand(T, k)
    probs = torch.zeros(T * k + 1, device="cuda")
    probs[plan.rows.long()] = d["probs"].cuda()
    want_ids, want_probs = torch.full((T * k,), -1, dtype=torch.int32), torch.zeros(T * k)
    rows = plan.rows.cpu()
    for t in range(T):
        for j in range(k):
            if rows[t, j] >= 0:
                want_ids[rows[t, j]], want_probs[rows[t, j]] = request[t], d["probs"][t, j]
    assert torch.equal(ids[:-1].cpu(), want_ids) and torch.equal(probs[:-1].cpu(), want_probs)
