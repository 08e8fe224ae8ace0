"""dispatch_plan / dispatch / combine against plain sorts, copies and 64-bit sums."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_mxfp8_amd as g
from mm_util import DTYPES, assert_close, floor_step, half_step, ints, randn

pytestmark = pytest.mark.gpu


def _experts(T, k, E, seed, bad=0.0):
    r = np.random.RandomState(seed)
    ids = r.randint(0, E, size=(T, k)).astype(np.int64)
    if bad:
        ids[r.rand(T, k) < bad] = r.choice([-1, E, -2 ** 31, 2 ** 31 - 1])
    return ids.astype(np.int32)


def _order(ids, E):
    """Rows of the slots by a plain stable sort."""
    flat = ids.reshape(-1).astype(np.int64)
    ok = (flat >= 0) & (flat < E)
    slots = np.flatnonzero(ok)
    order = slots[np.argsort(flat[slots], kind="stable")]
    rows = np.full(flat.size, -1, np.int32)
    rows[order] = np.arange(order.size)
    return np.bincount(flat[ok], minlength=E).astype(np.int32), rows.reshape(ids.shape), order


@pytest.mark.parametrize("T,k,E,bad", [(1, 1, 1, 0), (8, 8, 128, 0), (3, 6, 5, 0.3), (64, 1, 64, 0), (1024, 1, 7, 0.1),
                                       (1025, 1, 1024, 0), (777, 3, 1000, 0.2), (8192, 8, 128, 0), (40000, 8, 3, 0.01),
                                       (5, 2, 4, 1.0), (0, 4, 9, 0), (16384, 1, 300, 0.1), (16385, 1, 300, 0.1),
                                       (2049, 6, 1024, 0.01), (1500, 8, 1, 0.5)])
def test_plan_is_the_stable_order(T, k, E, bad):
    print(f"plan T={T} k={k} E={E} bad={bad}", flush=True)
    ids = _experts(T, k, E, 1, bad)
    plan = g.dispatch_plan(torch.from_numpy(ids).cuda(), E)
    splits, rows, _ = _order(ids, E)
    assert np.array_equal(plan.m_splits.cpu().numpy(), splits)
    assert np.array_equal(plan.rows.cpu().numpy(), rows)


def test_plan_order_output():
    """The C ABI's inverse (slot at each row), -1 behind the last used row."""
    import ctypes
    ids = _experts(3000, 2, 50, 2, 0.1)
    n, E = ids.size, 50
    d = torch.from_numpy(ids).cuda()
    m, rows, order = (torch.full((s,), -7, dtype=torch.int32, device="cuda") for s in (E, n, n))
    need = ctypes.c_size_t(0)
    assert g.lib().gmlp_dispatch_plan_ws_bytes(n, E, ctypes.byref(need)) == 0
    ws = torch.empty(max(need.value, 16), dtype=torch.uint8, device="cuda")
    assert g.lib().gmlp_dispatch_plan(g._p(d), n, E, g._p(m), g._p(rows), g._p(order), g._p(ws), ws.numel(), g._stream()) == 0
    splits, want, o = _order(ids, E)
    got = order.cpu().numpy()
    assert np.array_equal(m.cpu().numpy(), splits) and np.array_equal(rows.cpu().numpy(), want.reshape(-1))
    assert np.array_equal(got[:o.size], o) and (got[o.size:] == -1).all()


SHAPES = [(1, 1, 1, 8), (8, 8, 128, 7168), (5, 3, 4, 33), (37, 6, 64, 2048), (130, 11, 9, 264), (64, 2, 3, 1)]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("T,k,E,H", SHAPES)
@pytest.mark.parametrize("bad", [0.0, 0.2])
def test_moves_and_gradients(T, k, E, H, bad, dt):
    print(f"moves T={T} k={k} E={E} H={H} bad={bad} {dt}", flush=True)
    dtype = DTYPES[dt]
    ids = _experts(T, k, E, 3, bad)
    _, rows, order = _order(ids, E)
    plan = g.dispatch_plan(torch.from_numpy(ids).cuda(), E)
    x, v, dy, dxg = randn((T, H), dtype, 1), randn((T * k, H), dtype, 2), randn((T, H), dtype, 3), randn((T * k, H), dtype, 4)
    probs = torch.rand((T, k), generator=torch.Generator().manual_seed(5))
    xg = torch.zeros((T * k, H), dtype=dtype)
    xg[:order.size] = x[torch.from_numpy(order // k)]
    assert torch.equal(g.dispatch_forward(x.cuda(), plan).cpu(), xg)
    keep = torch.full((T * k, H), 9.0, dtype=dtype, device="cuda")
    g.dispatch_forward(x.cuda(), plan, out=keep)
    assert torch.equal(keep[:order.size].cpu(), xg[:order.size]) and bool((keep[order.size:] == 9).all())
    r = torch.from_numpy(rows.astype(np.int64))
    live = (r >= 0).double()
    pv = v.double()[r.clamp(min=0)] * live[:, :, None]
    pg = dxg.double()[r.clamp(min=0)] * live[:, :, None]
    p64 = probs.double()
    assert_close(g.combine_forward(v.cuda(), plan, probs.cuda()), (pv * p64[:, :, None]).sum(1),
                 (pv * p64[:, :, None]).abs().sum(1), k, "combine")
    assert_close(g.combine_forward(v.cuda(), plan), pv.sum(1), pv.abs().sum(1), k, "combine without probs")
    assert_close(g.dispatch_backward(dxg.cuda(), plan), pg.sum(1), pg.abs().sum(1), k, "dispatch gradient")
    dv, dp = g.combine_backward(dy.cuda(), v.cuda(), plan, probs.cuda())
    want = torch.zeros((T * k, H), dtype=torch.float64)
    t = torch.from_numpy(order // k)
    want[:order.size] = dy.double()[t] * p64.reshape(-1)[torch.from_numpy(order)][:, None]
    assert_close(dv, want, want.abs(), 1, "combine gradient")
    prod = pv * dy.double()[:, None, :]
    assert_close(dp, prod.sum(2), prod.abs().sum(2), H, "probs gradient")
    assert not dp.cpu()[r < 0].any()
    dv1, none = g.combine_backward(dy.cuda(), v.cuda(), plan)
    assert none is None and torch.equal(dv1[:order.size].cpu(), dy[t]) and not dv1[order.size:].any()


def test_strided_rows_and_transposed_inputs():
    T, k, E, H = 20, 4, 6, 40
    ids = _experts(T, k, E, 3)
    plan = g.dispatch_plan(torch.from_numpy(ids).cuda(), E)
    x, v = randn((T, H), torch.bfloat16, 1).cuda(), randn((T * k, H), torch.bfloat16, 2).cuda()
    for pad, off in ((8, 0), (8, 8), (3, 1)):
        def view(t):
            big = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
            big[:, off:off + t.shape[1]] = t
            return big[:, off:off + t.shape[1]]
        assert torch.equal(g.dispatch_forward(view(x), plan), g.dispatch_forward(x, plan))
        o = view(torch.zeros_like(x))
        g.combine_forward(view(v), plan, out=o)
        assert torch.equal(o, g.combine_forward(v, plan))
    assert torch.equal(g.dispatch_forward(x.t().contiguous().t(), plan), g.dispatch_forward(x, plan))


def test_nan_in_unused_rows_reaches_nothing():
    ids = np.array([[0, -1], [1, 0], [7, 2]], np.int32)
    plan = g.dispatch_plan(torch.from_numpy(ids).cuda(), 3)
    v = torch.ones((6, 16), dtype=torch.bfloat16, device="cuda")
    v[4:] = float("nan")
    probs = torch.tensor([[1, float("nan")], [1, 1], [float("inf"), 1]], device="cuda")
    y = g.combine_forward(v, plan, probs)
    assert torch.equal(y.cpu().float(), torch.tensor([1.0, 2.0, 1.0])[:, None].expand(3, 16))


@pytest.mark.parametrize("H", [3, 9, 13, 17, 250])
def test_odd_rows_count_every_element_once(H):
    """Rows that are not whole 16-byte chunks, an infinity in the overlap of the last two loads: it
    reaches its own column and the one product that holds it, exactly."""
    T, k, E = 6, 2, 3
    plan = g.dispatch_plan(torch.from_numpy(_experts(T, k, E, 9)).cuda(), E)
    v = ints((T * k, H), torch.bfloat16, 1, 1, 3).cuda()
    dy = ints((T, H), torch.bfloat16, 2, 1, 3).cuda()
    dv, dp = g.combine_backward(dy, v, plan, torch.ones((T, k), device="cuda"))
    r = plan.rows.long()
    assert torch.equal(dp.double(), (dy.double()[:, None, :] * v.double()[r]).sum(2))
    dyi = dy.clone()
    dyi[4, max(H - 9, 0)] = float("inf")
    dv2, dp2 = g.combine_backward(dyi, v, plan, torch.ones((T, k), device="cuda"))
    rows = torch.arange(T) != 4
    assert torch.equal(dp2[rows.cuda()], dp[rows.cuda()]) and bool((dp2[4] == float("inf")).all())
    assert torch.equal(dv2[r[4]], dyi[4].expand(k, H))


def test_autograd_against_formula_and_differences():
    T, k, E, H = 9, 3, 4, 24
    ids = _experts(T, k, E, 6, 0.1)
    plan = g.dispatch_plan(torch.from_numpy(ids).cuda(), E)
    x, dy = ints((T, H), torch.bfloat16, 1).cuda(), ints((T, H), torch.bfloat16, 2, -1, 1).cuda()
    probs = ints((T, k), torch.float32, 3, 0, 3).cuda()

    def f(xx, pp):
        return g.combine(g.dispatch(xx, plan), plan, pp)
    xr, pr = x.clone().requires_grad_(), probs.clone().requires_grad_()
    f(xr, pr).backward(dy)
    live = (plan.rows >= 0).double()
    assert torch.equal(xr.grad.double(), dy.double() * (probs.double() * live).sum(1, keepdim=True))
    assert torch.equal(pr.grad.double(), live * (dy.double() * x.double()).sum(1, keepdim=True))

    def loss(xx, pp):
        return float((f(xx, pp).double() * dy.double()).sum())
    for seed in range(3):
        ex, ep = ints((T, H), torch.bfloat16, 10 + seed, 0, 1).cuda(), ints((T, k), torch.float32, 20 + seed, 0, 1).cuda()
        assert loss(x + ex, probs) - loss(x - ex, probs) == 2 * float((xr.grad.double() * ex.double()).sum())
        assert loss(x, probs + ep) - loss(x, probs - ep) == 2 * float((pr.grad.double() * ep.double()).sum())


def test_graph_replays_and_side_stream():
    T, k, E, H = 300, 8, 64, 512
    e1, e2 = (torch.from_numpy(_experts(T, k, E, s)).cuda() for s in (7, 8))
    experts = e1.clone()
    x = randn((T, H), torch.bfloat16, 1).cuda()
    probs = torch.rand((T, k), device="cuda")

    def step():
        plan = g.dispatch_plan(experts, E)
        xg = g.dispatch_forward(x, plan)
        y = g.combine_forward(xg, plan, probs)
        dv, dp = g.combine_backward(x, xg, plan, probs)
        return plan.m_splits, plan.rows, xg, y, dv, dp, g.dispatch_backward(dv, plan)
    refs = []
    for e in (e1, e2):
        experts.copy_(e)
        refs.append([t.clone() for t in step()])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(refs[1], other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(4):
        experts.copy_(e1 if r % 2 == 0 else e2)
        for t in out:
            t.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(refs[r % 2], out)), r
    del graph
