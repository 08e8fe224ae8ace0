"""residual_norm / rms_norm against the formulas in 64 bits."""
import math

import pytest
import torch

import nvfp4_block_scaled_mxfp8_amd as g
from block_util import assert_norm, norm_forms
from mm_util import DTYPES, randn

pytestmark = pytest.mark.gpu
GATES = ["none", "channel", "token", "full"]


def _make(T, H, dt, gate, pre, post, wide, seed=1, std=1.0):
    dtype = DTYPES[dt]
    pt = torch.float32 if wide else dtype
    r = lambda shape, i, t=dtype, s=1.0: randn(shape, t, seed * 100 + i, s)
    shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[gate]
    return dict(x=r((T, H), 1, s=std), branch=r((T, H), 2, s=0.5 * std), weight=1 + r((H,), 3, pt, 0.2) if pre else None,
                branch_weight=1 + r((H,), 4, pt, 0.2) if post else None, gate=r(shape, 5, pt) if shape else None)


def _cuda(t):
    return t.cuda() if t is not None else None


def _run(c, scale, eps, dy, dh, dev=None):
    dev = dev or {k: _cuda(v) for k, v in c.items()}
    kw = {k: dev[k] for k in ("weight", "branch_weight", "gate")}
    y, h, stats = g.residual_norm_forward(dev["x"], dev["branch"], scale=scale, eps=eps, **kw)
    got = {"y": y, "h": h}
    got.update(g.residual_norm_backward(_cuda(dy), _cuda(dh), dev["x"], dev["branch"], stats, scale=scale, eps=eps, **kw))
    return got


def _check(c, scale=1.0, eps=1e-6, seed=9, dev=None, dtype=None, dy=True):
    T, H = c["x"].shape
    dtype = c["x"].dtype
    dy = randn((T, H), dtype, seed) if dy else None
    dh = randn((T, H), dtype, seed + 1) if c["weight"] is not None else None
    got = _run(c, scale, eps, dy, dh, dev)
    want = norm_forms(c["x"], c["branch"], c["weight"], c["branch_weight"], c["gate"], scale, eps, dy, dh)
    # roundings on the way of each: y: scale x gate x weight x root x branch (the root two itself) and the sum;
    # h three more; the row sums of the backward H each, and two of them behind each other for dbranch; column sums T
    terms = {"y": 8, "h": 16, "dx": H + 32, "dweight": T + 32, "dgate": 2 * H + T + 64, "dbranch": 4 * H + 64,
             "dbranch_weight": T + H + 64}
    for name, form in want.items():
        assert got[name] is not None, name
        assert_norm(got[name], form, terms[name], name)
    for name, t in got.items():
        assert (t is None) == (name not in want), name
    return got


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (2, 8), (5, 9), (4, 512), (6, 513), (3, 1024), (5, 1025), (2, 2048), (2, 2049), (9, 2056),
                                 (3, 7168), (2, 8192), (2, 8200), (1, 16384), (1, 16392), (2, 32767), (1, 32768)])
def test_all_parts(T, H, gate, dt):
    print(f"norm T={T} H={H} gate={gate} {dt}", flush=True)
    _check(_make(T, H, dt, gate, True, True, False), scale=0.5)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("pre,post", [(True, False), (False, True), (False, False), (True, True)])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_every_combination(pre, post, gate, wide, dt):
    print(f"norm combination pre={pre} post={post} gate={gate} wide={wide} {dt}", flush=True)
    _check(_make(37, 264, dt, gate, pre, post, wide), scale=-1.25, eps=1e-3)
    _check(_make(5, 2304, dt, gate, pre, post, wide), scale=1.0)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("H", [3, 5000, 8001, 12000, 20001])
def test_fp32_parameters_of_long_rows(H, gate, dt):
    """Every kernel of the backward with fp32 parameters and gates, whole and ragged rows."""
    print(f"norm long H={H} gate={gate} {dt}", flush=True)
    _check(_make(3, H, dt, gate, True, True, True), scale=0.5)


@pytest.mark.parametrize("T,H", [(1, 64), (700, 200), (1025, 72), (2500, 1001)])
def test_column_sums_of_many_rows(T, H):
    print(f"norm columns T={T} H={H}", flush=True)
    _check(_make(T, H, "bf16", "channel", True, True, True), scale=0.25)


def test_more_rows_than_workgroups_of_long_rows():
    _check(_make(1100, 2200, "fp16", "channel", True, True, False), scale=0.5)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("T,H", [(4, 40), (3, 7168), (2049, 16)])
def test_rms_norm(T, H, dt):
    x, dh = randn((T, H), DTYPES[dt], 1), randn((T, H), DTYPES[dt], 2)
    w = 1 + randn((H,), DTYPES[dt], 3, 0.2)
    h, stats = g.rms_norm_forward(x.cuda(), w.cuda(), 1e-5)
    dx, dw = g.rms_norm_backward(dh.cuda(), x.cuda(), w.cuda(), stats, 1e-5)
    want = norm_forms(x, None, w, None, None, 1.0, 1e-5, None, dh)
    assert_norm(h, want["h"], 16, "h")
    assert_norm(dx, want["dx"], H + 32, "dx")
    assert_norm(dw, want["dweight"], T + 32, "dweight")
    xr, wr = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    g.rms_norm(xr, wr, 1e-5).backward(dh.cuda())
    assert torch.equal(xr.grad, dx) and torch.equal(wr.grad, dw)


def test_no_rows():
    c = _make(0, 24, "bf16", "channel", True, True, True)
    dev = {k: _cuda(v) for k, v in c.items()}
    e = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    kw = {k: dev[k] for k in ("weight", "branch_weight", "gate")}
    y, h, stats = g.residual_norm_forward(e, e, **kw)
    r = g.residual_norm_backward(e, e, e, e, stats, **kw)
    assert y.shape == h.shape == r["dx"].shape == r["dbranch"].shape == (0, 24)
    for k in ("dweight", "dbranch_weight", "dgate"):
        assert torch.equal(r[k], torch.zeros(24, device="cuda")), k


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("gate", ["token", "full"])
def test_strides(gate, dt):
    c = _make(11, 100, dt, gate, True, True, False)
    ref = _run(c, 0.5, 1e-6, c["branch"], c["x"])
    for pad, off in ((4, 0), (3, 1), (12, 8)):
        def view(t):
            if t is None or t.dim() == 1:
                return _cuda(t)
            big = torch.full((t.shape[0], t.shape[1] + pad), math.nan, dtype=t.dtype, device="cuda")
            big[:, off:off + t.shape[1]] = t.cuda()
            return big[:, off:off + t.shape[1]]
        dev = {k: view(v) for k, v in c.items()}
        got = _run(c, 0.5, 1e-6, view(c["branch"]), view(c["x"]), dev)
        for k in ref:
            assert torch.equal(ref[k], got[k]), (k, pad, off)
        out = view(torch.zeros_like(c["x"]))
        kw = {k: dev[k] for k in ("weight", "branch_weight", "gate")}
        y, h, _ = g.residual_norm_forward(dev["x"], dev["branch"], scale=0.5, out=out, **kw)
        assert y is out and torch.equal(out, ref["y"]) and torch.equal(h, ref["h"])
    t = {k: _cuda(v.t().contiguous()).t() if v is not None and v.dim() == 2 else _cuda(v) for k, v in c.items()}
    got = _run(c, 0.5, 1e-6, c["branch"], c["x"], t)
    assert all(torch.equal(ref[k], got[k]) for k in ref)
    if gate == "token":                                          # one value for all tokens
        one = c["gate"][:1]
        dev = {k: _cuda(v) for k, v in c.items()}
        dev["gate"] = one.cuda().expand(11, 1)
        c["gate"] = one.expand(11, 1)
        _check(c, 0.5, dev=dev)


def test_in_place():
    for into in ("x", "branch"):
        c = {k: _cuda(v) for k, v in _make(9, 2304, "bf16", "token", True, True, False).items()}
        kw = {k: c[k] for k in ("weight", "branch_weight", "gate")}
        y, h, _ = g.residual_norm_forward(c["x"], c["branch"], scale=0.5, **kw)
        version = c[into]._version
        y2, h2, _ = g.residual_norm_forward(c["x"], c["branch"], scale=0.5, out=c[into], **kw)
        assert y2 is c[into] and torch.equal(y, y2) and torch.equal(h, h2) and c[into]._version == version + 1


def test_outputs_over_what_is_read_are_refused():
    big = torch.zeros((12, 64), dtype=torch.bfloat16, device="cuda")
    x, other, w = big[:8], torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for branch, out in ((other, big[1:9]), (big[1:9], x), (other, big[4:])):
        with pytest.raises(ValueError, match="overlaps"):
            g.residual_norm_forward(x, branch, w, out=out)
    wide = torch.zeros((8, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        g.residual_norm_forward(wide[:, :64], other, w, gate=wide[:, 64:], out=wide[:, 60:124])
    with pytest.raises(ValueError, match="overlaps"):
        g.residual_norm_forward(other, x, w, gate=wide[0, :64], out=wide[:, :64])
    y, _, _ = g.residual_norm_forward(wide[:, :64], other, w, out=wide[:, 64:])      # beside each other
    assert not y.any()
    with pytest.raises(ValueError, match="out"):
        g.residual_norm_forward(x, None, w, out=other)
    with pytest.raises(ValueError, match="stats"):
        g.residual_norm_backward(other, other, x, other, torch.zeros((2, 7), device="cuda"), w)
    with pytest.raises(ValueError, match="dh"):
        g.residual_norm_backward(other, None, x, other, torch.zeros((2, 8), device="cuda"), w)


@pytest.mark.parametrize("std", [1e-20, 1e-12, 1e12, 1e18, 1e36])
def test_small_and_large_rows(std):
    """Squares that leave fp32 at both ends, without eps: the norms are still the formula's."""
    c = _make(6, 300, "bf16", "none", True, True, True, std=std)
    # the branch joins as a vector of length 1; against rows this far from it a scale keeps the sum a sum
    x, b, w, bw = (_cuda(c[k]) for k in ("x", "branch", "weight", "branch_weight"))
    y, h, stats = g.residual_norm_forward(x, b, w, bw, scale=std, eps=0.0)
    want = norm_forms(c["x"], c["branch"], c["weight"], c["branch_weight"], None, float(torch.tensor(std)), 0.0)
    assert_norm(y, want["y"], 8, "y")
    assert_norm(h, want["h"], 16, "h")


def test_a_row_that_is_not_finite_stays_alone():
    for bad in (math.nan, math.inf):
        for H in (72, 2304):
            c = _make(8, H, "bf16", "full", True, True, False)
            ref = _run(c, 0.5, 1e-6, c["branch"], c["x"])
            c["x"][3, 5] = bad
            c["branch"][6, 2] = bad
            got = _run(c, 0.5, 1e-6, c["branch"], c["x"])
            rows = torch.tensor([0, 1, 2, 4, 5, 7])
            for k in ("y", "h", "dx", "dbranch", "dgate"):
                assert torch.equal(ref[k][rows], got[k][rows]), (k, bad, H)
            assert torch.isnan(got["dx"][6].float()).any()


@pytest.mark.parametrize("H", [72, 2304, 9000])
@pytest.mark.parametrize("gate", ["none", "channel", "full"])
def test_infinities_reach_no_gradient_that_has_not_their_formula(gate, H):
    """Without norms dx is dy and dbranch = scale gate dy, whatever x and branch hold; with one of the norms the
    other side's rows stay as finite as their formula."""
    c = _make(4, H, "bf16", gate, False, False, False)
    ref = _run(c, 0.5, 1e-6, c["branch"], None)
    dy = c["branch"].clone()
    c["x"][1, 3] = math.inf
    c["branch"][2, 5] = -math.inf
    c["branch"][0, 7] = math.nan
    got = _run(c, 0.5, 1e-6, dy, None)
    assert torch.equal(got["dx"].cpu(), dy) and torch.equal(got["dx"], ref["dx"]) and torch.equal(got["dbranch"], ref["dbranch"])
    c = _make(4, H, "bf16", gate, False, True, False)
    ref = _run(c, 0.5, 1e-6, dy, None)
    c["x"][1, 3] = math.inf
    got = _run(c, 0.5, 1e-6, dy, None)
    for n in ("dx", "dbranch", "dbranch_weight", "dgate"):
        assert got[n] is None or torch.equal(got[n], ref[n]), n


def test_gradients_against_differences():
    """<grad, v> against central differences of the loss, taken in 64 bits on the CPU."""
    for gate in GATES:
        c = _make(7, 48, "bf16", gate, True, True, True, seed=3)
        dy, dh = randn((7, 48), torch.bfloat16, 31), randn((7, 48), torch.bfloat16, 32)
        got = _run(c, 0.5, 1e-6, dy, dh)

        def loss(d):
            f = norm_forms(d["x"], d["branch"], d["weight"], d["branch_weight"], d["gate"], 0.5, 1e-6)
            return float((f["y"][0] * dy.double()).sum() + (f["h"][0] * dh.double()).sum())
        for name in ("x", "branch", "weight", "branch_weight", "gate"):
            if c[name] is None:
                continue
            v = torch.randn(c[name].shape, generator=torch.Generator().manual_seed(33)).double()
            h = 2.0 ** -12
            slope = (loss({**c, name: c[name].double() + h * v}) - loss({**c, name: c[name].double() - h * v})) / (2 * h)
            grad = got["d" + name].cpu().double()
            # each element of the gradient is rounded once (2^-8 for 16 bits); differences leave h^2 of third derivatives
            assert abs(slope - float((grad * v).sum())) <= 2.0 ** -8 * float((grad * v).abs().sum()) + 1e-4, (gate, name)


def test_autograd():
    c = _make(33, 136, "bf16", "channel", True, True, True)
    dy, dh = randn((33, 136), torch.bfloat16, 41).cuda(), randn((33, 136), torch.bfloat16, 42).cuda()
    names = ("x", "branch", "weight", "branch_weight", "gate")

    def leaves():
        return [c[n].cuda().requires_grad_() for n in names]
    ref = _run(c, 0.5, 1e-6, dy, dh)
    l = leaves()
    y, h = g.residual_norm(*l, scale=0.5)
    torch.autograd.backward([y, h], [dy, dh])
    for n, t in zip(names, l):
        assert torch.equal(t.grad, ref["d" + n]), n
    # only one of the two outputs used
    l = leaves()
    y, h = g.residual_norm(*l, scale=0.5)
    y.backward(dy)
    r = g.residual_norm_backward(dy, None, *[c[n].cuda() for n in ("x", "branch")], _stats(c), branch_weight=c["branch_weight"].cuda(),
                                 gate=c["gate"].cuda(), scale=0.5)
    assert l[2].grad is None and torch.equal(l[0].grad, r["dx"]) and torch.equal(l[1].grad, r["dbranch"])
    l = leaves()
    y, h = g.residual_norm(*l, scale=0.5)
    h.backward(dh)
    r = _run(c, 0.5, 1e-6, None, dh)
    for n, t in zip(names, l):
        assert torch.equal(t.grad, r["d" + n]), n
    # frozen inputs get none
    l = leaves()
    for i in (0, 2, 4):
        l[i].requires_grad_(False)
    torch.autograd.backward(list(g.residual_norm(*l, scale=0.5)), [dy, dh])
    assert l[0].grad is None and l[2].grad is None and l[4].grad is None
    assert torch.equal(l[1].grad, ref["dbranch"]) and torch.equal(l[3].grad, ref["dbranch_weight"])
    # an input written in place before the backward is noticed
    l = leaves()
    x = l[0] * 1
    y, h = g.residual_norm(x, *l[1:], scale=0.5)
    x.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        h.backward(dh)


def _stats(c):
    return g.residual_norm_forward(*[c[n].cuda() for n in ("x", "branch", "weight", "branch_weight", "gate")], scale=0.5)[2]


def test_graph_replays_and_side_stream():
    a, b = (_make(130, 2304, "bf16", "channel", True, True, True, seed=s) for s in (5, 6))
    live = {k: v.cuda() for k, v in a.items()}

    def step():
        return [t for t in _run(a, 0.5, 1e-6, live["branch"], live["x"], live).values()]
    refs = []
    for c in (a, b):
        for k in live:
            live[k].copy_(c[k])
        refs.append([t.clone() for t in step()])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(refs[1], other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(4):
        for k in live:
            live[k].copy_((a if r % 2 == 0 else b)[k])
        for t in out:
            t.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(refs[r % 2], out)), r
    del graph


def test_more_rows_than_one_grid_row_holds():
    """Past 2^24 workgroups the grid is folded (rows of one element: h = sign(y) |w| without eps)."""
    T = (1 << 26) + 11
    x = torch.ones((T, 1), dtype=torch.bfloat16, device="cuda")
    x[1::2] = -3.0
    w = torch.full((1,), 2.0, dtype=torch.bfloat16, device="cuda")
    h, stats = g.rms_norm_forward(x, w, 0.0)
    assert torch.equal(h, 2 * torch.sign(x))
    dx, dw = g.rms_norm_backward(torch.ones_like(x), x, w, stats, 0.0)
    # the norm of one element is its sign: no slope but roundings of (1 - yh^2) / |x|, two steps of fp32 each
    assert float(dx.float().abs().max()) <= 2 * 2.0 ** -21 and float(dw.float().abs()) <= T


TINY = 2.0 ** -133                                # the smallest bf16 number


@pytest.mark.parametrize("H", [7, 300, 2304, 5000, 9000, 20001])
def test_rows_of_subnormals_without_eps(H):
    """Without eps a norm does not depend on its row's size, down to rows of the smallest numbers, whose factor has no
    place in fp32: values and gradients, beside ordinary rows, rows at the border and one of zeros (0 / 0)."""
    T = 9
    k = torch.randint(-9, 10, (T, H), generator=torch.Generator().manual_seed(1)).float()
    k[:, 0] = 5.0
    # sizes 2^-133, around 2^-128 and 2^-126, ordinary; the largest that one element can bring among zeros
    x = (k * torch.tensor([TINY, TINY, 2.0 ** -130, 2.0 ** -129, 2.0 ** -127, 2.0 ** -125, 1.0, 2.0 ** 100, 1.0])[:, None]).to(torch.bfloat16)
    x[1, 1:] = 0
    x[8] = 0
    x[8, 2] = 2.0 ** -122
    w = 1 + randn((H,), torch.float32, 2, 0.2)
    # the gradient for x of a row of size s is of size dh / s
    dh = (randn((T, H), torch.float32, 3) * 2.0 ** -20).to(torch.bfloat16)
    zero = torch.cat([x, torch.zeros((1, H), dtype=torch.bfloat16)])
    h, stats = g.rms_norm_forward(x.cuda(), w.cuda(), 0.0)
    dx, dw = g.rms_norm_backward(dh.cuda(), x.cuda(), w.cuda(), stats, 0.0)
    want = norm_forms(x, None, w, None, None, 1.0, 0.0, None, dh)
    assert_norm(h, want["h"], 16, "h")
    assert_norm(dx, want["dx"], H + 32, "dx")
    assert_norm(dw, want["dweight"], T + 32, "dweight")
    hz, _ = g.rms_norm_forward(zero.cuda(), w.cuda(), 0.0)
    assert torch.equal(hz[:T], h) and bool(torch.isnan(hz[T]).all())
    # the branch's own norm, around ordinary rows; the sum of two such rows
    c = dict(x=randn((T, H), torch.bfloat16, 4), branch=x, weight=w, branch_weight=1 + randn((H,), torch.float32, 5, 0.2),
             gate=1 + randn((T, H), torch.bfloat16, 6, 0.2))
    for gate, kind in ((None, "none"), (c["gate"], "full"), (c["gate"][:, :1].contiguous(), "token"), (c["gate"][0].contiguous(), "channel")):
        print(f"norm subnormal H={H} gate={kind}", flush=True)
        c["gate"] = gate
        dy = (randn((T, H), torch.float32, 7) * 2.0 ** -20).to(torch.bfloat16)
        got = _run(c, 0.5, 0.0, dy, dh)
        want = norm_forms(c["x"], x, w, c["branch_weight"], gate, 0.5, 0.0, dy, dh)
        terms = {"y": 8, "h": 16, "dx": H + 32, "dweight": T + 32, "dgate": 2 * H + T + 64, "dbranch": 4 * H + 64, "dbranch_weight": T + H + 64}
        for name, form in want.items():
            assert_norm(got[name], form, terms[name], f"{name} {kind}")
    c = dict(x=x, branch=(x.float().roll(1, 1) * 4).to(torch.bfloat16), weight=w, branch_weight=None, gate=None)
    got = _run(c, 1.0, 0.0, None, dh)
    for name, form in norm_forms(x, c["branch"], w, None, None, 1.0, 0.0, None, dh).items():
        assert_norm(got[name], form, {"y": 8, "h": 16, "dx": H + 32, "dweight": T + 32, "dbranch": 4 * H + 64}[name], f"{name} sum")


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("H", [3, 264, 5000, 12000, 20001])
def test_every_kernel_without_eps(H, gate, dt):
    """Ordinary rows, parameters of both types."""
    print(f"norm without eps H={H} gate={gate} {dt}", flush=True)
    for wide in (False, True):
        _check(_make(4, H, dt, gate, True, True, wide), scale=0.5, eps=0.0)
