"""route / route_forward / route_backward against a plain sort and sums in 64 bits."""
import math

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_mxfp8_amd as g
from block_util import plain_choice, plain_dlogits, plain_probs, route_tol

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _logits(T, E, dtype, seed, std=1.5, masked=0.0):
    gen = torch.Generator().manual_seed(seed)
    x = (std * torch.randn((T, E), generator=gen)).to(dtype)
    if masked:
        x[torch.rand((T, E), generator=gen) < masked] = -math.inf
    return x


def _bias(E, seed, std=0.2):
    return std * torch.randn(E, generator=torch.Generator().manual_seed(seed))


def _same(a, b):
    return (math.isnan(a) and math.isnan(b)) or a == b


def _check(logits, k, score, bias=None, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0, dprobs=None,
           dev_logits=None):
    """The choice exactly, probabilities and the gradient within their bounds."""
    dl = dev_logits if dev_logits is not None else logits.cuda()
    how = dict(renormalize=renormalize, scale=scale)
    experts, probs = g.route_forward(dl, k, score, bias=bias.cuda() if bias is not None else None, groups=groups,
                                     top_groups=top_groups, group_best=group_best, **how)
    T, E = logits.shape
    rows = logits.double().tolist()
    b64 = bias.double().tolist() if bias is not None else None
    ex, pr = experts.cpu().tolist(), probs.cpu().double().tolist()
    dlog = g.route_backward(dprobs.cuda(), dl, experts, score, **how).cpu().double().tolist() if dprobs is not None else None
    out_type = torch.finfo(logits.dtype)
    scale32 = float(np.float32(scale))
    for t in range(T):
        want = plain_choice(rows[t], k, score, b64, groups, top_groups, group_best)
        assert ex[t] == want, (t, ex[t], want)
        finite = [v for v in rows[t] if math.isfinite(v)]
        spread = min(max(finite, default=0.0) - min(finite, default=0.0), 104.0)
        rel = route_tol(E, spread)
        pw = plain_probs(rows[t], want, score, renormalize, scale32)
        for j in range(k):
            assert _same(pr[t][j], pw[j]) or abs(pr[t][j] - pw[j]) <= rel * abs(pw[j]) + 2.0 ** -126 * max(1, abs(scale)), (t, j, pr[t][j], pw[j])
        if dlog is None:
            continue
        dw, mag = plain_dlogits(rows[t], want, dprobs[t].double().tolist(), score, renormalize, scale32)
        for e in range(E):
            tol = out_type.eps / 2 * abs(dw[e]) * (1 + 2.0 ** -8) + (2 * rel + (k + 8) * 2.0 ** -23) * mag[e] + out_type.tiny * out_type.eps + 2.0 ** -120
            assert _same(dlog[t][e], dw[e]) or abs(dlog[t][e] - dw[e]) <= tol, (t, e, dlog[t][e], dw[e], tol)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (17, 33, 5), (40, 64, 8), (33, 65, 6), (31, 128, 8), (18, 130, 12), (9, 256, 8),
                                   (7, 257, 16), (5, 512, 17), (5, 513, 8), (3, 1024, 64), (6, 1000, 13)])
def test_choice_weights_and_gradient(T, E, k, score, renorm, dt):
    print(f"route T={T} E={E} k={k} {score} renorm={renorm} {dt}", flush=True)
    logits = _logits(T, E, TYPES[dt], 1)
    dprobs = torch.randn((T, k), generator=torch.Generator().manual_seed(2))
    _check(logits, k, score, None, renormalize=renorm, scale=1.0 if renorm else 2.5, dprobs=dprobs)
    _check(logits, k, score, _bias(E, 3), renormalize=renorm, scale=0.5, dprobs=dprobs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,best,k", [(32, 4, 2, 1, 4), (256, 8, 4, 2, 8), (96, 8, 3, 2, 7), (64, 64, 9, 2, 9), (60, 4, 1, 2, 15),
                                                 (512, 8, 2, 2, 20), (1024, 64, 5, 1, 64), (40, 2, 2, 2, 3), (12, 3, 2, 1, 8)])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_groups(E, groups, top, best, k, score, with_bias, dt):
    print(f"route groups E={E} groups={groups} top={top} best={best} k={k} {score} bias={with_bias} {dt}", flush=True)
    for masked in (0.0, 0.6):
        _check(_logits(21, E, TYPES[dt], 4, masked=masked), k, score, _bias(E, 5) if with_bias else None, groups, top, best)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(16, 8), (128, 12), (300, 20)])
def test_ties_go_to_the_lowest_index(E, k, score, dt):
    """Few different values: whole runs of equal logits, across every border of lanes and loads; signed zeros are equal."""
    gen = torch.Generator().manual_seed(6)
    logits = torch.randint(-1, 2, (13, E), generator=gen).to(TYPES[dt])
    logits[3] = 0.0
    logits[4] = 1.0
    logits[5, ::2] = -0.0
    logits[5, 1::2] = 0.0
    _check(logits, k, score)
    _check(logits, k, score, torch.zeros(E))
    _check(logits, k, score, torch.randint(-1, 2, (E,), generator=gen).float())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_ties_are_decided_in_64_bits(score):
    """Logits and biases so near each other that the sums are equal in 32 bits and in order only in 64."""
    E, k, T = 64, 9, 16
    r = np.random.RandomState(7)
    logits = np.full((T, E), 0.25, np.float32)
    for t in range(T):
        steps = r.randint(0, 12, E)
        for e in range(E):
            for _ in range(steps[e]):
                logits[t, e] = np.nextafter(logits[t, e], np.float32(9), dtype=np.float32)
    bias = np.full(E, 0.125, np.float32)
    for e in range(E):
        for _ in range(r.randint(0, 3)):
            bias[e] = np.nextafter(bias[e], np.float32(9), dtype=np.float32)
    logits, bias = torch.from_numpy(logits), torch.from_numpy(bias)
    _check(logits, k, score, bias)
    _check(logits, k, score, bias, groups=8, top_groups=3, group_best=2)
    _check(logits, k, score, None, groups=8, top_groups=3, group_best=2)
    _check(logits, k, score, -torch.sigmoid(logits[0]).contiguous())          # sums around zero
    _check(logits * 1e-3, k, score, 1000.0 * bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [24, 200, 700])
def test_masked_experts_and_empty_rows(E, renorm, score):
    logits = _logits(12, E, torch.float32, 8)
    logits[0] = -math.inf                                  # nothing
    logits[1, 1:] = -math.inf                              # one expert
    logits[2, :-3] = -math.inf                             # fewer than k
    logits[3] = torch.finfo(torch.float32).min             # the lowest number is no mask
    logits[4, ::2] = torch.finfo(torch.float32).min
    logits[11] = -math.inf
    dprobs = torch.randn((12, 6), generator=torch.Generator().manual_seed(9))
    dprobs[0] = math.nan                                   # of slots that found none: nothing reaches a gradient
    dprobs[2, 3:] = math.inf
    for bias in (None, _bias(E, 10)):
        _check(logits, 6, score, bias, renormalize=renorm, dprobs=dprobs)
        _check(logits, 6, score, bias, groups=4, top_groups=2, group_best=2, renormalize=renorm, dprobs=dprobs)
    masked = _bias(E, 11)
    masked[::3] = -math.inf
    _check(logits, 6, score, masked, renormalize=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_infinities_and_nan_stay_in_their_rows(renorm, score):
    logits = _logits(6, 40, torch.float32, 12)
    clean = logits.clone()
    logits[1, 7] = math.nan
    logits[2, 9] = math.inf
    logits[4, 5] = logits[4, 20] = math.nan
    for bias in (None, _bias(40, 13)):
        _check(logits, 5, score, bias, renormalize=renorm)
        ref = g.route_forward(clean.cuda(), 5, score, bias=bias.cuda() if bias is not None else None, renormalize=renorm)
        got = g.route_forward(logits.cuda(), 5, score, bias=bias.cuda() if bias is not None else None, renormalize=renorm)
        for r in (0, 3, 5):
            assert torch.equal(ref[0][r], got[0][r]) and torch.equal(ref[1][r], got[1][r])


@pytest.mark.parametrize("renorm", [True, False])
def test_large_logits_keep_their_ratios(renorm):
    """Scores that leave fp32, at both ends: the renormalized weights are still the formula's."""
    base = torch.linspace(-3, 3, 20)
    logits = torch.stack([base - 200, base + 200, base * 30, base - 95, base * 1e4, base * 1e30])
    dprobs = torch.randn((6, 5), generator=torch.Generator().manual_seed(1))
    for score in ("softmax", "sigmoid"):
        _check(logits, 5, score, None, renormalize=renorm, dprobs=dprobs if renorm else None)


def test_an_expert_named_twice_has_the_sum():
    logits = _logits(3, 20, torch.float32, 14)
    experts = torch.tensor([[1, 1, 5], [2, 7, 2], [19, 20, -1]], dtype=torch.int32)
    dprobs = torch.randn((3, 3), generator=torch.Generator().manual_seed(15))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = g.route_backward(dprobs.cuda(), logits.cuda(), experts.cuda(), score, renorm).cpu().double()
            for t in range(3):
                row = logits[t].double().tolist()
                want, mag = plain_dlogits(row, experts[t].tolist(), dprobs[t].double().tolist(), score, renorm, 1.0)
                tol = (2 * route_tol(20, max(row) - min(row)) + 2.0 ** -20) * torch.tensor(mag, dtype=torch.float64)
                assert bool(((got[t] - torch.tensor(want, dtype=torch.float64)).abs() <= tol).all()), (score, renorm, t)


@pytest.mark.parametrize("dt", list(TYPES))
def test_strided_and_transposed_logits(dt):
    logits = _logits(19, 50, TYPES[dt], 16)
    dprobs = torch.randn((19, 4), generator=torch.Generator().manual_seed(17))
    for pad, off in ((6, 0), (3, 1), (14, 8)):
        big = torch.full((19, 50 + pad), math.nan, dtype=TYPES[dt], device="cuda")
        big[:, off:off + 50] = logits.cuda()
        _check(logits, 4, "softmax", _bias(50, 18), renormalize=False, dprobs=dprobs, dev_logits=big[:, off:off + 50])
    _check(logits, 4, "sigmoid", dprobs=dprobs, dev_logits=logits.t().contiguous().cuda().t())
    _check(logits[:1].expand(5, 50), 4, "sigmoid", dev_logits=logits[:1].cuda().expand(5, 50))


def _sorted_choice(logits, k, score, bias, groups, top, best):
    """The choice for many rows by stable sorts in 64 bits on the device (finite logits)."""
    l = logits.double()
    T, E = l.shape
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    c = s + bias.double() if bias is not None else s
    order = c if bias is not None else l
    if groups > 1:
        by = c if bias is not None or best > 1 else l
        value = by.view(T, groups, -1).sort(dim=2, descending=True).values[:, :, :best].sum(2)
        at = value.sort(dim=1, descending=True, stable=True).indices[:, :top]
        keep = torch.zeros((T, groups), dtype=torch.bool, device=l.device).scatter_(1, at, True)
        order = order.masked_fill(~keep.repeat_interleave(E // groups, 1), -math.inf)
    return order.sort(dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32)


@pytest.mark.parametrize("spread", ["wide", "crowded", "equal"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top,best", [(128, 8, 1, 1, 1), (256, 8, 1, 1, 1), (256, 8, 8, 4, 2), (64, 15, 1, 1, 1), (256, 6, 8, 3, 1),
                                                 (512, 10, 1, 1, 1), (1024, 20, 16, 4, 2), (16, 1, 1, 1, 1), (16, 15, 1, 1, 1)])
def test_many_rows_against_sorts_in_64_bits(E, k, groups, top, best, score, spread):
    """wide: as routers give them; crowded: values within a few hundred roundings of each other, some equal; equal: few values."""
    print(f"route many E={E} k={k} groups={groups} {score} {spread}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(31)
    T = 20000
    r = torch.randn((T, E), generator=gen, device="cuda")
    if spread == "crowded":
        r = 1.0 + torch.randint(0, 300, (T, E), generator=gen, device="cuda") * 2.0 ** -23 + torch.randint(0, 3, (T, 1), generator=gen, device="cuda")
    elif spread == "equal":
        r = torch.randint(-2, 3, (T, E), generator=gen, device="cuda").float()
    small = 0.2 * torch.randn(E, generator=gen, device="cuda")
    # a softmax in torch and one here differ by 2^-50: sums that near each other are left to the tests of single rows
    for bias in (None, small, small * 2.0 ** -20) if score == "sigmoid" or spread == "wide" else (None,):
        if groups > 1 and best > 1 and spread != "wide" and score == "softmax":
            continue
        for dt in (torch.float32, torch.bfloat16):
            l = r.to(dt)
            got, _ = g.route_forward(l, k, score, bias=bias, groups=groups, top_groups=top, group_best=best)
            want = _sorted_choice(l, k, score, bias, groups, top, best)
            bad = (got != want).any(1)
            if bool(bad.any()):
                # 1 / (1 + exp) here and in torch may round differently in the last of 64 bits: only sums that near may differ
                rows = bad.nonzero()[:, 0]
                assert rows.numel() <= 3, (rows.numel(), rows[:4], got[rows[0]], want[rows[0]])
                s = torch.sigmoid(l[rows].double()) if score == "sigmoid" else torch.softmax(l[rows].double(), 1)
                c = s + (bias.double() if bias is not None else 0)
                a, b = c.gather(1, got[rows].long()), c.gather(1, want[rows].long())
                assert bool(((a - b).abs() <= 2.0 ** -50).all()), (got[rows[0]], want[rows[0]])


def test_no_tokens():
    e, p = g.route_forward(torch.empty((0, 8), device="cuda"), 2)
    assert e.shape == (0, 2) and p.shape == (0, 2)
    assert g.route_backward(p, torch.empty((0, 8), device="cuda"), e).shape == (0, 8)


def test_autograd_is_the_backward_and_the_slope():
    """Against the explicit call and against differences of the probabilities in the same experts."""
    logits = _logits(30, 48, torch.float32, 19).cuda()
    for score, renorm in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        l = logits.clone().requires_grad_()
        experts, probs = g.route(l, 6, score, renormalize=renorm, scale=1.5)
        assert not experts.requires_grad and probs.requires_grad
        d = torch.randn((30, 6), generator=torch.Generator().manual_seed(20)).cuda()
        probs.backward(d)
        assert torch.equal(l.grad, g.route_backward(d, logits, experts, score, renorm, 1.5))
        # p(l + h v) - p(l - h v) = 2 h <grad, v> + O(h^3); h = 2^-7 leaves 2^-14 of third derivatives (at most 2 |v|^3 each)
        v = torch.randn(logits.shape, generator=torch.Generator().manual_seed(21)).clamp(-2, 2).cuda()
        h = 2.0 ** -7

        def loss(x):
            rows = x.double()
            if score == "sigmoid":
                s = 1 / (1 + torch.exp(-rows))
            else:
                s = torch.softmax(rows, 1)
            s = s.gather(1, experts.long())
            return (1.5 * (s / s.sum(1, keepdim=True) if renorm else s) * d.double()).sum()
        slope = (loss(logits + h * v) - loss(logits - h * v)) / (2 * h)
        assert abs(float(slope - (l.grad.double() * v.double()).sum())) <= 1e-3 * float((l.grad.abs() * v.abs()).sum()) + 1e-4 * 30 * 6
    with pytest.raises(RuntimeError):
        l = logits.clone().requires_grad_()
        _, probs = g.route(l, 6)
        (first,) = torch.autograd.grad(probs.sum(), l, create_graph=True)
        first.sum().backward()


def test_experts_feed_a_dispatch_plan():
    logits = _logits(100, 16, torch.bfloat16, 22, masked=0.8).cuda()
    experts, probs = g.route_forward(logits, 4)
    plan = g.dispatch_plan(experts, 16)
    x = torch.randn((100, 32), device="cuda", dtype=torch.bfloat16)
    y = g.combine_forward(g.dispatch_forward(x, plan), plan, probs)
    live = (experts >= 0).any(1)
    # renormalized weights sum to 1 within k + 1 half steps, combine rounds once
    assert bool(((y.float() - x.float() * live[:, None]).abs() <= (2.0 ** -8 + 2.0 ** -18) * x.float().abs()).all())


def test_graph_replays_and_side_stream():
    l1, l2 = _logits(513, 128, torch.float32, 23).cuda(), _logits(513, 128, torch.float32, 24).cuda()
    logits, bias = l1.clone(), _bias(128, 25).cuda()
    d = torch.randn((513, 8), device="cuda")

    def step():
        a = g.route_forward(logits, 8, "sigmoid", bias=bias, groups=4, top_groups=2, group_best=2)
        b = g.route_forward(logits, 8, renormalize=False)
        return (*a, *b, g.route_backward(d, logits, a[0], "sigmoid"), g.route_backward(d, logits, b[0], renormalize=False))
    refs = []
    for l in (l1, l2):
        logits.copy_(l)
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
        logits.copy_(l1 if r % 2 == 0 else l2)
        for t in out:
            t.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(refs[r % 2], out)), r
    del graph


def test_more_rows_than_one_grid_row_holds():
    """Past 2^24 workgroups the grid is folded: two experts, every row's choice and weight."""
    T = (1 << 28) + 37
    logits = torch.zeros((T, 2), dtype=torch.float16, device="cuda")
    logits[1::2, 1] = 1.0
    logits[T - 1, 0] = 2.0
    experts, probs = g.route_forward(logits, 1, renormalize=False)
    want = (logits[:, 1] > logits[:, 0]).to(torch.int32)
    assert torch.equal(experts[:, 0], want)
    # the three rows there are
    for a, b in ((0.0, 0.0), (0.0, 1.0), (2.0, 0.0), (2.0, 1.0)):
        at = (logits[:, 0] == a) & (logits[:, 1] == b)
        if bool(at.any()):
            p = max(math.exp(a), math.exp(b)) / (math.exp(a) + math.exp(b))
            assert bool(((probs[:, 0][at].double() - p).abs() <= route_tol(2, 2) * p).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("E,groups,top,k", [(8, 2, 2, 7), (32, 4, 2, 8), (64, 4, 3, 7), (256, 8, 1, 9), (512, 4, 2, 20)])
@pytest.mark.parametrize("dt", list(TYPES))
def test_infinities_and_nan_in_groups(E, groups, top, k, best, score, dt):
    """A row with an infinite logit has no softmax that is a number: its experts are chosen all the same, NaN first."""
    logits = _logits(9, E, TYPES[dt], 41, masked=0.2)
    logits[1, 3] = logits[2, E - 1] = logits[3, E // 2] = logits[3, 0] = math.inf
    logits[4, 1] = logits[5, E - 2] = math.nan
    logits[5, 2] = logits[6, E // 2 - 1] = math.inf
    logits[6] = torch.where(logits[6] == math.inf, logits[6], torch.full_like(logits[6], -math.inf))
    some = _bias(E, 42)
    high = some.clone()
    high[::5] = math.inf
    low = some.clone()
    low[1::3] = -math.inf
    for bias in (None, some, high, low):
        _check(logits, k, score, bias, groups, top, best)
        _check(logits, k, score, bias, groups, top, best, renormalize=False)
