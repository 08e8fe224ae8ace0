"""lora (low-rank adapters of many requests) against the 64-bit formulas."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_mxfp8_amd as g
from mm_util import DTYPES, floor_step, half_step, ints, np_ids, randn

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -23          # a whole unit of an fp32 partial sum, allowed at every addition
SPLIT = 2.0 ** -17        # a factor kept as two 16-bit values (bf16: 2^-18 of it; fp16: less)

# M, K, N, R, L, share of rows without an adapter
CASES = {
    "one": (1, 8, 8, 1, 1, 0.0),
    "decode": (32, 1024, 512, 16, 16, 0.1),
    "rank3": (37, 65, 50, 3, 4, 0.2),
    "rank8": (100, 264, 136, 8, 3, 0.0),
    "rank24": (70, 512, 320, 24, 5, 0.1),
    "rank64": (300, 1000, 264, 64, 2, 0.1),
    "rank128": (129, 640, 512, 128, 3, 0.0),
    "rank100": (65, 136, 72, 100, 2, 0.5),
    "none": (20, 64, 64, 16, 2, 1.0),
    "many": (500, 128, 128, 8, 200, 0.0),
    "tiles64": (1100, 64, 4100, 16, 3, 0.1),          # expand tiles of 64 positions, shrink of 16
    "tiles128": (5000, 64, 6000, 24, 2, 0.1),        # of 128 and 32
    "long": (3000, 256, 520, 16, 3, 0.05),
    "long33": (2100, 200, 264, 33, 1, 0.0),
    "no_rows": (0, 64, 64, 8, 2, 0.0),
}


def _case(name, dt, make=randn):
    M, K, N, R, L, drop = CASES[name]
    d = {"base": make((M, N), dt, 1), "x": make((M, K), dt, 2), "a": make((L, R, K), dt, 3, *((K ** -0.5,) if make is randn else ())),
         "b": make((L, N, R), dt, 4), "dy": make((M, N), dt, 5), "ids": torch.from_numpy(np_ids(M, L, 6, drop)),
         "scales": 0.25 + torch.rand(L, generator=torch.Generator().manual_seed(7))}
    if name == "many":
        d["ids"][:] = torch.from_numpy(np_ids(M, 60, 6))          # most adapters have no row
    return d


def _reference(d):
    """Outputs and the errors they may have: {name: (value, tolerance)} in 64 bits."""
    x, a, b, dy, s = (d[k].double() for k in ("x", "a", "b", "dy", "scales"))
    M, K = x.shape
    N, R = b.shape[1], b.shape[2]
    dt = d["x"].dtype
    y, ty = d["base"].double().clone(), torch.zeros(M, N, dtype=torch.float64)
    dx, tdx = torch.zeros(M, K, dtype=torch.float64), torch.zeros(M, K, dtype=torch.float64)
    da, tda = torch.zeros_like(a), torch.zeros_like(a)
    db, tdb = torch.zeros_like(b), torch.zeros_like(b)
    for l in range(a.shape[0]):
        m = (d["ids"] == l).nonzero().flatten()
        n = m.numel()
        if n == 0:
            continue
        u, eu = x[m] @ a[l].t(), (K + 8) * F32 * (x[m].abs() @ a[l].abs().t())
        du, edu = s[l] * (dy[m] @ b[l]), (N + 8) * F32 * s[l] * (dy[m].abs() @ b[l].abs())
        eu, edu = eu + SPLIT * u.abs() + 2.0 ** -38 * u.abs().max(), edu + SPLIT * du.abs() + 2.0 ** -38 * du.abs().max()
        y[m] += s[l] * (u @ b[l].t())
        ty[m] = s[l] * (eu @ b[l].abs().t()) + (2 * R + 8) * F32 * (s[l] * (u.abs() @ b[l].abs().t()) + d["base"][m].double().abs())
        dx[m] = du @ a[l]
        tdx[m] = edu @ a[l].abs() + (2 * R + 8) * F32 * (du.abs() @ a[l].abs())
        da[l] = du.t() @ x[m]
        tda[l] = edu.t() @ x[m].abs() + (2 * n + 8) * F32 * (du.abs().t() @ x[m].abs())
        db[l] = s[l] * (dy[m].t() @ u)
        tdb[l] = s[l] * (dy[m].abs().t() @ eu) + (2 * n + 8) * F32 * s[l] * (dy[m].abs().t() @ u.abs())
    out = {}
    for k, v, t in (("y", y, ty), ("dx", dx, tdx), ("da", da, tda), ("db", db, tdb)):
        out[k] = (v, t * (1 + 2.0 ** -7) + half_step(dt) * v.abs() + floor_step(dt))
    return out


def _close(got, ref, what):
    want, tol = ref
    out = got.detach().cpu().double()
    err = (out - want).abs()
    # a value past the type's largest by more than its tolerance rounds to infinity
    over = want.abs() - tol > torch.finfo(got.dtype).max * (1 + half_step(got.dtype))
    bad = torch.where(over, out != want.sign() * float("inf"), ~(err <= tol))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol.clamp(min=1e-300)).max()):.2f} of the tolerance"


def _run(d, **kw):
    v = {k: t.cuda() for k, t in d.items()}
    y, ctx = g.lora_forward(v["base"], v["x"], v["a"], v["b"], v["ids"], v["scales"])
    r = g.lora_backward(v["dy"], v["x"], v["a"], v["b"], ctx, **kw)
    r["y"] = y
    return r


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_gradients_against_64_bits(name, dt):
    print(f"lora {name} {dt}", flush=True)
    d = _case(name, DTYPES[dt])
    ref, got = _reference(d), _run(d)
    for k in ("y", "dx", "da", "db"):
        _close(got[k], ref[k], f"{name} {dt} {k}")
    none = (d["ids"] < 0)
    assert torch.equal(got["y"].cpu()[none], d["base"][none]) and not got["dx"].cpu()[none].any()
    for l in range(d["a"].shape[0]):
        if not (d["ids"] == l).any():
            assert not got["da"][l].any() and not got["db"][l].any()


@pytest.mark.parametrize("name", ["decode", "rank3", "long"])
def test_in_place_without_base_without_scales(name):
    d = _case(name, torch.bfloat16)
    v = {k: t.cuda() for k, t in d.items()}
    y, ctx = g.lora_forward(v["base"], v["x"], v["a"], v["b"], v["ids"], v["scales"])
    same = v["base"].clone()
    y2, _ = g.lora_forward(same, v["x"], v["a"], v["b"], v["ids"], v["scales"], out=same)
    assert y2 is same and torch.equal(y, same)
    zero, _ = g.lora_forward(torch.zeros_like(v["base"]), v["x"], v["a"], v["b"], v["ids"], v["scales"])
    y3, _ = g.lora_forward(None, v["x"], v["a"], v["b"], v["ids"], v["scales"])
    assert torch.equal(y3, zero)
    ones, _ = g.lora_forward(v["base"], v["x"], v["a"], v["b"], v["ids"], torch.ones_like(v["scales"]))
    y4, _ = g.lora_forward(v["base"], v["x"], v["a"], v["b"], v["ids"])
    assert torch.equal(y4, ones)
    r = g.lora_backward(v["dy"], v["x"], v["a"], v["b"], ctx)
    add = randn(tuple(v["x"].shape), torch.bfloat16, 9).cuda()
    ra = g.lora_backward(v["dy"], v["x"], v["a"], v["b"], ctx, dx_add=add, need_da=False, need_db=False)
    assert ra["da"] is None and ra["db"] is None
    none = (v["ids"] < 0)
    assert torch.equal(ra["dx"][none], add[none])
    ref = _reference(d)["dx"]
    want = ref[0] + add.cpu().double()
    _close(ra["dx"], (want, ref[1] + half_step(torch.bfloat16) * want.abs() + 8 * F32 * add.cpu().double().abs()), "dx_add")
    only = g.lora_backward(v["dy"], v["x"], v["a"], v["b"], ctx, need_dx=False)
    assert only["dx"] is None and torch.equal(only["da"], r["da"]) and torch.equal(only["db"], r["db"])


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("name", ["rank8", "rank24", "rank3"])
def test_strides_and_offsets(name, dt):
    print(f"lora strides {name} {dt}", flush=True)
    d = _case(name, DTYPES[dt])
    ref = _reference(d)
    v = {k: t.cuda() for k, t in d.items()}
    for pad, off in ((8, 0), (8, 8), (3, 1)):
        def view(t):
            big = torch.full(tuple(t.shape[:-1]) + (t.shape[-1] + pad,), float("nan"), dtype=t.dtype, device="cuda")
            w = big[..., off:off + t.shape[-1]]
            w.copy_(t)
            return w
        w = {k: view(v[k]) for k in ("base", "x", "a", "b", "dy")}
        y, ctx = g.lora_forward(w["base"], w["x"], w["a"], w["b"], v["ids"], v["scales"])
        r = g.lora_backward(w["dy"], w["x"], w["a"], w["b"], ctx)
        r["y"] = y
        for k in ("y", "dx", "da", "db"):
            _close(r[k], ref[k], f"{name} {dt} pad {pad} off {off} {k}")
    bt = v["b"].transpose(1, 2).contiguous().transpose(1, 2)          # R not contiguous: copied
    assert torch.equal(g.lora_forward(v["base"], v["x"], v["a"], bt, v["ids"], v["scales"])[0],
                       g.lora_forward(v["base"], v["x"], v["a"], v["b"], v["ids"], v["scales"])[0])


@pytest.mark.parametrize("bad", [-1, 5, 2 ** 31 - 1, -2 ** 31])
def test_ids_outside_mean_no_adapter(bad):
    d = _case("rank24", torch.bfloat16)
    d["ids"][d["ids"] < 0] = -1
    a = _run(d)
    d["ids"][d["ids"] < 0] = bad
    b = _run(d)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_nan_and_infinity_stay_where_they_belong():
    """A NaN row reaches its own row and its adapter's gradients only; an unused adapter's NaN nothing."""
    d = _case("rank24", torch.bfloat16)
    d["ids"][:] = torch.arange(70) % 3
    d["a"][4] = float("nan")
    d["b"][3] = float("inf")
    clean = _run(d)
    assert all(bool(t.isfinite().all()) for t in (clean["y"], clean["dx"], clean["da"][:3], clean["db"][:3]))
    e = {k: t.clone() for k, t in d.items()}
    e["x"][7] = float("nan")            # adapter 1
    got = _run(e)
    rows = torch.arange(70) != 7
    assert torch.equal(got["y"][rows], clean["y"][rows]) and bool(got["y"][7].isnan().all())
    assert torch.equal(got["dx"], clean["dx"])
    assert bool(got["da"][1].isnan().all()) and torch.equal(got["da"][0], clean["da"][0]) and torch.equal(got["db"][2], clean["db"][2])


def _elementwise(d):
    """y, dx, da, db by the formulas, every product written out in 64 bits (an infinity times zero is NaN)."""
    x, a, b, dy, s = (d[k].double() for k in ("x", "a", "b", "dy", "scales"))
    out = {"y": d["base"].double().clone(), "dx": torch.zeros_like(x), "da": torch.zeros_like(a), "db": torch.zeros_like(b)}
    for l in range(a.shape[0]):
        m = (d["ids"] == l).nonzero().flatten()
        if m.numel() == 0:
            continue
        u = (x[m][:, None] * a[l]).sum(2)
        du = s[l] * (dy[m][:, :, None] * b[l]).sum(1)
        out["y"][m] += s[l] * (u[:, None] * b[l]).sum(2)
        out["dx"][m] = (du[:, :, None] * a[l]).sum(1)
        out["da"][l] = (du[:, :, None] * x[m][:, None]).sum(0)
        out["db"][l] = s[l] * (dy[m][:, :, None] * u[:, None]).sum(0)
    return out


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("R", [4, 24, 100])
@pytest.mark.parametrize("where", ["b", "a", "x", "dy"])
@pytest.mark.parametrize("whole", [True, False])
def test_infinities_as_in_the_formula(whole, where, R, dt):
    """An infinity in a factor gives infinities of the formula's sign, and NaN where the formula has one: the
    rank-sized factors' second 16-bit value (zero, or of the other sign) does not turn them into NaN.
    Whole numbers: every finite result is exact."""
    M, K, N, L = 140, 24, 40, 2
    make = (lambda s, i, lo: ints(s, DTYPES[dt], i, lo, 1)) if whole else (lambda s, i, lo: randn(s, DTYPES[dt], i))
    d = {"base": make((M, N), 1, -1), "x": make((M, K), 2, -1), "a": make((L, R, K), 3, -1), "b": make((L, N, R), 4, -1),
         "dy": make((M, N), 5, -1), "ids": (torch.arange(M) % 3 - 1).to(torch.int32), "scales": torch.tensor([1.0, 2.0])}
    inf = float("inf")
    if where == "b":
        d["b"][0, 3, 1], d["b"][1, N - 1, R - 1] = inf, -inf
    elif where == "a":
        d["a"][0, 2, 5], d["a"][1, R - 1, K - 1] = -inf, inf
    elif where == "x":
        d["x"][1, 4], d["x"][M - 1, K - 1] = inf, -inf
    else:
        d["dy"][4, 7], d["dy"][M - 1, N - 1] = -inf, inf
    ref, got = _elementwise(d), _run(d)
    for k, want in ref.items():
        v = got[k].cpu().double()
        assert torch.equal(v.isnan(), want.isnan()), (k, int(v.isnan().sum()), int(want.isnan().sum()))
        assert torch.equal(v == inf, want == inf) and torch.equal(v == -inf, want == -inf), k
        if whole:
            assert torch.equal(v[want.isfinite()], want[want.isfinite()].to(DTYPES[dt]).double()), k


def test_large_factors_keep_their_value():
    """A finite u past the operands' largest value stays finite: in fp16 beside another rank's infinity (u =
    inf, 120001), in bf16 between its largest value and fp32's."""
    ids = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, a, b = torch.zeros(1, 16), torch.zeros(1, 2, 16), torch.tensor([[[1.0, -1.0], [-0.5, 0.25]]])
    x[0, :2] = torch.tensor([1.0, 40000.0])
    a[0, :, :2] = torch.tensor([[float("inf"), 1.0], [1.0, 3.0]])
    y, _ = g.lora_forward(None, x.half().cuda(), a.half().cuda(), b.half().cuda(), ids)
    assert y.tolist() == [[float("inf"), -float("inf")]]
    x[0, :2] = torch.tensor([2.0 ** 127, 2.0 ** 119])
    a = torch.zeros(1, 1, 16)
    a[0, 0, :2] = torch.tensor([1.9921875, 1.5])         # u = 2^127 1.998046875
    b = torch.tensor([[[2.0 ** -126], [-(2.0 ** -125)]]])
    t = torch.bfloat16
    y, _ = g.lora_forward(None, x.to(t).cuda(), a.to(t).cuda(), b.to(t).cuda(), ids)
    assert y.tolist() == [[4.0, -8.0]]                   # 3.99609375 and -7.9921875 to eight bits


def test_fp16_range():
    """fp16: u above 65504 and du below 2^-24 keep their bits (powers of two through the factors)."""
    M, K, N, R = 20, 64, 64, 16
    for up in (2.0 ** 9, 2.0 ** -9):
        x = (ints((M, K), torch.float32, 1, 1, 3) * up).half()
        a = (ints((1, R, K), torch.float32, 2, 1, 2) * up).half()
        b = (ints((1, N, R), torch.float32, 3, 1, 2) / (up * up if up > 1 else 1)).half()
        dy = (ints((M, N), torch.float32, 4, 1, 3) * (1 if up > 1 else 2.0 ** -12)).half()
        d = {"base": torch.zeros(M, N).half(), "x": x, "a": a, "b": b, "dy": dy, "ids": torch.zeros(M, dtype=torch.int32),
             "scales": torch.ones(1)}
        ref, got = _reference(d), _run(d)
        for k in ("y", "dx", "da", "db"):
            _close(got[k], ref[k], f"range {up} {k}")


@pytest.mark.parametrize("dt", list(DTYPES))
def test_autograd_against_formula_and_differences(dt):
    """Small integers: all exact; the gradients equal the formulas and central differences."""
    dtype = DTYPES[dt]
    M, K, N, R, L = 13, 16, 24, 4, 3
    ids = torch.tensor([0, 1, 0, -1, 1, 0, 0, 1, 1, 0, -1, 0, 1], dtype=torch.int32)
    t = {"base": ints((M, N), dtype, 1), "x": ints((M, K), dtype, 2, -1, 1), "a": ints((L, R, K), dtype, 3, -1, 1),
         "b": ints((L, N, R), dtype, 4, -1, 1)}
    dy = ints((M, N), dtype, 5, -1, 1).cuda()
    scales = torch.tensor([1.0, 2.0, 1.0]).cuda()
    leaf = {k: v.cuda().requires_grad_() for k, v in t.items()}
    g.lora(leaf["base"], leaf["x"], leaf["a"], leaf["b"], ids.cuda(), scales).backward(dy)
    d = dict(t, dy=dy.cpu(), ids=ids, scales=scales.cpu())
    ref = _reference(d)
    assert torch.equal(leaf["base"].grad, dy)
    for k, n in (("x", "dx"), ("a", "da"), ("b", "db")):
        assert torch.equal(leaf[k].grad.cpu().double(), ref[n][0]), k

    def loss(**kw):
        v = {k: kw.get(k, leaf[k].detach()) for k in leaf}
        y, _ = g.lora_forward(v["base"], v["x"], v["a"], v["b"], ids.cuda(), scales)
        return float((y.double() * dy.double()).sum())
    for k in ("base", "x", "a", "b"):
        e = ints(tuple(t[k].shape), dtype, 30, 0, 1).cuda()
        p = leaf[k].detach()
        assert loss(**{k: p + e}) - loss(**{k: p - e}) == 2 * float((leaf[k].grad.double() * e.double()).sum()), k


def test_graph_replays_and_side_stream():
    d = _case("long", torch.bfloat16)
    v = {k: t.cuda() for k, t in d.items()}
    ids2 = v["ids"].flip(0).clone()
    ids1 = v["ids"].clone()

    def step():
        y, ctx = g.lora_forward(v["base"], v["x"], v["a"], v["b"], v["ids"], v["scales"])
        r = g.lora_backward(v["dy"], v["x"], v["a"], v["b"], ctx)
        return y, r["dx"], r["da"], r["db"]
    refs = []
    for i in (ids1, ids2):
        v["ids"].copy_(i)
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
        v["ids"].copy_(ids1 if r % 2 == 0 else ids2)
        for t in out:
            t.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(refs[r % 2], out)), r
    del graph
