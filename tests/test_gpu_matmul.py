"""grouped_matmul (bf16 / fp16 products grouped by expert) against plain 64-bit products."""
import pytest
import torch

import nvfp4_block_scaled_mxfp8_amd as g
from mm_util import DTYPES, assert_close, ints, product, randn, spans

pytestmark = pytest.mark.gpu

# (splits, M, N, K): one row, empty and one-row groups, more than 64 groups, rows behind the last
# group, sizes on both sides of the tiles' and of the 16-byte loads' multiples
CASES = {
    "one": ([1], 1, 1, 1),
    "toy": ([64, 128], 192, 256, 128),
    "ragged": ([0, 1, 0, 37, 5], 50, 40, 24),
    "odd": ([3, 0, 100], 103, 33, 17),
    "many": ([i % 3 for i in range(70)] + [0] * 59 + [4], 80, 72, 64),
    "k_tail": ([130, 0, 257], 390, 264, 200),
    "wide": ([500, 0, 1, 700], 1201, 512, 640),
    "odd_k": ([128, 65], 193, 128, 129),
    "odd_n": ([128, 65], 193, 129, 128),
    "empty": ([0, 0, 0], 5, 64, 64),
    "no_rows": ([0, 0], 0, 64, 64),
    "no_rows_long": ([0, 0], 0, 1000, 1024),      # a contraction that would be cut into parts
    "tall": ([1000], 1000, 8, 2048),
    # the 256 x 256 stream: column tiles enough, groups of several row tiles and a ragged one, rows behind
    # the last group; as forward, as dgrad (and the other as a contraction cut into parts)
    "stream_n": ([700, 0, 1200, 49], 2048, 8200, 72),
    "stream_k": ([700, 0, 1200, 49], 2048, 72, 8200),
    "stream_one": ([2400], 2400, 6656, 200),
    # weight gradients by the stream: with few and with many tiles a group, and more groups than are sorted
    "stream_w": ([0, 65, 1, 300, 64, 0, 17, 128, 5], 600, 1032, 1544),
    "stream_x": ([3, 0, 150, 140], 300, 2056, 2056),
    "stream_g": ([i % 2 for i in range(1100)] + [77], 700, 64, 72),
}


def _case(name, dt, make=randn):
    splits, M, N, K = CASES[name]
    G = len(splits)
    d = {"x": make((M, K), dt, 1), "w": make((G, N, K), dt, 2), "dy": make((M, N), dt, 3)}
    d["splits"] = splits
    return d, M, N, K


def _up(d):
    r = {k: v.cuda() for k, v in d.items() if k != "splits"}
    r["m"] = torch.tensor(d["splits"], dtype=torch.int32, device="cuda")
    return r


def _check_all(d, dev, M, N, K, y, dx, dw, what):
    sp, used = spans(d["splits"], M)
    for i, (a, b) in enumerate(sp):
        if b > a:
            assert_close(y[a:b], *product(d["x"][a:b], d["w"][i].t()), K, f"{what} y group {i}")
            assert_close(dx[a:b], *product(d["dy"][a:b], d["w"][i]), N, f"{what} dx group {i}")
        assert_close(dw[i], *product(d["dy"][a:b].t(), d["x"][a:b]), b - a, f"{what} dw group {i}")
    assert not y[used:].any() and not dx[used:].any(), what


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("name", list(CASES))
def test_products_against_64_bits(name, dt):
    print(f"products {name} {dt}", flush=True)
    d, M, N, K = _case(name, DTYPES[dt])
    v = _up(d)
    y = g.grouped_matmul_forward(v["x"], v["w"], v["m"])
    dx = g.grouped_matmul_dgrad(v["dy"], v["w"], v["m"])
    dw = g.grouped_matmul_wgrad(v["dy"], v["x"], v["m"])
    _check_all(d, v, M, N, K, y, dx, dw, f"{name} {dt}")
    dw32 = g.grouped_matmul_wgrad(v["dy"], v["x"], v["m"], g.OUT_FP32)
    assert dw32.dtype == torch.float32 and torch.equal(dw32.to(dw.dtype), dw)
    acc = randn(tuple(dw.shape), torch.float32, 9).cuda()
    want = acc + dw32
    r = g.grouped_matmul_wgrad(v["dy"], v["x"], v["m"], g.OUT_FP32_ACCUMULATE, out=acc)
    assert r is acc and torch.equal(acc, want)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("name", ["ragged", "k_tail", "wide", "odd", "stream_k", "stream_w"])
def test_strides_and_offsets(name, dt):
    """Views: rows inside wider tensors, starts that are not 16-byte aligned, weights with gaps, and
    transposed inputs (copied).  The same bits as the contiguous tensors where the kernel is the same."""
    print(f"strides {name} {dt}", flush=True)
    d, M, N, K = _case(name, DTYPES[dt])
    v = _up(d)
    for pad, off in ((8, 0), (8, 8), (3, 1), (1, 0)):
        def view(t):
            big = torch.full(tuple(t.shape[:-1]) + (t.shape[-1] + pad,), float("nan"), dtype=t.dtype, device="cuda")
            w = big[..., off:off + t.shape[-1]]
            w.copy_(t)
            return w
        xs, ws, dys = view(v["x"]), view(v["w"]), view(v["dy"])
        y = view(torch.zeros((M, N), dtype=v["x"].dtype, device="cuda"))
        guard = torch.as_strided(y, (M, N + pad), (N + pad, 1), y.storage_offset() - off).clone()
        g.grouped_matmul_forward(xs, ws, v["m"], out=y)
        after = torch.as_strided(y, (M, N + pad), (N + pad, 1), y.storage_offset() - off)
        outside = torch.ones(N + pad, dtype=torch.bool, device="cuda")
        outside[off:off + N] = False
        assert torch.equal(after[:, outside].isnan(), guard[:, outside].isnan())
        _check_all(d, v, M, N, K, y, g.grouped_matmul_dgrad(dys, ws, v["m"]), g.grouped_matmul_wgrad(dys, xs, v["m"]),
                   f"{name} {dt} pad {pad} off {off}")
    xt = v["x"].t().contiguous().t()
    assert torch.equal(g.grouped_matmul_forward(xt, v["w"], v["m"]), g.grouped_matmul_forward(v["x"], v["w"], v["m"]))


@pytest.mark.parametrize("name", ["ragged", "wide", "stream_n", "stream_k"])
def test_given_output_keeps_rows_behind(name):
    d, M, N, K = _case(name, torch.bfloat16)
    v = _up(d)
    _, used = spans(d["splits"], M)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full((M, K), 7.0, dtype=torch.bfloat16, device="cuda")
    g.grouped_matmul_forward(v["x"], v["w"], v["m"], out=y)
    g.grouped_matmul_dgrad(v["dy"], v["w"], v["m"], out=dx)
    assert bool((y[used:] == 7).all()) and bool((dx[used:] == 7).all())
    assert torch.equal(y[:used], g.grouped_matmul_forward(v["x"], v["w"], v["m"])[:used])


@pytest.mark.parametrize("splits", [[100, 100, 100], [-5, 20, 2 ** 31 - 1, 2 ** 31 - 1], [40, -1, 30], [2 ** 31 - 1] * 70])
def test_bad_splits_are_clamped(splits):
    """Splits that pass M or are negative: clamped, flagged, nothing outside the rows touched."""
    M, N, K = 128, 72, 64
    G = len(splits)
    d = {"x": randn((M, K), torch.bfloat16, 1), "w": randn((G, N, K), torch.bfloat16, 2),
         "dy": randn((M, N), torch.bfloat16, 3), "splits": splits}
    v = _up(d)
    ws = torch.zeros(g.grouped_matmul_ws_bytes(g.GEMM_FPROP, G, M, N, K), dtype=torch.uint8, device="cuda")
    y = g.grouped_matmul_forward(v["x"], v["w"], v["m"], ws=ws)
    total = sum(max(s, 0) for s in splits)
    want = (1 if min(splits) < 0 else 0) | (2 if total > M else 0) | (4 if total < M else 0)
    assert g.read_device_flags(ws) == want
    _check_all(d, v, M, N, K, y, g.grouped_matmul_dgrad(v["dy"], v["w"], v["m"]),
               g.grouped_matmul_wgrad(v["dy"], v["x"], v["m"]), f"splits {splits[:4]}")


@pytest.mark.parametrize("K", [64, 200, 17])
def test_nan_and_infinity_stay_in_their_rows(K):
    """A NaN or infinite row reaches its own output row only, an expert's NaN weights only its own
    rows, and rows behind the last group no gradient."""
    splits, M, N = [70, 0, 61], 140, 136
    d = {"x": randn((M, K), torch.bfloat16, 1), "w": randn((3, N, K), torch.bfloat16, 2),
         "dy": randn((M, N), torch.bfloat16, 3), "splits": splits}
    v = _up(d)
    y0 = g.grouped_matmul_forward(v["x"], v["w"], v["m"])
    dw0 = g.grouped_matmul_wgrad(v["dy"], v["x"], v["m"])
    x = v["x"].clone()
    x[5, K - 1] = float("nan")
    x[69, 0] = float("inf")
    x[131:] = float("nan")
    dy = v["dy"].clone()
    dy[131:] = float("inf")
    w = v["w"].clone()
    w[1] = float("nan")
    y = g.grouped_matmul_forward(x, w, v["m"])
    rows = torch.ones(M, dtype=torch.bool)
    rows[5] = rows[69] = False
    assert torch.equal(y[rows], y0[rows])
    assert bool(y[5].isnan().all()) and bool((~y[69].isfinite()).all())
    dw = g.grouped_matmul_wgrad(dy, x, v["m"])
    assert torch.equal(dw[1:], dw0[1:])
    assert bool(dw[0, :, K - 1].isnan().all())
    if K > 1:
        assert torch.equal(dw[0, :, 1:K - 1], dw0[0, :, 1:K - 1])


def test_nan_and_infinity_stay_in_their_rows_of_the_stream():
    """The same for the 256 x 256 stream: rows, weights and gradients beside the ones that are not finite,
    contraction and row tails inside a tile."""
    splits, M, N, K = [700, 0, 1200, 49], 2048, 8200, 72
    d = {"x": randn((M, K), torch.bfloat16, 1), "w": randn((4, N, K), torch.bfloat16, 2), "splits": splits}
    v = _up(d)
    y0 = g.grouped_matmul_forward(v["x"], v["w"], v["m"])
    x, w = v["x"].clone(), v["w"].clone()
    bad = [0, 255, 699, 700, 1899, 1948]
    x[bad, K - 1] = float("nan")
    x[1949:] = float("inf")
    w[1] = float("nan")
    y = g.grouped_matmul_forward(x, w, v["m"])
    rows = torch.ones(M, dtype=torch.bool)
    rows[bad] = False
    assert torch.equal(y[rows], y0[rows]) and bool(y[bad].isnan().all())
    splits, M, N, K = [0, 65, 1, 300, 64, 0, 17, 128, 5], 600, 1032, 1544
    m = torch.tensor(splits, dtype=torch.int32, device="cuda")
    x, dy = randn((M, K), torch.bfloat16, 3).cuda(), randn((M, N), torch.bfloat16, 4).cuda()
    dw0 = g.grouped_matmul_wgrad(dy, x, m)
    x[580:] = float("nan")
    dy[580:] = float("inf")
    x[66, 5] = float("nan")                              # the first row of group 3
    dw = g.grouped_matmul_wgrad(dy, x, m)
    others = [0, 1, 2, 4, 5, 6, 7, 8]
    assert torch.equal(dw[others], dw0[others])
    cols = torch.arange(K) != 5
    assert torch.equal(dw[3][:, cols], dw0[3][:, cols]) and bool(dw[3][:, 5].isnan().all())


@pytest.mark.parametrize("dt", list(DTYPES))
def test_autograd_against_formula_and_differences(dt):
    """Integer inputs small enough that every result is exact: the gradients equal the formula's bit
    for bit, and a central difference of sum(dy y) along random directions equals <grad, direction>."""
    dtype = DTYPES[dt]
    splits, M, N, K = [5, 0, 9], 16, 24, 16
    x, w, dy = ints((M, K), dtype, 1), ints((3, N, K), dtype, 2), ints((M, N), dtype, 3, -1, 1)
    m = torch.tensor(splits, dtype=torch.int32, device="cuda")
    xd, wd = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    y = g.grouped_matmul(xd, wd, m)
    y.backward(dy.cuda())
    sp, used = spans(splits, M)
    for i, (a, b) in enumerate(sp):
        assert torch.equal(xd.grad[a:b].cpu().double(), dy[a:b].double() @ w[i].double())
        assert torch.equal(wd.grad[i].cpu().double(), dy[a:b].double().t() @ x[a:b].double())
    assert not xd.grad[used:].any()

    def loss(xx, ww):
        return float((g.grouped_matmul_forward(xx, ww, m).double() * dy.cuda().double()).sum())
    for seed in range(3):
        ex, ew = ints((M, K), dtype, 10 + seed, 0, 1).cuda(), ints((3, N, K), dtype, 20 + seed, 0, 1).cuda()
        dxdir = loss(xd.detach() + ex, wd.detach()) - loss(xd.detach() - ex, wd.detach())
        dwdir = loss(xd.detach(), wd.detach() + ew) - loss(xd.detach(), wd.detach() - ew)
        assert dxdir == 2 * float((xd.grad.double() * ex.double()).sum())
        assert dwdir == 2 * float((wd.grad.double() * ew.double()).sum())


def test_autograd_partial_and_main_grad():
    splits, M, N, K = [30, 34], 64, 64, 128
    m = torch.tensor(splits, dtype=torch.int32, device="cuda")
    x, w = randn((M, K), torch.bfloat16, 1).cuda(), randn((2, N, K), torch.bfloat16, 2).cuda()
    dy = randn((M, N), torch.bfloat16, 3).cuda()
    xr = x.clone().requires_grad_()
    g.grouped_matmul(xr, w, m).backward(dy)
    assert torch.equal(xr.grad, g.grouped_matmul_dgrad(dy, w, m))
    wr = w.clone().requires_grad_()
    wr.main_grad = torch.ones(w.shape, dtype=torch.float32, device="cuda")
    g.grouped_matmul(x, wr, m, accumulate_main_grad=True).backward(dy)
    assert wr.grad is None
    assert torch.equal(wr.main_grad, 1 + g.grouped_matmul_wgrad(dy, x, m, g.OUT_FP32))


def test_side_stream_and_graph_replays():
    """The three products on a side stream and captured, each replay against the eager bits."""
    d, M, N, K = _case("wide", torch.bfloat16)
    v = _up(d)

    def step():
        return (g.grouped_matmul_forward(v["x"], v["w"], v["m"]), g.grouped_matmul_dgrad(v["dy"], v["w"], v["m"]),
                g.grouped_matmul_wgrad(v["dy"], v["x"], v["m"]))
    ref = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(ref, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(3):
        for t in out:
            t.fill_(3)
        step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, out):
            assert torch.equal(a, b), r
    del graph
