"""Kernels of the bf16 / fp16 operators that only sizes of some weight reach: weights loaded once, tiles of
many positions at high rank, non-temporal moves, tables of many groups; and bad splits there."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_mxfp8_amd as g
from mm_util import DTYPES, assert_close, np_ids, product, randn, spans
from test_gpu_lora import _close, _reference, _run

pytestmark = pytest.mark.gpu


def _grouped(splits, M, N, K, dt, wgrad=True):
    """Forward, dgrad (and wgrad) against 64-bit products, new outputs and given ones."""
    x, dy = randn((M, K), dt, 1), randn((M, N), dt, 3)
    w = torch.empty((len(splits), N, K), dtype=dt, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(2))
    m = torch.tensor(splits, dtype=torch.int32, device="cuda")
    sp, used = spans(splits, M)
    for i, (a, b) in enumerate(sp):
        if a == b:
            w[i] = float("nan")                          # no row's: reaches nothing
    xd, dyd = x.cuda(), dy.cuda()
    y, dx = g.grouped_matmul_forward(xd, w, m), g.grouped_matmul_dgrad(dyd, w, m)
    keep = torch.full((M, N), 5.0, dtype=dt, device="cuda")
    g.grouped_matmul_forward(xd, w, m, out=keep)
    dw = g.grouped_matmul_wgrad(dyd, xd, m) if wgrad else None
    assert torch.equal(keep[:used], y[:used]) and bool((keep[used:] == 5).all())
    for i, (a, b) in enumerate(sp):
        if b > a:
            wi = w[i].cpu()
            assert_close(y[a:b], *product(x[a:b], wi.t()), K, f"y group {i}")
            assert_close(dx[a:b], *product(dy[a:b], wi), N, f"dx group {i}")
        if wgrad:
            assert_close(dw[i], *product(dy[a:b].t(), x[a:b]), b - a, f"dw group {i}")
    assert not y[used:].any() and not dx[used:].any()


@pytest.mark.parametrize("dt", list(DTYPES))
def test_weights_that_are_loaded_once(dt):
    """64 experts' weights of 604 MB: groups of one row tile (non-temporal) beside ones of two."""
    splits = [0, 1, 2, 200, 129, 128, 127, 0, 64, 65] + [1 + i % 5 for i in range(53)] + [300]
    print(f"weights once {dt}", flush=True)
    _grouped(splits, sum(splits) + 11, 2048, 2304, DTYPES[dt], wgrad=False)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_weights_that_are_loaded_once_in_parts(dt):
    """One group's weights of 525 MB and few rows: a contraction cut into parts, non-temporal.  Every 41st column
    and the last ones."""
    print(f"weights once in parts {dt}", flush=True)
    M, N, K = 50, 32000, 8200
    t = DTYPES[dt]
    w = torch.empty((1, N, K), dtype=t, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(2))
    x, m = randn((M, K), t, 1), torch.tensor([47], dtype=torch.int32, device="cuda")
    cols = list(range(0, N, 41)) + list(range(N - 9, N))
    y = g.grouped_matmul_forward(x.cuda(), w, m)
    assert_close(y[:47, cols], *product(x[:47], w[0, cols].cpu().t()), K, "y")
    dx = g.grouped_matmul_dgrad(x.cuda(), w.view(1, K, N), m)          # the same memory as [K, N]
    assert_close(dx[:47, cols], *product(x[:47], w.view(K, N)[:, cols].cpu()), K, "dx")
    assert not y[47:].any() and not dx[47:].any()


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("N,K", [(33, 17), (40, 24), (129, 264), (5, 700)])
def test_long_groups_of_small_weight_gradients(N, K, dt):
    """Few tiles and many rows: weight gradients cut into parts, aligned and not."""
    print(f"parts of wgrad {N} x {K} {dt}", flush=True)
    _grouped([1200, 3, 0, 2000], 3210, N, K, DTYPES[dt])


@pytest.mark.parametrize("rest", [0, 70])
@pytest.mark.parametrize("G", [1023, 1024, 1100])
def test_more_groups_than_the_table_sorts(G, rest):
    """Row tiles of 256 over more than 1024 groups (the rows behind the last one count as one)."""
    splits = [(i * 37) % 400 for i in range(G)]
    splits[5:8] = [0, 1, 700]
    splits[0] += max(0, 161 * G - sum(splits))
    print(f"table of {G} groups, {rest} rows behind", flush=True)
    M, N, K = sum(splits) + rest, 64, 72
    dt = torch.bfloat16
    x, dy, w = randn((M, K), dt, 1), randn((M, N), dt, 3), randn((G, N, K), dt, 2)
    m = torch.tensor(splits, dtype=torch.int32, device="cuda")
    y, dx = g.grouped_matmul_forward(x.cuda(), w.cuda(), m), g.grouped_matmul_dgrad(dy.cuda(), w.cuda(), m)
    sp, used = spans(splits, M)
    for i in sorted({0, 1, 5, 6, 7, 8, 511, 1000, 1022, G - 1}):
        a, b = sp[i]
        assert_close(y[a:b], *product(x[a:b], w[i].t()), K, f"y group {i}")
        assert_close(dx[a:b], *product(dy[a:b], w[i]), N, f"dx group {i}")
    assert not y[used:].any() and not dx[used:].any()
    # every row, by its sum over the columns: N terms of one rounding each, half a step 2^-8 of the term
    group = torch.repeat_interleave(torch.arange(G), torch.tensor(splits))
    want = (x[:used].double() * w.double().sum(1)[group]).sum(1)
    mag = (x[:used].double().abs() * w.double().abs().sum(1)[group]).sum(1)
    assert bool(((y[:used].cpu().double().sum(1) - want).abs() <= mag * (2.0 ** -8 * 1.01 + K * 2.0 ** -23)).all())


@pytest.mark.parametrize("splits", [[900, 900, 900, 900], [-5, 1000, 2 ** 31 - 1, 2 ** 31 - 1], [1500, -1, 300, 7], [0, 0, 2 ** 31 - 1, 0]])
@pytest.mark.parametrize("M,N,K", [(2048, 8200, 72), (2048, 72, 8200), (130, 72, 1024), (130, 1024, 72), (1200, 72, 64)])
def test_bad_splits_in_tables_and_parts(M, N, K, splits):
    """Negative splits and ones that pass M in the stream's table, in a contraction cut into parts and in
    weight gradients of both: clamped, flagged, nothing else touched."""
    print(f"bad splits {splits} of {M} x {N} x {K}", flush=True)
    total = sum(max(s, 0) for s in splits)
    want = (1 if min(splits) < 0 else 0) | (2 if total > M else 0) | (4 if total < M else 0)
    m = torch.tensor(splits, dtype=torch.int32, device="cuda")
    x, w, dy = (randn(s, torch.bfloat16, i).cuda() for i, s in enumerate(((M, K), (4, N, K), (M, N))))
    for layout, call, n, k in ((g.GEMM_FPROP, lambda ws: g.grouped_matmul_forward(x, w, m, ws=ws), N, K),
                               (g.GEMM_DGRAD, lambda ws: g.grouped_matmul_dgrad(dy, w, m, ws=ws), K, N),
                               (g.GEMM_WGRAD, lambda ws: g.grouped_matmul_wgrad(dy, x, m, ws=ws), N, K)):
        ws = torch.zeros(g.grouped_matmul_ws_bytes(layout, 4, M, n, k), dtype=torch.uint8, device="cuda")
        call(ws)
        assert g.read_device_flags(ws) == want, layout
    _grouped(splits, M, N, K, torch.bfloat16)


# M, K, N, R, L: shrink by 32 positions (16 waves a workgroup, or 8 above 64 ranks and past 512 tiles), expand by
# 64 and by 128, ranks above 32, aligned and not
TILES = {
    "64": (5000, 256, 2000, 64, 3), "64wide": (5000, 256, 6000, 64, 3), "128": (5000, 256, 2000, 128, 3),
    "128wide": (5000, 256, 6000, 128, 2), "64odd": (5000, 251, 1999, 64, 3), "60oddwide": (5000, 251, 5999, 60, 3),
    "100odd": (5000, 251, 1999, 100, 2), "128oddwide": (5000, 251, 5999, 128, 2), "16odd": (5000, 251, 1999, 16, 2),
    "many40": (17000, 64, 264, 40, 5), "many128odd": (17000, 61, 263, 128, 5), "many12odd": (17000, 61, 263, 12, 5),
}


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("name", list(TILES))
def test_adapters_by_large_tiles(name, dt):
    print(f"adapters {name} {dt}", flush=True)
    M, K, N, R, L = TILES[name]
    t = DTYPES[dt]
    d = {"base": randn((M, N), t, 1), "x": randn((M, K), t, 2), "a": randn((L, R, K), t, 3, K ** -0.5), "b": randn((L, N, R), t, 4),
         "dy": randn((M, N), t, 5), "ids": torch.from_numpy(np_ids(M, L, 6, 0.1)),
         "scales": 0.25 + torch.rand(L, generator=torch.Generator().manual_seed(7))}
    ref, got = _reference(d), _run(d)
    for k in ("y", "dx", "da", "db"):
        _close(got[k], ref[k], f"{name} {dt} {k}")
    none = d["ids"] < 0
    assert torch.equal(got["y"].cpu()[none], d["base"][none]) and not got["dx"].cpu()[none].any()


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("R", [12, 16, 28, 32, 60, 64, 100, 128])
@pytest.mark.parametrize("M,K,N", [(90, 72, 136), (90, 71, 135), (5000, 24, 2000), (5000, 23, 1999), (5000, 24, 6000),
                                   (5000, 23, 5999), (17000, 72, 64), (17000, 71, 63)])
def test_adapters_of_every_tile_and_alignment(M, K, N, R, dt):
    """Every kernel of the forward: tiles of 16 and 32 positions with 8 and 16 waves, of 16, 64 and 128, each
    group of ranks, rows and weights of whole 16-byte chunks or not."""
    print(f"adapters M={M} K={K} N={N} R={R} {dt}", flush=True)
    t, L = DTYPES[dt], 3
    d = {"base": randn((M, N), t, 1), "x": randn((M, K), t, 2), "a": randn((L, R, K), t, 3, K ** -0.5), "b": randn((L, N, R), t, 4),
         "dy": torch.zeros((M, N), dtype=t), "ids": torch.from_numpy(np_ids(M, L, 6, 0.1)), "scales": torch.tensor([0.5, 1.0, 1.75])}
    v = {k: e.cuda() for k, e in d.items()}
    y, _ = g.lora_forward(v["base"], v["x"], v["a"], v["b"], v["ids"], v["scales"])
    _close(y, _reference(d)["y"], f"{R} {dt}")


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("H", [4104, 4101])
def test_moves_past_the_cache(H, dt):
    """Rows in expert order of 135 MB: the non-temporal forms, with probabilities and dropped slots."""
    print(f"moves past the cache H={H} {dt}", flush=True)
    T, k, E = 5500, 3, 9
    t = DTYPES[dt]
    ids = torch.from_numpy(np.random.RandomState(1).randint(-1, E, size=(T, k)).astype(np.int32))
    plan = g.dispatch_plan(ids.cuda(), E)
    used = int(plan.m_splits.sum())
    gen = torch.Generator("cuda").manual_seed(2)
    x, dy = (torch.empty((T, H), dtype=t, device="cuda").normal_(generator=gen) for _ in range(2))
    v = torch.empty((T * k, H), dtype=t, device="cuda").normal_(generator=gen)
    probs = torch.rand((T, k), generator=gen, device="cuda")
    r = plan.rows.long()
    live = (r >= 0)
    xg = g.dispatch_forward(x, plan)
    assert torch.equal(xg[r[live]], x[:, None].expand(T, k, H)[live]) and not xg[used:].any()
    y, y1, dx = g.combine_forward(v, plan, probs), g.combine_forward(v, plan), g.dispatch_backward(v, plan)
    dv, dp = g.combine_backward(dy, v, plan, probs)
    assert not dv[used:].any() and torch.equal(y1, dx)
    for a in range(0, T, 500):
        s = slice(a, a + 500)
        pv = torch.where(live[s, :, None], v[r[s].clamp(min=0)].double(), 0.0)
        p = probs[s].double()[:, :, None]
        assert_close(y[s], (pv * p).sum(1).cpu(), (pv * p).abs().sum(1).cpu(), k, "combine")
        assert_close(y1[s], pv.sum(1).cpu(), pv.abs().sum(1).cpu(), k, "combine without probs")
        prod = pv * dy[s].double()[:, None]
        assert_close(dp[s], prod.sum(2).cpu(), prod.abs().sum(2).cpu(), H, "probs gradient")
        want = (dy[s].double()[:, None] * p)[live[s]]
        assert_close(dv[r[s][live[s]]], want.cpu(), want.abs().cpu(), 1, "combine gradient")
