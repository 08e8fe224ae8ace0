"""grouped_matmul_w4 against products in 64 bits with the weights that the codes stand for."""
import math

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_mxfp8_amd as g
from block_util import int4_values, nvfp4_values
from mm_util import DTYPES, assert_close, randn, spans

pytestmark = pytest.mark.gpu


def _int4(G, N, K, group, dtype, seed, zeros=True):
    gen = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, generator=gen)
    scales = ((0.5 + torch.rand((G, N, K // group), generator=gen)) / math.sqrt(K)).to(dtype)
    z = torch.randint(0, 16, (G, N, K // group), dtype=torch.uint8, generator=gen) if zeros else None
    return codes, scales, z


def _nvfp4(G, N, K, seed):
    gen = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, generator=gen)
    scales = torch.randint(0, 0x7F, (G, N, K // 16), dtype=torch.uint8, generator=gen)
    amax = (0.01 + torch.rand(G, generator=gen))
    return codes, scales, amax


def _handle(w, kind):
    dev = [t.cuda() if t is not None else None for t in w]
    if kind == "nvfp4":
        return g.QTensor(g.NVFP4_RHT, {"row_data": dev[0].reshape(-1), "row_scale": dev[1].reshape(-1), "amax_pre": dev[2]})
    return g.Int4Weights(*dev)


def _values(w, kind):
    return nvfp4_values(*w) if kind == "nvfp4" else int4_values(*w)


def _make(kind, G, N, K, dtype, seed=1):
    if kind == "nvfp4":
        return _nvfp4(G, N, K, seed)
    return _int4(G, N, K, int(kind), dtype, seed, zeros=seed % 2 == 1)


def _check(x, w, kind, splits, what="y", dev_x=None):
    M, K = x.shape
    values = _values(w, kind)
    y = g.grouped_matmul_w4(dev_x if dev_x is not None else x.cuda(), _handle(w, kind), torch.tensor(splits, dtype=torch.int32, device="cuda"))
    want = torch.zeros((M, values.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(want)
    ranges, used = spans(splits, M)
    for i, (a, b) in enumerate(ranges):
        want[a:b] = x[a:b].double() @ values[i].t()
        mag[a:b] = x[a:b].double().abs() @ values[i].abs().t()
    # K exact products, a scale for each group of them (NVFP4: the division at the end)
    assert_close(y, want, mag, 2 * K, what)
    assert not y[used:].any()
    return y


KINDS = ["32", "64", "128", "nvfp4"]


def _k(kind, K):
    step = 32 if kind == "nvfp4" else int(kind)
    return max(step, K // step * step)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits,M,N,K", [([1], 1, 1, 32), ([1], 1, 64, 128), ([3, 0, 2], 5, 17, 96), ([1, 16, 17], 34, 65, 160), ([0, 0], 4, 33, 256),
                                          ([40, 1, 0, 70], 115, 130, 544), ([9], 9, 200, 4096), ([2, 2, 2], 9, 48, 1056), ([64, 65], 129, 96, 384),
                                          ([5, -3, 900], 12, 40, 640), ([200], 200, 80, 288)])
def test_products(splits, M, N, K, kind, dt):
    K = _k(kind, K)
    print(f"w4 splits={splits} M={M} N={N} K={K} {kind} {dt}", flush=True)
    dtype = DTYPES[dt]
    for seed in (1, 2):
        w = _make(kind, len(splits), N, K, dtype, seed)
        _check(randn((M, K), dtype, 3), w, kind, splits)


# what the launcher takes: four column tiles a workgroup (more than 4 rows a group, 512 tiles or more); spans with one
# row tile (2048 tiles or more, K of 512 or more), with several (more than 16 rows a group); K whole spans, with whole
# chunks behind them, with a part of one; rows of scales that begin at every alignment
LARGE = {"columns": ([9, 0, 20], 31, 2005, 416), "columns_long": ([30], 30, 4999, 1100), "spans": ([5, 0, 16, 17], 40, 5001, 1024),
         "spans_tail": ([1, 0, 2, 30, 1], 36, 5003, 1190), "spans_one": ([3, 3, 3, 3, 3, 3], 21, 5010, 512),
         "rows": ([100, 3, 64], 170, 2901, 1190), "rows_whole": ([33, 200, 1], 240, 2900, 1024)}


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", list(LARGE))
def test_products_of_many_tiles(case, kind, dt):
    splits, M, N, K = LARGE[case]
    K = _k(kind, K)
    print(f"w4 large {case} splits={splits} M={M} N={N} K={K} {kind} {dt}", flush=True)
    for seed in (1, 2):
        w = _make(kind, len(splits), N, K, DTYPES[dt], seed)
        _check(randn((M, K), DTYPES[dt], 3), w, kind, splits)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [8, 60])
def test_rows_of_every_size_in_spans(rows, kind, dt):
    """Rows as large and as small as the type has them, large beside small within a span, subnormals, zeros; then
    rows that are not finite, which stay alone."""
    dtype = DTYPES[dt]
    splits = [rows, 0, 1, 2] if rows < 16 else [rows, 20]
    M, N, K = sum(splits), 6001 if rows < 16 else 4003, _k(kind, 1100)
    # weights of about 2^-12, so that sums of the largest rows stay in the type
    if kind == "nvfp4":
        w = list(_make(kind, len(splits), N, K, dtype))
        w[2] = w[2] * 2.0 ** -10
    else:
        w = list(_make(kind, len(splits), N, K, dtype))
        w[1] = (w[1].float() * 2.0 ** -9).to(dtype)
    x = randn((M, K), dtype, 3)
    f = torch.finfo(dtype)
    top = 2.0 ** 126 if dt == "bf16" else 2.0 ** 14
    x[0] = (x[0].float().clamp(-1.9, 1.9) * top).to(dtype)
    x[1] = (x[1].float() * f.tiny).to(dtype)
    x[2] = (x[2].float() * f.tiny * f.eps * 4).to(dtype)                      # subnormals
    x[3] = 0
    x[4] = (x[4].float() * torch.pow(2.0, torch.arange(K) % 40 - 30.0)).to(dtype)
    x[5, ::3] = top / 4
    x[6, 600:] = 0
    ref = _check(x, w, kind, splits)
    bad = x.clone()
    bad[4, 9], bad[5, 700], bad[6, 130] = math.nan, math.inf, -math.inf
    y = g.grouped_matmul_w4(bad.cuda(), _handle(w, kind), torch.tensor(splits, dtype=torch.int32, device="cuda"))
    keep = torch.tensor([i for i in range(M) if i not in (4, 5, 6)])
    assert torch.equal(y[keep], ref[keep]) and bool(torch.isnan(y[4]).all())
    for row, k, sign in ((5, 700, 1), (6, 130, -1)):
        v = _values(w, kind)[0, :, k]
        got = y[row].cpu().double()
        assert bool(torch.isnan(got[v == 0]).all()) and torch.equal(got[v != 0], sign * torch.sign(v[v != 0]) * math.inf)


@pytest.mark.parametrize("kind", KINDS)
def test_strides_and_a_given_output_in_spans(kind):
    for splits, M, N in (([3, 9, 1, 8], 30, 5009), ([60, 20], 90, 4005)):
        K = _k(kind, 1100)
        w = _make(kind, len(splits), N, K, torch.bfloat16)
        x = randn((M, K), torch.bfloat16, 3)
        ref = _check(x, w, kind, splits)
        m, used = torch.tensor(splits, dtype=torch.int32, device="cuda"), sum(splits)
        for pad, off in ((3, 1), (24, 8)):
            big = torch.full((M, K + pad), math.nan, dtype=torch.bfloat16, device="cuda")
            big[:, off:off + K] = x.cuda()
            out = torch.full((M, N + pad), 7.0, dtype=torch.bfloat16, device="cuda")
            g.grouped_matmul_w4(big[:, off:off + K], _handle(w, kind), m, out=out[:, off:off + N])
            assert torch.equal(out[:used, off:off + N], ref[:used])
            out[:used, off:off + N] = 7.0
            assert bool((out == 7.0).all())


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("kind", KINDS)
def test_every_element_is_at_its_place(kind, dt):
    """Rows of the identity read every weight back: exact, one element at a time."""
    dtype = DTYPES[dt]
    K = 256
    w = _make(kind, 1, 50, K, dtype)
    y = g.grouped_matmul_w4(torch.eye(K, dtype=dtype).cuda(), _handle(w, kind), torch.tensor([K], dtype=torch.int32, device="cuda"))
    want = _values(w, kind)[0].t()
    if kind == "nvfp4":
        # one fp32 division, then the rounding
        assert_close(y, want, want.abs(), 0, "values")
    else:
        assert torch.equal(y.cpu().double(), want.to(dtype).double())


@pytest.mark.parametrize("dt", list(DTYPES))
def test_every_code_under_every_scale(dt):
    """All sixteen codes with all zeros, and with all E4M3 scales that are numbers."""
    dtype = DTYPES[dt]
    codes = torch.tensor([i | (i << 4) for i in range(16)], dtype=torch.uint8)[None, :, None].expand(16, 16, 16).contiguous()
    zeros = torch.arange(16, dtype=torch.uint8)[:, None, None].expand(16, 16, 1).contiguous()
    w = (codes, torch.full((16, 16, 1), 0.5, dtype=dtype), zeros)
    x = torch.zeros((16, 32), dtype=dtype)
    x[:, 7] = 2.0
    y = g.grouped_matmul_w4(x.cuda(), _handle(w, "32"), torch.ones(16, dtype=torch.int32, device="cuda"))
    assert torch.equal(y.cpu().double(), (torch.arange(16)[None, :] - torch.arange(16)[:, None]).double())
    codes = torch.tensor([i | (i << 4) for i in range(16)], dtype=torch.uint8)[None, :, None].expand(127, 16, 16).contiguous()
    scales = torch.arange(127, dtype=torch.uint8)[:, None, None].expand(127, 16, 2).contiguous()
    w = (codes, scales, torch.full((127,), 2688.0))                   # S = 1
    x = torch.zeros((127, 32), dtype=dtype)
    x[:, 19] = 1.0
    y = g.grouped_matmul_w4(x.cuda(), _handle(w, "nvfp4"), torch.ones(127, dtype=torch.int32, device="cuda"))
    assert torch.equal(y.cpu().double(), nvfp4_values(*w)[:, :, 19])


@pytest.mark.parametrize("dt", list(DTYPES))
def test_quantized_weights_of_the_library(dt):
    """What weight_quantize makes with the NVFP4 recipe, stacked, as it stands."""
    if dt == "fp16":
        w16 = randn((3, 128, 256), torch.bfloat16, 5, 0.02)
    else:
        w16 = randn((3, 256, 384), torch.bfloat16, 5, 0.02)
    q = g.weight_quantize(w16.cuda(), g.recipe("nvfp4", 0x1234))
    E, N, K = w16.shape
    x = randn((7, K), DTYPES[dt], 6)
    y = g.grouped_matmul_w4(x.cuda(), q, torch.tensor([2, 4, 1], dtype=torch.int32, device="cuda"))
    values = nvfp4_values(q.bufs["row_data"].cpu().view(E, N, K // 2), q.bufs["row_scale"].cpu().view(E, N, K // 16), q.bufs["amax_pre"].cpu())
    # the values are the weights within the format's step: half of 2/6 of the block's largest at most, and 2^-4 of its scale
    assert float((values - w16.double()).abs().max()) <= 0.25 * float(w16.abs().max())
    at = torch.tensor([0, 0, 1, 1, 1, 1, 2])
    want = torch.stack([x[i].double() @ values[at[i]].t() for i in range(7)])
    mag = torch.stack([x[i].double().abs() @ values[at[i]].abs().t() for i in range(7)])
    assert_close(y, want, mag, 2 * K, "y")


@pytest.mark.parametrize("kind", KINDS)
def test_strided_rows_and_a_given_output(kind):
    K = _k(kind, 384)
    splits, M, N = [3, 20], 30, 70
    w = _make(kind, 2, N, K, torch.bfloat16)
    x = randn((M, K), torch.bfloat16, 3)
    ref = _check(x, w, kind, splits)
    m = torch.tensor(splits, dtype=torch.int32, device="cuda")
    for pad, off in ((8, 0), (3, 1), (24, 8)):
        big = torch.full((M, K + pad), math.nan, dtype=torch.bfloat16, device="cuda")
        big[:, off:off + K] = x.cuda()
        out = torch.full((M, N + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        y = g.grouped_matmul_w4(big[:, off:off + K], _handle(w, kind), m, out=out[:, off:off + N])
        assert torch.equal(y[:23], ref[:23])
        rest = out.clone()
        rest[:23, off:off + N] = 7.0
        assert bool((rest == 7.0).all())                              # rows behind the groups, columns beside: as they were
    assert torch.equal(g.grouped_matmul_w4(x.cuda().t().contiguous().t(), _handle(w, kind), m), ref)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", list(DTYPES))
def test_rows_that_are_not_finite_or_large_stay_alone(kind, dt):
    K = _k(kind, 256)
    dtype = DTYPES[dt]
    w = _make(kind, 1, 40, K, dtype)
    x = randn((20, K), dtype, 3)
    ref = _check(x, w, kind, [20])
    x[4, 9] = math.nan
    x[11, 100] = math.inf
    y = g.grouped_matmul_w4(x.cuda(), _handle(w, kind), torch.tensor([20], dtype=torch.int32, device="cuda"))
    rows = torch.tensor([i for i in range(20) if i not in (4, 11)])
    assert torch.equal(y[rows], ref[rows]) and bool(torch.isnan(y[4]).all())
    v = _values(w, kind)[0, :, 100]
    want = torch.where(v == 0, math.nan, torch.sign(v) * math.inf)
    got = y[11].cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[v != 0], want[v != 0])
    # one large element beside zeros: within range as long as the result is
    big = torch.zeros((1, K), dtype=dtype)
    big[0, 33] = torch.finfo(dtype).max / 64
    _check(big, w, kind, [1])


@pytest.mark.parametrize("dt", list(DTYPES))
def test_the_largest_rows(dt):
    """Products of the largest rows with the largest integers pass the type's range before the scale brings them back."""
    dtype = DTYPES[dt]
    big = torch.zeros((2, 256), dtype=dtype)
    big[0, 33] = big[1, 200] = torch.finfo(dtype).max
    codes = torch.full((1, 16, 128), 0xFF, dtype=torch.uint8)
    codes[:, ::2] = 0
    zeros = torch.zeros((1, 16, 8), dtype=torch.uint8)
    zeros[:, ::2] = 15
    _check(big, (codes, torch.full((1, 16, 8), 2.0 ** -6, dtype=dtype), zeros), "32", [2])
    scales = torch.full((1, 16, 16), 0x7E, dtype=torch.uint8)         # 448: the weights are +-0.5
    codes[:, ::4] = 0x77
    _check(big, (codes, scales, torch.full((1,), 0.5)), "nvfp4", [2])
    # weights as large and as small as bf16 has them
    x = randn((3, 256), dtype, 4)
    for amax in (1e38, 1e-30, 0.0) if dt == "bf16" else (1e3, 1e-3, 0.0):
        _check(x * (1e-3 if amax > 1 or amax == 0 else 1), (codes, scales, torch.full((1,), amax)), "nvfp4", [3])


def test_scales_that_are_not_finite_reach_their_column_only():
    codes, scales, zeros = _int4(1, 20, 128, 32, torch.bfloat16, 1)
    x = randn((3, 128), torch.bfloat16, 2)
    ref = _check(x, (codes, scales, zeros), "32", [3])
    scales[0, 6, 2] = math.nan
    y = g.grouped_matmul_w4(x.cuda(), _handle((codes, scales, zeros), "32"), torch.tensor([3], dtype=torch.int32, device="cuda"))
    cols = torch.tensor([i for i in range(20) if i != 6])
    assert torch.equal(y[:, cols], ref[:, cols]) and bool(torch.isnan(y[:, 6]).all())


def test_many_groups_and_random_splits():
    r = np.random.RandomState(3)
    for G, M in ((128, 64), (300, 500), (64, 509)):
        splits = r.multinomial(M - 3, np.full(G, 1.0 / G)).tolist()
        for kind, dtype in (("64", torch.bfloat16), ("nvfp4", torch.float16)):
            print(f"w4 groups G={G} M={M} {kind}", flush=True)
            w = _make(kind, G, 72, 192, dtype)
            _check(randn((M, 192), dtype, 4), w, kind, splits)


def test_outputs_over_what_is_read_and_codes_off_their_alignment_are_refused():
    codes, scales, zeros = (t.cuda() for t in _int4(2, 64, 64, 32, torch.bfloat16, 1))
    m = torch.tensor([2, 2], dtype=torch.int32, device="cuda")
    big = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    w = g.Int4Weights(codes, scales, zeros)
    with pytest.raises(ValueError, match="overlaps"):
        g.grouped_matmul_w4(big[:4], w, m, out=big[2:6])
    y = g.grouped_matmul_w4(big[:4], w, m, out=big[4:])
    assert not y.any()
    for off in (1, 8):
        room = torch.zeros(codes.numel() + 16, dtype=torch.uint8, device="cuda")
        shifted = room[off:off + codes.numel()].view(codes.shape)
        with pytest.raises(g.GmlpError, match="aligned"):
            g.grouped_matmul_w4(big[:4], g.Int4Weights(shifted, scales, zeros), m)
    with pytest.raises(ValueError, match="no gradient"):
        g.grouped_matmul_w4(big[:4].clone().requires_grad_(), w, m)
    with torch.no_grad():
        g.grouped_matmul_w4(big[:4].clone().requires_grad_(), w, m)


def test_no_rows_and_determinism():
    w = _handle(_make("32", 2, 24, 64, torch.bfloat16), "32")
    m = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert g.grouped_matmul_w4(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w, m).shape == (0, 24)
    w = _handle(_make("nvfp4", 4, 1000, 2048, torch.bfloat16), "nvfp4")
    x, m = randn((50, 2048), torch.bfloat16, 1).cuda(), torch.tensor([9, 1, 30, 10], dtype=torch.int32, device="cuda")
    ref = g.grouped_matmul_w4(x, w, m)
    for _ in range(5):
        assert torch.equal(ref, g.grouped_matmul_w4(x, w, m))


@pytest.mark.parametrize("kind", KINDS)
def test_one_group_short_of_the_rows(kind):
    """A dense layer's split size may say less than all rows, down to none."""
    w = _make(kind, 1, 50, 256, torch.bfloat16)
    x = randn((9, 256), torch.bfloat16, 3)
    for m in (9, 4, 0, -2, 100):
        _check(x, w, kind, [m])
        out = torch.full((9, 50), 7.0, dtype=torch.bfloat16, device="cuda")
        g.grouped_matmul_w4(x.cuda(), _handle(w, kind), torch.tensor([m], dtype=torch.int32, device="cuda"), out=out)
        assert bool((out[max(m, 0):] == 7.0).all()) and (m <= 0 or not bool((out[:m] == 7.0).all()))
    _check(randn((40, 256), torch.bfloat16, 3), w, kind, [17])


def test_graph_replays_and_two_streams():
    a, b = (_make("64", 6, 300, 1024, torch.bfloat16, s) for s in (1, 3))
    x = randn((33, 1024), torch.bfloat16, 5).cuda()
    live = [t.cuda() for t in a]
    m1, m2 = (torch.tensor(s, dtype=torch.int32, device="cuda") for s in ([3, 0, 20, 1, 9, 0], [33, 0, 0, 0, 0, 0]))
    m = m1.clone()

    def step():
        return g.grouped_matmul_w4(x, g.Int4Weights(*live), m)
    refs = []
    for w, s in ((a, m1), (b, m2)):
        for t, v in zip(live, w):
            t.copy_(v)
        m.copy_(s)
        refs.append(step().clone())
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(step())
    torch.cuda.synchronize()
    assert torch.equal(got[0], refs[1]) and torch.equal(got[1], refs[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for r in range(4):
        for t, v in zip(live, a if r % 2 == 0 else b):
            t.copy_(v)
        m.copy_(m1 if r % 2 == 0 else m2)
        out.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, refs[r % 2]), r
    del graph


def test_codes_past_four_gigabytes():
    """The last group's codes and scales lie behind 2^32 bytes."""
    G, N, K = 20, 16384, 32768                                        # 5.4 GB of codes
    free, _ = torch.cuda.mem_get_info()
    if free < 16 << 30:
        pytest.skip("needs 16 GB")
    codes = torch.zeros((G, N, K // 2), dtype=torch.uint8, device="cuda").fill_(0x88)
    codes[-1] = 0x9B
    scales = torch.ones((G, N, K // 128), dtype=torch.bfloat16, device="cuda")
    scales[-1, -5:] = 2.0
    x = torch.zeros((3, K), dtype=torch.bfloat16, device="cuda")
    x[:, -2:] = torch.tensor([[1.0, 0.0], [0.0, 1.0], [1.0, 1.0]])
    splits = [0] * G
    splits[-1] = 3
    y = g.grouped_matmul_w4(x, g.Int4Weights(codes, scales), torch.tensor(splits, dtype=torch.int32, device="cuda"))
    want = torch.tensor([3.0, 1.0, 4.0], dtype=torch.bfloat16, device="cuda")
    assert torch.equal(y[:, :-5], want[:, None].expand(3, N - 5)) and torch.equal(y[:, -5:], 2 * want[:, None].expand(3, 5))


def test_more_tiles_than_one_grid_row_holds():
    """Past 2^24 workgroups the grid is folded: 16-row tiles of 2^18 x 16 rows, 65 column tiles."""
    M, N, K = (1 << 22) + 5, 4100, 32
    free, _ = torch.cuda.mem_get_info()
    if free < 90 << 30:
        pytest.skip("needs 90 GB")
    codes = torch.full((1, N, K // 2), 0x99, dtype=torch.uint8, device="cuda")
    scales = torch.ones((1, N, 1), dtype=torch.float16, device="cuda")
    x = torch.zeros((M, K), dtype=torch.float16, device="cuda")
    x[:, 3] = (torch.arange(M, device="cuda") % 97).to(torch.float16)
    y = g.grouped_matmul_w4(x, g.Int4Weights(codes, scales), torch.tensor([M], dtype=torch.int32, device="cuda"))
    assert torch.equal(y.amin(1), x[:, 3]) and torch.equal(y.amax(1), x[:, 3])


def _in_spans(kind, seed, K=1190, rows=16, N=16400):
    """bf16 rows of one tile over columns enough to fill the device: x, weights that are 0 at every 64th element of K, K."""
    K = _k(kind, K)
    w = _make(kind, 1, N, K, torch.bfloat16, 2)                        # integers without zeros: 8 is 0
    w[0].view(N, K // 2)[:, ::32] = 0x08 if kind != "nvfp4" else 0x00
    w[0].view(N, K // 2)[:, ::32] |= 0x90
    return randn((rows, K), torch.bfloat16, seed), w, K


@pytest.mark.parametrize("kind", KINDS)
def test_elements_beside_far_larger_ones_keep_their_bits(kind):
    """The row's largest elements meet weights of 0, so that every bit of the others is seen: from 2^-24 to 2^-84 of the
    largest, within one span, in the last part of K, alone and among ordinary elements."""
    x, w, K = _in_spans(kind, 3)
    ordinary = x.clone()
    for r in range(16):
        small = torch.zeros(K) if r % 2 else x[r].float() * 2.0 ** -(24 + 4 * r)
        small[130 + r] = (1 + 127 / 128) * 2.0 ** -(24 + 4 * r)
        small[K - 3] = (1 + 3 / 128) * 2.0 ** -(24 + 4 * r)
        if r != 6:
            small[700 + r] = -(1 + 65 / 128) * 2.0 ** -(24 + 4 * r)
        small[::64] = 0
        if r != 6:
            small[64::512] = 1.0
        small[960 if kind == "128" else 1088] = -1.5
        x[r] = small.to(torch.bfloat16)
    print(f"w4 spread {kind}", flush=True)
    _check(x, w, kind, [16])
    # rows are by themselves: the same beside others
    m = torch.tensor([16], dtype=torch.int32, device="cuda")
    mixed = torch.where((torch.arange(16) % 3 == 0)[:, None], x, ordinary)
    ref = [g.grouped_matmul_w4(t.cuda(), _handle(w, kind), m) for t in (x, ordinary)]
    y = g.grouped_matmul_w4(mixed.cuda(), _handle(w, kind), m)
    for r in range(16):
        assert torch.equal(y[r], ref[0 if r % 3 == 0 else 1][r]), r


def test_rows_and_nvfp4_weights_at_opposite_ends():
    """Rows and global scales whose powers of two together leave fp32 while the result does not: tiny rows by tiny
    weights, huge rows by huge weights that are 0, tiny rows by huge weights."""
    x, w, K = _in_spans("nvfp4", 4)
    for p in range(16):
        x[p] = (x[p].float().clamp(-1.9, 1.9) * 2.0 ** -(64 + p)).to(torch.bfloat16)
    x[13] = 0
    _check(x, (w[0], w[1], torch.full((1,), 2.0 ** -48)), "nvfp4", [16])
    huge = torch.full((1,), 3e38)
    x, w, K = _in_spans("nvfp4", 5)
    w[0][:, ::2] = 0                                                  # columns of zeros
    for p in range(16):
        x[p] = (x[p].float().clamp(-1.9, 1.9) * 2.0 ** -(17 + 7 * p)).to(torch.bfloat16)
    _check(x, (w[0], w[1], huge), "nvfp4", [16])
    x[3] = (x[3].float() * 2.0 ** 38 * 2.0 ** 100).to(torch.bfloat16)
    y = g.grouped_matmul_w4(x.cuda(), _handle((w[0], w[1], huge), "nvfp4"), torch.tensor([16], dtype=torch.int32, device="cuda"))
    assert not y[:, ::2].any()                                        # (the others are past the largest number)


def test_quantized_weights_say_what_they_are():
    rec = g.recipe("nvfp4", 0x1234)
    w16 = randn((2, 128, 256), torch.bfloat16, 5, 0.02).cuda()
    m = torch.tensor([2, 2], dtype=torch.int32, device="cuda")
    for w in (w16, list(w16)):
        q = g.weight_quantize(w, rec)
        assert q.shape == (2, 128, 256) and g.weight_quantize(w, rec, out=q).shape == (2, 128, 256)
        assert g.grouped_matmul_w4(randn((4, 256), torch.bfloat16, 6).cuda(), q, m).shape == (4, 128)
        with pytest.raises(ValueError, match="^w:"):
            g.grouped_matmul_w4(randn((4, 128), torch.bfloat16, 6).cuda(), q, m)
    out = g.alloc_grouped_q(rec, 256, 256, 2)
    out.shape = (2, 128, 256)
    assert g.group_quantize(w16.view(256, 256), torch.tensor([128, 128], dtype=torch.int32, device="cuda"), rec, out=out).shape is None


def _folds(blocks, threads):
    """A launch's threads along x are counted in 32 bits, in whole rounds over eight XCDs."""
    return blocks > (2 ** 32 - 1) // threads // 8 * 8


@pytest.mark.parametrize("kernel", ["split", "spans"])
def test_grids_of_more_than_2_32_threads(kernel):
    """Both kernels with their grids folded.  Split K, four column tiles a workgroup (more than 4 rows, K of 480: four waves);
    spans of two row tiles (more than 16 rows, groups of 32: eight waves).  The spans of one row tile share their code
    for the block's number, and would fold only past 130 GB of weights."""
    M, N, K, row_tile, columns, threads = {"split": ((1 << 22) + 5, 4100, 480, 16, 64, 256),
                                           "spans": ((1 << 21) + 33, 16385, 512, 32, 128, 512)}[kernel]
    assert _folds(-(-M // row_tile) * -(-N // columns), threads)
    free, _ = torch.cuda.mem_get_info()
    if free < 90 << 30:
        pytest.skip("needs 90 GB")
    print(f"w4 folded {kernel}", flush=True)
    codes = torch.full((1, N, K // 2), 0x99, dtype=torch.uint8, device="cuda")
    codes[0, N - 3] = 0xAA                                              # a column of twos
    scales = torch.ones((1, N, K // 32), dtype=torch.float16, device="cuda")
    x = torch.zeros((M, K), dtype=torch.float16, device="cuda")
    x[:, 3] = (torch.arange(M, device="cuda") % 97).to(torch.float16)
    x[:, K - 1] = (torch.arange(M, device="cuda") % 89).to(torch.float16)
    y = g.grouped_matmul_w4(x, g.Int4Weights(codes, scales), torch.tensor([M], dtype=torch.int32, device="cuda"))
    want = x[:, 3] + x[:, K - 1]
    assert torch.equal(y[:, N - 3], 2 * want)
    y[:, N - 3] = want
    assert torch.equal(y.amin(1), want) and torch.equal(y.amax(1), want)
