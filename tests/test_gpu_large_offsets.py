"""The 16-bit operators on tensors whose byte offsets pass 32 bits (several GB), checked at their far
ends, and calls that overlap on two streams."""
import pytest
import torch

import nvfp4_block_scaled_mxfp8_amd as g
from mm_util import half_step

pytestmark = pytest.mark.gpu


def _rows(M, C, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty((M, C), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)


def _near(got, want, mag, terms, what):
    """One rounding of the result, and each of `terms` additions off by a unit of a partial sum."""
    got, want = got.double(), want.double()
    tol = half_step(torch.bfloat16) * want.abs() * 1.01 + (terms + 8) * 2.0 ** -23 * mag.double() + 1e-30
    assert bool(((got - want).abs() <= tol).all()), what


@pytest.mark.parametrize("N", [16, 2048])
def test_grouped_products_past_4_gb(N):
    """x of 4.9 GB; a group of 2.9 GB as contraction (N = 2048: the stream's weight gradient)."""
    M, K = 300000, 8192
    splits = [120000, 0, 180000]
    print(f"products past 4 GB, N = {N}", flush=True)
    x, dy = _rows(M, K, 1), _rows(M, N, 2)
    w = _rows(3 * N, K, 3).view(3, N, K)
    m = torch.tensor(splits, dtype=torch.int32, device="cuda")
    y = g.grouped_matmul_forward(x, w, m)
    dx = g.grouped_matmul_dgrad(dy, w, m)
    for rows in (slice(0, 40), slice(119980, 120030), slice(299960, 300000)):
        for r in range(rows.start, rows.stop, 13):
            e = 0 if r < 120000 else 2
            xr, wr = x[r].double(), w[e, :16].double()
            _near(y[r, :16], wr @ xr, wr.abs() @ xr.abs(), K, ("y", r))
            dr, wc = dy[r].double(), w[e, :, -16:].double()
            _near(dx[r, -16:], dr @ wc, dr.abs() @ wc.abs(), N, ("dx", r))
    del y, dx
    dw = g.grouped_matmul_wgrad(dy, x, m)
    assert not dw[1].any()
    for e, (a, b) in ((0, (0, 120000)), (2, (120000, 300000))):
        want = torch.zeros((4, 64), dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(want)
        for s in range(a, b, 30000):
            d, xs = dy[s:s + 30000, -4:].double().t().contiguous(), x[s:s + 30000, -64:].double()
            want += d @ xs
            mag += d.abs() @ xs.abs()
        _near(dw[e, -4:, -64:], want, mag, b - a, ("dw", e))


def test_adapters_past_4_gb():
    M, K, N, R = 300000, 8192, 16, 4
    x, base, dy = _rows(M, K, 1), _rows(M, N, 2), _rows(M, N, 3)
    a, b = _rows(2 * R, K, 4).view(2, R, K) / 64, _rows(2 * N, R, 5).view(2, N, R)
    ids = (torch.arange(M, device="cuda") % 3 - 1).to(torch.int32)
    y, ctx = g.lora_forward(base, x, a, b, ids)
    r = g.lora_backward(dy, x, a, b, ctx)
    for m in (0, 1, 2, 262143, 262145, 299997, 299998, 299999):
        l = int(ids[m])
        if l < 0:
            assert torch.equal(y[m], base[m]) and not r["dx"][m].any()
            continue
        u, bl, al = a[l].double() @ x[m].double(), b[l].double(), a[l].double()
        mu = a[l].double().abs() @ x[m].double().abs()
        _near(y[m], base[m].double() + bl @ u, base[m].double().abs() + bl.abs() @ mu, K + 2 * R + 64, ("y", m))
        du = bl.t() @ dy[m].double()
        mdu = bl.abs().t() @ dy[m].double().abs()
        _near(r["dx"][m], du @ al, mdu @ al.abs(), N + 2 * R + 64, ("dx", m))
    want, mag = torch.zeros((R, 8), dtype=torch.float64, device="cuda"), torch.zeros((R, 8), dtype=torch.float64, device="cuda")
    rows = (ids == 1).nonzero().flatten()
    for s in rows.split(20000):
        du = dy[s].double() @ b[1].double()
        want += du.t().contiguous() @ x[s][:, -8:].double()
        mag += (dy[s].double().abs() @ b[1].double().abs()).t().contiguous() @ x[s][:, -8:].double().abs()
    _near(r["da"][1][:, -8:], want, mag, rows.numel() + 64, "da")


def test_dispatch_past_4_gb():
    T, k, E, H = 40000, 8, 16, 7168
    x = _rows(T, H, 1)
    experts = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    plan = g.dispatch_plan(experts, E)
    xg = g.dispatch_forward(x, plan)
    t = torch.tensor([0, 1, 19999, 39998, 39999], device="cuda")
    assert torch.equal(xg[plan.rows[t].long()], x[t][:, None, :].expand(-1, k, -1))
    assert torch.equal(xg[-1], x[(plan.rows == T * k - 1).nonzero()[0, 0]])
    y = g.combine_forward(xg, plan)
    assert torch.equal(y[t], (x[t].float() * k).to(torch.bfloat16))       # k equal terms: exact in fp32 (k = 8)


def test_calls_on_two_streams_at_once():
    """Two different calls of each operator in flight together: the bits of each alone."""
    def job(seed):
        x, dy = _rows(4096, 512, seed), _rows(4096, 768, seed + 1)
        w = _rows(4 * 768, 512, seed + 2).view(4, 768, 512)
        m = torch.tensor([1000, 0, 3000 - 90 * seed, 50], dtype=torch.int32, device="cuda")
        a, b = _rows(3 * 16, 512, seed + 3).view(3, 16, 512), _rows(3 * 768, 16, seed + 4).view(3, 768, 16)
        ids = (torch.arange(4096, device="cuda") * (seed + 3) % 4 - 1).to(torch.int32)
        experts = (torch.arange(8192, device="cuda") * 7919 % (5 + seed)).to(torch.int32).view(4096, 2)
        torch.cuda.synchronize()

        def run():
            y = g.grouped_matmul_forward(x, w, m)
            z, ctx = g.lora_forward(y, x, a, b, ids)
            r = g.lora_backward(dy, x, a, b, ctx)
            plan = g.dispatch_plan(experts, 16)
            xg = g.dispatch_forward(x, plan)
            return [y, z, g.grouped_matmul_dgrad(dy, w, m), g.grouped_matmul_wgrad(dy, x, m), r["dx"], r["da"], r["db"],
                    plan.rows, xg, g.combine_forward(xg, plan)]
        return run
    jobs = [job(1), job(9)]
    alone = [[t.clone() for t in j()] for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        out = [None, None]
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                out[i] = jobs[i]()
        torch.cuda.synchronize()
        for i in range(2):
            for j, (p, q) in enumerate(zip(alone[i], out[i])):
                assert torch.equal(p, q), (i, j)


def test_moves_of_more_tokens_than_one_row_of_blocks():
    """2^24 tokens and more: as many workgroups of 256 threads pass the 32 bits of a launch's threads along x."""
    T, H, E = (1 << 24) + 5, 8, 3
    print("moves of 2^24 + 5 short rows", flush=True)
    experts = (torch.arange(T, device="cuda") % 4).to(torch.int32).view(T, 1)         # expert 3: dropped
    plan = g.dispatch_plan(experts, E)
    used = int(plan.m_splits.sum())
    x = (torch.arange(T, device="cuda") % 251).to(torch.bfloat16)[:, None] + torch.arange(H, device="cuda").to(torch.bfloat16) * 0
    xg = g.dispatch_forward(x, plan)
    live = plan.rows[:, 0] >= 0
    assert torch.equal(xg[plan.rows[live, 0].long()], x[live]) and not xg[used:].any()
    _, dp = g.combine_backward(x, xg, plan, torch.ones((T, 1), device="cuda"), need_dv=False)
    assert torch.equal(dp[:, 0], torch.where(live, (x.float() * x.float()).sum(1), torch.zeros((), device="cuda")))
    del x, xg, dp
    H = 1032                                             # one token a workgroup in dispatch and combine too
    print("moves of 2^24 + 5 rows of 1032", flush=True)
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    x.copy_((torch.arange(T, device="cuda") % 251).to(torch.bfloat16)[:, None])
    x[:, -1] = (torch.arange(T, device="cuda") % 127).to(torch.bfloat16)
    xg = g.dispatch_forward(x, plan)
    for c in (0, 7, H - 9, H - 1):
        assert torch.equal(xg[plan.rows[live, 0].long(), c], x[live, c]) and not xg[used:, c].any()
    want = [torch.where(live, x[:, c], torch.zeros((), dtype=x.dtype, device="cuda")) for c in (0, 7, H - 9, H - 1)]
    g.combine_forward(xg, plan, out=x)
    for c, w in zip((0, 7, H - 9, H - 1), want):
        assert torch.equal(x[:, c], w)


def test_adapters_of_more_rows_than_one_row_of_blocks():
    """2^28 rows and more: their tiles of 32 by workgroups of 512 threads pass the 32 bits of a launch's
    threads along x.  Small integers, so every value is exact."""
    M, K, N, R, L = (1 << 28) + 37, 8, 8, 1, 2
    print("adapters of 2^28 + 37 short rows", flush=True)
    x = (torch.arange(M, device="cuda", dtype=torch.int32) % 13).to(torch.bfloat16)[:, None].expand(M, K).contiguous()
    ids = (torch.arange(M, device="cuda", dtype=torch.int32) % 3 - 1).to(torch.int32)
    a = torch.ones((L, R, K), dtype=torch.bfloat16, device="cuda")
    b = torch.arange(1, N + 1, device="cuda").to(torch.bfloat16).view(1, N, 1).expand(L, N, R).contiguous()
    y, ctx = g.lora_forward(None, x, a, b, ids)
    for c in (0, N - 1):                                  # 8 x (c + 1): at most 8 x 12 x 8 = 768, in steps of 8 (c + 1)
        want = torch.where(ids >= 0, x[:, 0].float() * (8 * (c + 1)), torch.zeros((), device="cuda")).to(torch.bfloat16)
        assert torch.equal(y[:, c], want), c
    y.fill_(1)
    dx = g.lora_backward(y, x, a, b, ctx, need_da=False, need_db=False)["dx"]
    want = torch.where(ids >= 0, torch.full((), float(sum(range(1, N + 1))), device="cuda"), torch.zeros((), device="cuda"))
    assert torch.equal(dx[:, 0], want.to(torch.bfloat16)) and torch.equal(dx[:, K - 1], want.to(torch.bfloat16))


def test_products_of_more_tiles_than_one_row_of_blocks():
    """4096 groups of one row and 2^19 + 128 columns: the tiles' workgroups of 256 threads pass the 32 bits of a
    launch's threads along x.  A contraction of one element, small integers: exact."""
    G, N = 4096, (1 << 19) + 128
    print("products of 2^24 + 4096 tiles", flush=True)
    m = torch.ones(G, dtype=torch.int32, device="cuda")
    x = (torch.arange(G, device="cuda") % 7 - 3).to(torch.bfloat16)[:, None].contiguous()
    w = ((torch.arange(G, device="cuda")[:, None] + torch.arange(N, device="cuda", dtype=torch.int32)) % 13).to(torch.bfloat16)
    want = x * w
    assert torch.equal(g.grouped_matmul_forward(x, w[:, :, None], m), want)
    assert torch.equal(g.grouped_matmul_dgrad(x, w[:, None, :], m), want)
    assert torch.equal(g.grouped_matmul_wgrad(w, x, m)[:, :, 0], want)
    assert torch.equal(g.grouped_matmul_wgrad(x, w, m)[:, 0], want)
