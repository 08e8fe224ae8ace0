"""The bf16 / fp16 operators beside the quantized grouped MLP, as workloads that can be timed.

Three families, each computed in plain torch (own = False) or by this package's kernels (own = True):

  gmm    products grouped by expert with ragged sizes: y = x w[g]^T, and in training dx = dy w[g]
         and dw[g] = dy_g^T x_g
  lora   low-rank adapters of many requests beside a shared projection: y = base + s b (a x) with the
         adapter chosen by each row, and in training dx, da, db
  moe    tokens brought into expert order and back: the order itself, the gather (dispatch), the
         weighted sum over a token's experts (combine), and in training their gradients

A case is a dict of plain values; see listed() for what each stands for.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the smallest product: two experts of a toy model, where the launch is all there is
        dict(name="gmm_tiny", op="gmm", dtype="bf16", train=False, G=2, M=192, N=256, K=128, skew="equal"),
        # decoding 8 tokens at top-8 over 128 experts of a large layer: the read of the experts' weights
        dict(name="gmm_decode", op="gmm", dtype="bf16", train=False, G=128, M=64, N=4096, K=7168, skew="multinomial"),
        # serving a mixed batch with Zipf routing over 64 experts, some of them empty
        dict(name="gmm_serve", op="gmm", dtype="fp16", train=False, G=64, M=6144, N=2816, K=2048, skew="zipf"),
        # sizes that no tile divides: odd rows, columns and contraction, forward and gradients
        dict(name="gmm_odd", op="gmm", dtype="fp16", train=True, G=5, M=1003, N=1001, K=333, skew="dirichlet"),
        # a training step's second projection, eight near-equal experts
        dict(name="gmm_train", op="gmm", dtype="bf16", train=True, G=8, M=32768, N=4096, K=1536, skew="multinomial"),
        # a training step's first projection at 128 experts with uneven counts: the largest products
        dict(name="gmm_train_large", op="gmm", dtype="bf16", train=True, G=128, M=65536, N=4096, K=7168,
             skew="dirichlet"),
        # decoding 32 requests, one token each, over 16 adapters of rank 16
        dict(name="lora_decode", op="lora", dtype="bf16", train=False, M=32, K=4096, N=4096, R=16, L=16, spread=32),
        # prefill of two dozen requests of uneven length, rank 64, some without an adapter
        dict(name="lora_prefill", op="lora", dtype="fp16", train=False, M=6001, K=7168, N=4096, R=64, L=12, spread=24),
        # training eight adapters at once on packed sequences
        dict(name="lora_train", op="lora", dtype="bf16", train=True, M=16384, K=4096, N=4096, R=16, L=8, spread=32),
        # routing 8 tokens of a decode step
        dict(name="moe_decode", op="moe", dtype="bf16", train=False, T=8, k=8, E=128, H=7168),
        # routing a prefill with top-6 over 64 experts
        dict(name="moe_prefill", op="moe", dtype="fp16", train=False, T=2049, k=6, E=64, H=2048),
        # routing a training step's tokens, with the gradients of both directions
        dict(name="moe_train", op="moe", dtype="bf16", train=True, T=8192, k=8, E=128, H=7168),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A feature size: mostly a multiple of 8, as hidden sizes are, sometimes any number."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.25 else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["gmm", "gmm", "lora", "moe"])
    dtype = rng.choice(["bf16", "fp16"])
    train = rng.random() < 0.5
    while True:
        if op == "gmm":
            c = dict(op=op, dtype=dtype, train=train, G=_log(rng, 1, 128), M=_log(rng, 1, 65536),
                     N=_size(rng, 64, 8192), K=_size(rng, 64, 8192),
                     skew=rng.choice(["equal", "multinomial", "zipf", "dirichlet"]))
            fits = (c["M"] * c["N"] * c["K"] <= 65536 * 4096 * 7168 and c["G"] * c["N"] * c["K"] <= 128 * 4096 * 7168)
        elif op == "lora":
            c = dict(op=op, dtype=dtype, train=train, M=_log(rng, 1, 16384), K=_size(rng, 256, 8192),
                     N=_size(rng, 256, 8192), R=rng.choice([4, 8, 16, 24, 32, 64, 128]), L=_log(rng, 1, 64),
                     spread=_log(rng, 1, 64))
            fits = True
        else:
            c = dict(op=op, dtype=dtype, train=train, T=_log(rng, 1, 8192), k=rng.randint(1, 8),
                     E=_log(rng, 8, 256), H=_size(rng, 256, 7168))
            fits = True
        if fits:
            return c


def _splits(c, r):
    G, M = c["G"], c["M"]
    if c["skew"] == "equal":
        s = np.full(G, M // G)
        s[: M - int(s.sum())] += 1
    elif c["skew"] == "multinomial":
        s = r.multinomial(M, np.full(G, 1.0 / G))
    elif c["skew"] == "dirichlet":
        s = r.multinomial(M, r.dirichlet(np.full(G, 0.5)))
    else:
        p = 1.0 / (1.0 + r.permutation(G)) ** 1.2
        p[r.permutation(G)[: G // 16]] = 0.0
        s = r.multinomial(M, p / p.sum())
    return [int(v) for v in s]


def _randn(gen, shape, std, dt):
    t = torch.empty(shape, dtype=dt, device="cuda")
    return t.normal_(0.0, std, generator=gen)


def prepare(case, seed):
    r = np.random.RandomState(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    st = dict(case)
    if case["op"] == "gmm":
        G, M, N, K = case["G"], case["M"], case["N"], case["K"]
        st["host_splits"] = _splits(case, r)
        st["m_splits"] = torch.tensor(st["host_splits"], dtype=torch.int32, device="cuda")
        st["x"] = _randn(gen, (M, K), 1.0, dt)
        st["w"] = _randn(gen, (G, N, K), 1.0 / math.sqrt(K), dt)
        if case["train"]:
            st["dy"] = _randn(gen, (M, N), 1.0, dt)
    elif case["op"] == "lora":
        M, N, K, R, L = case["M"], case["N"], case["K"], case["R"], case["L"]
        # requests are runs of rows; about one in ten has no adapter
        cuts = np.sort(r.randint(0, M + 1, size=min(case["spread"], M) - 1)) if M > 1 else np.zeros(0, int)
        if M <= case["spread"]:
            cuts = np.arange(1, M)
        lens = np.diff(np.concatenate([[0], cuts, [M]]))
        ids = np.concatenate([np.full(n, -1 if r.rand() < 0.1 else r.randint(L), dtype=np.int32) for n in lens])
        st["ids"] = torch.from_numpy(ids.astype(np.int32)).cuda()
        st["rows"] = [(a, torch.from_numpy(np.flatnonzero(ids == a)).cuda()) for a in range(L) if (ids == a).any()]
        st["base"] = _randn(gen, (M, N), 1.0, dt)
        st["x"] = _randn(gen, (M, K), 1.0, dt)
        st["a"] = _randn(gen, (L, R, K), 1.0 / math.sqrt(K), dt)
        st["b"] = _randn(gen, (L, N, R), 1.0 / math.sqrt(R), dt)
        st["scales"] = torch.from_numpy((0.5 + 1.5 * r.rand(L)).astype(np.float32)).cuda()
        if case["train"]:
            st["dy"] = _randn(gen, (M, N), 1.0, dt)
    else:
        T, k, E, H = case["T"], case["k"], case["E"], case["H"]
        score = torch.rand((T, E), generator=gen, device="cuda") + 0.3 * torch.rand((1, E), generator=gen, device="cuda")
        top, idx = score.topk(min(k, E), dim=1)
        st["k"] = int(idx.shape[1])
        st["experts"] = idx.to(torch.int32).contiguous()
        st["probs"] = torch.softmax(top, dim=1).contiguous()
        st["x"] = _randn(gen, (T, H), 1.0, dt)
        st["v"] = _randn(gen, (T * st["k"], H), 1.0, dt)       # the experts' outputs, in expert order
        if case["train"]:
            st["dy"] = _randn(gen, (T, H), 1.0, dt)
            st["dxg"] = _randn(gen, (T * st["k"], H), 1.0, dt)
    return st


# ------------------------------------------------------------------------------------ plain forms
def _gmm_plain(s):
    x, w, dt = s["x"], s["w"], s["x"].dtype
    y = torch.zeros((s["M"], s["N"]), dtype=dt, device=x.device)
    dx = torch.zeros_like(x) if s["train"] else None
    dw = torch.zeros_like(w) if s["train"] else None
    r0 = 0
    for g, m in enumerate(s["host_splits"]):
        if m == 0:
            continue
        xg, wg = x[r0:r0 + m].float(), w[g].float()
        y[r0:r0 + m] = (xg @ wg.t()).to(dt)
        if s["train"]:
            dyg = s["dy"][r0:r0 + m].float()
            dx[r0:r0 + m] = (dyg @ wg).to(dt)
            dw[g] = (dyg.t() @ xg).to(dt)
        r0 += m
    return {"y": y, "dx": dx, "dw": dw} if s["train"] else {"y": y}


def _lora_plain(s):
    x, a, b, dt = s["x"], s["a"], s["b"], s["x"].dtype
    y = s["base"].clone()
    out = {"y": y}
    if s["train"]:
        out["dx"], out["da"], out["db"] = torch.zeros_like(x), torch.zeros_like(a), torch.zeros_like(b)
    for l, rows in s["rows"]:
        xl, al, bl, sc = x[rows].float(), a[l].float(), b[l].float(), s["scales"][l]
        u = xl @ al.t()
        y[rows] = (s["base"][rows].float() + sc * (u @ bl.t())).to(dt)
        if s["train"]:
            dyl = s["dy"][rows].float()
            du = sc * (dyl @ bl)
            out["dx"][rows] = (du @ al).to(dt)
            out["da"][l] = (du.t() @ xl).to(dt)
            out["db"][l] = (sc * (dyl.t() @ u)).to(dt)
    return out


def _moe_plain(s):
    T, k, E, H, dt = s["T"], s["k"], s["E"], s["H"], s["x"].dtype
    flat = s["experts"].reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    rows = torch.empty_like(order)
    rows[order] = torch.arange(T * k, device=order.device)
    m_splits = (flat[None, :] == torch.arange(E, device=flat.device)[:, None]).sum(1)
    out = {"m_splits": m_splits.to(torch.int32), "rows": rows.view(T, k).to(torch.int32)}
    out["xg"] = s["x"][order // k]
    picked = s["v"][rows].view(T, k, H)
    p = s["probs"]
    out["y"] = (picked.float() * p[:, :, None]).sum(1).to(dt)
    if s["train"]:
        out["dx"] = s["dxg"][rows].view(T, k, H).float().sum(1).to(dt)
        dyf = s["dy"].float()
        dv = (dyf[order // k] * p.reshape(-1)[order][:, None]).to(dt)
        out["dv"] = dv
        out["dp"] = (picked.float() * dyf[:, None, :]).sum(2)
    return out


# ------------------------------------------------------------------------------------ this package's
def _own(s):
    import nvfp4_block_scaled_mxfp8_amd as gmlp
    if s["op"] == "gmm":
        y = gmlp.grouped_matmul_forward(s["x"], s["w"], s["m_splits"])
        if not s["train"]:
            return {"y": y}
        dx = gmlp.grouped_matmul_dgrad(s["dy"], s["w"], s["m_splits"])
        dw = gmlp.grouped_matmul_wgrad(s["dy"], s["x"], s["m_splits"])
        return {"y": y, "dx": dx, "dw": dw}
    if s["op"] == "lora":
        if not s["train"]:
            return {"y": gmlp.lora_forward(s["base"], s["x"], s["a"], s["b"], s["ids"], s["scales"])[0]}
        y, ctx = gmlp.lora_forward(s["base"], s["x"], s["a"], s["b"], s["ids"], s["scales"])
        g = gmlp.lora_backward(s["dy"], s["x"], s["a"], s["b"], ctx)
        return {"y": y, "dx": g["dx"], "da": g["da"], "db": g["db"]}
    plan = gmlp.dispatch_plan(s["experts"], s["E"])
    out = {"m_splits": plan.m_splits, "rows": plan.rows, "xg": gmlp.dispatch_forward(s["x"], plan),
           "y": gmlp.combine_forward(s["v"], plan, s["probs"])}
    if s["train"]:
        out["dx"] = gmlp.dispatch_backward(s["dxg"], plan)
        out["dv"], out["dp"] = gmlp.combine_backward(s["dy"], s["v"], plan, s["probs"])
    return out


def run(state):
    if own:
        return _own(state)
    return {"gmm": _gmm_plain, "lora": _lora_plain, "moe": _moe_plain}[state["op"]](state)


# ------------------------------------------------------------------------------------ what a pass needs
def work(case):
    if case["op"] == "gmm":
        G, M, N, K = case["G"], case["M"], case["N"], case["K"]
        # with few rows only the weights of the experts that have some are read; a uniform draw of M rows
        # leaves this many experts with one or more
        act = min(G, M) if case["skew"] == "equal" else G * (1.0 - (1.0 - 1.0 / G) ** M)
        one = 2.0 * M * N * K
        if not case["train"]:
            return {"bytes": 2 * (M * K + act * N * K + M * N), "flops": one}
        return {"bytes": 2 * (2 * M * K + 2 * M * N + act * N * K + G * N * K), "flops": 3 * one}
    if case["op"] == "lora":
        M, N, K, R, L = case["M"], case["N"], case["K"], case["R"], case["L"]
        act = min(L, M, case["spread"])
        ab = act * R * (K + N)
        fwd = 2 * (M * K + 2 * M * N + ab)
        if not case["train"]:
            return {"bytes": fwd, "flops": 2.0 * M * R * (K + N)}
        # x is read once for the forward's a x; its other reads and dy's are the backward's
        return {"bytes": fwd + 2 * (M * N + 2 * M * K + ab + L * R * (K + N)), "flops": 6.0 * M * R * (K + N)}
    T, H = case["T"], case["H"]
    k = min(case["k"], case["E"])
    b = 2 * H * (T + T * k) + 2 * H * (T * k + T) + 4 * T * k * 3 + 4 * case["E"]
    f = 2.0 * T * k * H
    if case["train"]:
        b += 2 * H * (T * k + T) + 2 * H * (T + 2 * T * k) + 4 * T * k * 2
        f += 4.0 * T * k * H
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------------------ from the definition
def exact(case, seed):
    """run()'s outputs in 64 bits, written from the definitions."""
    if case["op"] == "gmm" and case["train"] and case["G"] * case["N"] * case["K"] > 2 ** 29:
        return None                                            # tens of GB of 64-bit gradients
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "gmm":
        ends = np.cumsum(s["host_splits"])
        y = torch.zeros((s["M"], s["N"]), dtype=f, device="cuda")
        dx = torch.zeros((s["M"], s["K"]), dtype=f, device="cuda") if s["train"] else None
        dw = torch.zeros(s["w"].shape, dtype=f, device="cuda") if s["train"] else None
        for g in range(s["G"]):
            rows = slice(int(ends[g]) - s["host_splits"][g], int(ends[g]))
            if rows.start == rows.stop:
                continue
            wt = s["w"][g].to(f).t().contiguous()
            torch.matmul(s["x"][rows].to(f), wt, out=y[rows])
            if s["train"]:
                d = s["dy"][rows].to(f)
                torch.matmul(d, wt.t(), out=dx[rows])
                torch.matmul(d.t(), s["x"][rows].to(f), out=dw[g])
        return {"y": y, "dx": dx, "dw": dw} if s["train"] else {"y": y}
    if case["op"] == "lora":
        ids = s["ids"].long()
        y = s["base"].to(f)
        res = {"y": y}
        if s["train"]:
            res["dx"] = torch.zeros(s["x"].shape, dtype=f, device="cuda")
            res["da"] = torch.zeros(s["a"].shape, dtype=f, device="cuda")
            res["db"] = torch.zeros(s["b"].shape, dtype=f, device="cuda")
        for l in range(s["L"]):
            m = (ids == l).nonzero().flatten()
            if m.numel() == 0:
                continue
            delta = s["scales"][l].to(f) * (s["b"][l].to(f) @ s["a"][l].to(f))      # the adapter as one [N, K] matrix
            xm = s["x"][m].to(f)
            y[m] += xm @ delta.t()
            if s["train"]:
                d = s["dy"][m].to(f)
                res["dx"][m] = d @ delta
                outer = s["scales"][l].to(f) * (d.t() @ xm)                          # the gradient of that matrix
                res["da"][l] = s["b"][l].to(f).t() @ outer
                res["db"][l] = outer @ s["a"][l].to(f).t()
        return res
    ids = s["experts"].cpu().numpy()
    T, k = ids.shape
    rows = np.empty((T, k), dtype=np.int32)
    rank = np.argsort(ids.reshape(-1) * (T * k) + np.arange(T * k), kind="quicksort")
    rows.reshape(-1)[rank] = np.arange(T * k)
    res = {"m_splits": np.bincount(ids.reshape(-1), minlength=s["E"]).astype(np.int32), "rows": rows}
    R = torch.from_numpy(rows.astype(np.int64)).cuda()
    xg = torch.empty((T * k, s["H"]), dtype=f, device="cuda")
    y = torch.zeros((T, s["H"]), dtype=f, device="cuda")
    for j in range(k):
        xg[R[:, j]] = s["x"].to(f)
        y += s["probs"][:, j:j + 1].to(f) * s["v"][R[:, j]].to(f)
    res["xg"], res["y"] = xg, y
    if s["train"]:
        dx = torch.zeros((T, s["H"]), dtype=f, device="cuda")
        dv = torch.empty((T * k, s["H"]), dtype=f, device="cuda")
        dp = torch.empty((T, k), dtype=f, device="cuda")
        for j in range(k):
            dx += s["dxg"][R[:, j]].to(f)
            dv[R[:, j]] = s["probs"][:, j:j + 1].to(f) * s["dy"].to(f)
            dp[:, j] = (s["dy"].to(f) * s["v"][R[:, j]].to(f)).sum(1)
        res["dx"], res["dv"], res["dp"] = dx, dv, dp
    return res
