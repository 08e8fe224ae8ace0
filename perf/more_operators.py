"""The operators around the experts of a layer, as workloads that can be timed.

Three families, each in plain torch (own = False) or by this package's kernels (own = True):

  route  the experts of each token from the router's logits: softmax or sigmoid scores, a bias for balance,
         groups, top-k, weights; in training the gradient for the logits
  norm   the norms before and after a block, fused with its gate, the residual scale and the residual sum;
         in training all gradients
  w4     products grouped by expert with weights of 4 bits and scales by group, for few rows

A case is a dict of plain values; see listed() for what each stands for.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # routing 8 tokens of a decode step: a launch
        dict(name="route_decode", op="route", dtype="fp32", train=False, T=8, E=128, k=8, score="softmax", bias=False,
             groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0, pad=0),
        # a prefill of odd length, sigmoid scores with a bias for balance, four of eight groups, padding at the end
        dict(name="route_prefill_groups", op="route", dtype="fp32", train=False, T=2049, E=256, k=8, score="sigmoid",
             bias=True, groups=8, top_groups=4, group_best=2, renormalize=True, scale=2.5, pad=37),
        # a training step's routing of 8192 tokens, top-8 of 128, 16-bit logits, with the gradient
        dict(name="route_train", op="route", dtype="bf16", train=True, T=8192, E=128, k=8, score="softmax", bias=False,
             groups=1, top_groups=1, group_best=1, renormalize=False, scale=1.0, pad=0),
        # the largest: a long training batch over 256 experts with a bias
        dict(name="route_train_large", op="route", dtype="fp32", train=True, T=65536, E=256, k=8, score="sigmoid",
             bias=True, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0, pad=0),
        # between two blocks of a decode step of 8 tokens: the residual sum and the next block's norm
        dict(name="norm_decode", op="norm", dtype="bf16", train=False, T=8, H=7168, post=False, gate="none", scale=1.0,
             pre=True, wide=False),
        # a prefill with a norm behind the block as well and a gate by token
        dict(name="norm_prefill", op="norm", dtype="fp16", train=False, T=2049, H=2048, post=True, gate="token",
             scale=0.5, pre=True, wide=False),
        # odd sizes, a gate of every element, forward and gradients
        dict(name="norm_odd", op="norm", dtype="fp16", train=True, T=1003, H=1001, post=True, gate="full", scale=1.0,
             pre=True, wide=True),
        # a training step's 8192 tokens, both norms, a gate by channel, fp32 parameters
        dict(name="norm_train", op="norm", dtype="bf16", train=True, T=8192, H=7168, post=True, gate="channel",
             scale=0.25, pre=True, wide=True),
        # the smallest product: two experts of a toy model, where the launch is all there is
        dict(name="w4_tiny", op="w4", dtype="bf16", kind="int4", group=32, zeros=False, G=2, M=6, N=256, K=128,
             skew="equal"),
        # one token through one dense projection of a decode step
        dict(name="w4_token", op="w4", dtype="bf16", kind="int4", group=64, zeros=True, G=1, M=1, N=7168, K=4096,
             skew="equal"),
        # decoding 8 tokens at top-8 over 128 experts of a large layer, weights as the group quantizer leaves them
        dict(name="w4_decode", op="w4", dtype="bf16", kind="nvfp4", group=16, zeros=False, G=128, M=64, N=4096, K=7168,
             skew="multinomial"),
        # a serving batch with Zipf routing over 64 experts, some of them empty, odd columns
        dict(name="w4_serve", op="w4", dtype="fp16", kind="int4", group=128, zeros=True, G=64, M=509, N=2817, K=2048,
             skew="zipf"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A feature size: mostly a multiple of 8, as hidden sizes are, sometimes any number."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.25 else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["route", "norm", "w4"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = _log(rng, 4, 256) if groups == 1 else groups * _log(rng, 4, 256 // groups)
        top = rng.randint(1, groups)
        k = rng.randint(1, min(8, top * (E // groups)))
        T = _log(rng, 1, 65536)
        return dict(op=op, dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]), train=rng.random() < 0.5, T=T, E=E, k=k,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, top_groups=top,
                    group_best=rng.choice([1, 2]), renormalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    pad=rng.randint(0, T // 8))
    if op == "norm":
        while True:
            c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), train=rng.random() < 0.5, T=_log(rng, 1, 16384),
                     H=_size(rng, 256, 8192), post=rng.random() < 0.6,
                     gate=rng.choice(["none", "channel", "token", "full"]), scale=rng.choice([1.0, 0.25]),
                     pre=rng.random() < 0.8, wide=rng.random() < 0.5)
            if c["T"] * c["H"] * (2 if c["gate"] == "full" else 1) <= 8192 * 7168:
                return c
    while True:
        kind = rng.choice(["int4", "int4", "nvfp4"])
        group = 16 if kind == "nvfp4" else rng.choice([32, 64, 128])
        step = max(group, 32)
        c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), kind=kind, group=group,
                 zeros=kind == "int4" and rng.random() < 0.5, G=_log(rng, 1, 128), M=_log(rng, 1, 512),
                 N=32 * _log(rng, 2, 256) if kind == "nvfp4" else _size(rng, 64, 8192),
                 K=step * max(1, _log(rng, 128, 8192) // step), skew=rng.choice(["equal", "multinomial", "zipf"]))
        if c["G"] * c["N"] * c["K"] <= 128 * 4096 * 7168 and min(c["G"], c["M"]) * c["N"] * c["K"] <= 50 * 4096 * 7168:
            return c


def _splits(c, r):
    G, M = c["G"], c["M"]
    if c["skew"] == "equal":
        s = np.full(G, M // G)
        s[: M - int(s.sum())] += 1
    elif c["skew"] == "multinomial":
        s = r.multinomial(M, np.full(G, 1.0 / G))
    else:
        p = 1.0 / (1.0 + r.permutation(G)) ** 1.2
        p[r.permutation(G)[: G // 16]] = 0.0
        s = r.multinomial(M, p / p.sum())
    return [int(v) for v in s]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    st = dict(case)

    def randn(shape, std=1.0, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)

    def rand(shape):
        return torch.rand(shape, generator=gen, device="cuda")

    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # a router's logits: some experts are liked more by all tokens; rows of padding are masked whole
        logits = (1.5 * randn((T, E), 1.0, torch.float32) + 0.5 * randn((1, E), 1.0, torch.float32)).to(dt)
        if case["pad"]:
            logits[T - case["pad"]:] = -math.inf
        st["logits"] = logits
        st["bias_e"] = 0.2 * randn((E,), 1.0, torch.float32) if case["bias"] else None
        if case["train"]:
            st["dprobs"] = randn((T, k), 1.0, torch.float32)
    elif case["op"] == "norm":
        T, H = case["T"], case["H"]
        pt = torch.float32 if case["wide"] else dt
        # the residual stream has channels that are larger than the others
        st["x"] = (randn((T, H), 1.0, torch.float32) * torch.exp(0.7 * randn((1, H), 1.0, torch.float32))).to(dt)
        st["branch"] = randn((T, H), 0.5)
        st["w_post"] = (1.0 + randn((H,), 0.2, torch.float32)).to(pt) if case["post"] else None
        st["w_pre"] = (1.0 + randn((H,), 0.2, torch.float32)).to(pt) if case["pre"] else None
        shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[case["gate"]]
        st["g"] = None if shape is None else rand(shape).to(dt if case["gate"] == "full" else pt)
        if case["train"]:
            st["dy"] = randn((T, H))
            st["dh"] = randn((T, H)) if case["pre"] else None
    else:
        G, M, N, K = case["G"], case["M"], case["N"], case["K"]
        st["host_splits"] = _splits(case, np.random.RandomState(seed))
        st["m_splits"] = torch.tensor(st["host_splits"], dtype=torch.int32, device="cuda")
        st["x"] = randn((M, K))
        st["codes"] = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, generator=gen, device="cuda")
        n = K // case["group"]
        if case["kind"] == "nvfp4":
            # E4M3 block scales between 2 and 448, a global scale by expert as its largest weight sets it
            st["scales"] = torch.randint(0x40, 0x7F, (G, N, n), dtype=torch.uint8, generator=gen, device="cuda")
            st["amax"] = (4.0 + 2.0 * rand((G,))) / math.sqrt(K)
            st["zero"] = None
        else:
            st["scales"] = ((0.5 + rand((G, N, n))) / (4.0 * math.sqrt(K))).to(dt)
            st["zero"] = (torch.randint(5, 12, (G, N, n), dtype=torch.uint8, generator=gen, device="cuda")
                          if case["zeros"] else None)
    return st


# ------------------------------------------------------------------------------------ plain forms
def _route_plain(s):
    logits, k, E, T = s["logits"], s["k"], s["E"], s["T"]
    l32 = logits.float()
    live = l32 > -math.inf
    any_live = live.any(1, keepdim=True)
    top = torch.where(any_live, l32.max(1, keepdim=True).values, 0.0)

    def scores(l, m):
        if s["score"] == "sigmoid":
            return 1.0 / (1.0 + torch.exp(-l))
        e = torch.exp(l - m)
        return e / torch.where(any_live, e.sum(1, keepdim=True), 1.0)

    # what is compared: the logits where that is the order, 64 bits where sums are compared
    rank = l32
    wide = None
    if s["bias"] or (s["groups"] > 1 and s["group_best"] > 1):
        wide = scores(l32.double(), top.double())
        wide = torch.where(live, wide + s["bias_e"].double() if s["bias"] else wide, -math.inf)
    if s["bias"]:
        rank = wide
    if s["groups"] > 1:
        value = (rank if s["group_best"] == 1 else wide).view(T, s["groups"], -1)
        best = value.sort(dim=2, descending=True).values[:, :, : s["group_best"]]
        value = torch.where(best > -math.inf, best, 0.0).sum(2)
        value = torch.where(best[:, :, 0] > -math.inf, value, -math.inf)
        order = value.sort(dim=1, descending=True, stable=True).indices[:, : s["top_groups"]]
        allowed = torch.zeros((T, s["groups"]), dtype=torch.bool, device=rank.device).scatter_(1, order, True)
        rank = torch.where(allowed.repeat_interleave(E // s["groups"], 1), rank, -math.inf)
    value, idx = rank.sort(dim=1, descending=True, stable=True)
    idx, some = idx[:, :k], value[:, :k] > -math.inf
    if s["score"] == "softmax" and s["renormalize"]:
        chosen = l32.gather(1, idx)
        w = torch.exp(chosen - torch.where(some[:, :1], chosen.masked_fill(~some, -math.inf).max(1, keepdim=True).values, 0.0))
    else:
        w = scores(l32, top).gather(1, idx)
    w = torch.where(some, w, 0.0)
    if s["renormalize"]:
        w = w / torch.where(some[:, :1], w.sum(1, keepdim=True), 1.0)
    out = {"experts": torch.where(some, idx, -1).to(torch.int32), "probs": w * s["scale"]}
    if s["train"]:
        g = torch.where(some, s["dprobs"] * s["scale"], 0.0)
        dl = torch.zeros((T, E), device=rank.device)
        if s["renormalize"]:
            d = w * (g - (g * w).sum(1, keepdim=True))
            if s["score"] == "sigmoid":
                d = d / (1.0 + torch.exp(l32.gather(1, idx)))
            dl.scatter_(1, idx, torch.where(some, d, 0.0))
        elif s["score"] == "sigmoid":
            dl.scatter_(1, idx, torch.where(some, g * w * (1.0 - w), 0.0))
        else:
            p = scores(l32, top)
            dl.scatter_(1, idx, g)
            dl = torch.where(live, p * (dl - (g * w).sum(1, keepdim=True)), 0.0)
        out["dlogits"] = dl.to(logits.dtype)
    return out


_EPS = 1e-6


def _norm_plain(s):
    x, b, dt = s["x"].float(), s["branch"].float(), s["x"].dtype
    rb = torch.rsqrt((b * b).mean(1, keepdim=True) + _EPS)
    bhat = b * rb
    n = bhat * s["w_post"].float() if s["post"] else b
    gate = s["scale"] if s["g"] is None else s["scale"] * s["g"].float()
    y = x + gate * n
    out = {"y": y.to(dt)}
    if s["pre"]:
        ry = torch.rsqrt((y * y).mean(1, keepdim=True) + _EPS)
        yhat = y * ry
        out["h"] = (yhat * s["w_pre"].float()).to(dt)
    if s["train"]:
        d = s["dy"].float()
        if s["pre"]:
            dh = s["dh"].float()
            out["dw_pre"] = (dh * yhat).sum(0).to(s["w_pre"].dtype)
            dn = dh * s["w_pre"].float()
            d = d + ry * (dn - yhat * (dn * yhat).mean(1, keepdim=True))
        out["dx"] = d.to(dt)
        if s["g"] is not None:
            dg = s["scale"] * d * n
            dg = {"channel": lambda: dg.sum(0), "token": lambda: dg.sum(1, keepdim=True), "full": lambda: dg}[s["gate"]]()
            out["dgate"] = dg.to(s["g"].dtype)
        db = gate * d
        if s["post"]:
            out["dw_post"] = (db * bhat).sum(0).to(s["w_post"].dtype)
            dn = db * s["w_post"].float()
            db = rb * (dn - bhat * (dn * bhat).mean(1, keepdim=True))
        out["dbranch"] = db.to(dt)
    return out


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _w4_plain(s):
    x, dt = s["x"], s["x"].dtype
    N, K, group = s["N"], s["K"], s["group"]
    y = torch.zeros((s["M"], N), dtype=dt, device=x.device)
    values = torch.tensor(_E2M1, device=x.device)
    r0 = 0
    for g, m in enumerate(s["host_splits"]):
        if m == 0:
            continue
        c = s["codes"][g]
        c = torch.stack([c & 15, c >> 4], 2).view(N, K // group, group)
        if s["kind"] == "nvfp4":
            w = values[c.int()] * s["scales"][g].view(torch.float8_e4m3fn).float()[:, :, None]
            w = w / (2688.0 / s["amax"][g])
        else:
            zero = s["zero"][g].float()[:, :, None] if s["zeros"] else 8.0
            w = (c.float() - zero) * s["scales"][g].float()[:, :, None]
        y[r0:r0 + m] = (x[r0:r0 + m].float() @ w.view(N, K).t()).to(dt)
        r0 += m
    return {"y": y}


# ------------------------------------------------------------------------------------ this package's
def _own(s):
    import nvfp4_block_scaled_mxfp8_amd as gmlp
    if s["op"] == "route":
        experts, probs = gmlp.route_forward(s["logits"], s["k"], s["score"], bias=s["bias_e"], groups=s["groups"],
                                            top_groups=s["top_groups"], group_best=s["group_best"],
                                            renormalize=s["renormalize"], scale=s["scale"])
        out = {"experts": experts, "probs": probs}
        if s["train"]:
            out["dlogits"] = gmlp.route_backward(s["dprobs"], s["logits"], experts, s["score"],
                                                 renormalize=s["renormalize"], scale=s["scale"])
        return out
    if s["op"] == "norm":
        kw = dict(weight=s["w_pre"], branch_weight=s["w_post"], gate=s["g"], scale=s["scale"], eps=_EPS)
        y, h, stats = gmlp.residual_norm_forward(s["x"], s["branch"], **kw)
        out = {"y": y}
        if s["pre"]:
            out["h"] = h
        if s["train"]:
            g = gmlp.residual_norm_backward(s["dy"], s["dh"], s["x"], s["branch"], stats, **kw)
            out["dx"], out["dbranch"] = g["dx"], g["dbranch"]
            if s["pre"]:
                out["dw_pre"] = g["dweight"]
            if s["post"]:
                out["dw_post"] = g["dbranch_weight"]
            if s["g"] is not None:
                out["dgate"] = g["dgate"]
        return out
    if s["kind"] == "nvfp4":
        w = gmlp.QTensor(gmlp.NVFP4_RHT, {"row_data": s["codes"], "row_scale": s["scales"], "amax_pre": s["amax"]})
    else:
        w = gmlp.Int4Weights(s["codes"], s["scales"], s["zero"])
    return {"y": gmlp.grouped_matmul_w4(s["x"], w, s["m_splits"])}


def run(state):
    if own:
        return _own(state)
    return {"route": _route_plain, "norm": _norm_plain, "w4": _w4_plain}[state["op"]](state)


# ------------------------------------------------------------------------------------ what a pass needs
def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "fp32" else 2
        b, f = size * T * E + 8 * T * k + (4 * E if case["bias"] else 0), 4.0 * T * E + 4.0 * T * k
        if case["train"]:
            b += 2 * size * T * E + 8 * T * k
            f += 4.0 * T * E
        return {"bytes": b, "flops": f}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        wide = 4 if case["wide"] else 2
        params = wide * H * (case["post"] + case["pre"])
        gate = {"none": 0, "channel": wide * H, "token": wide * T, "full": 2 * T * H}[case["gate"]]
        b, f = 2 * T * H * (3 + case["pre"]) + params + gate, 10.0 * T * H
        if case["train"]:
            b += 2 * T * H * (5 + case["pre"]) + 2 * params + 2 * gate
            f += 20.0 * T * H
        return {"bytes": b, "flops": f}
    G, M, N, K = case["G"], case["M"], case["N"], case["K"]
    # the weights of the experts that have rows; a uniform draw of M rows leaves this many with one or more
    act = min(G, M) if case["skew"] == "equal" else G * (1.0 - (1.0 - 1.0 / G) ** M)
    scale = 1.0 if case["kind"] == "nvfp4" else 2.0 + case["zeros"]
    return {"bytes": act * N * (K / 2 + scale * K / case["group"]) + 2 * M * (K + N), "flops": 2.0 * M * N * K}


# ------------------------------------------------------------------------------------ from the definition
def _route_exact(s):
    l = s["logits"].double().cpu().numpy()
    T, E = l.shape
    live = np.isfinite(l)
    with np.errstate(over="ignore"):
        if s["score"] == "sigmoid":
            score = np.where(live, 0.5 * (1.0 + np.tanh(0.5 * np.where(live, l, 0.0))), 0.0)
        else:
            e = np.where(live, np.exp(np.where(live, l, 0.0)), 0.0)
            score = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    c = score + (s["bias_e"].double().cpu().numpy() if s["bias"] else 0.0)
    key = np.where(live, c if s["bias"] else l, -np.inf)
    if s["groups"] > 1:
        per = E // s["groups"]
        in_group = np.where(live, c, -np.inf).reshape(T, s["groups"], per)
        best = np.partition(in_group, per - s["group_best"], axis=2)[:, :, per - s["group_best"]:]
        value = np.where(np.isfinite(best.max(2)), np.where(np.isfinite(best), best, 0.0).sum(2), -np.inf)
        place = np.argsort(np.argsort(-value, axis=1, kind="stable"), axis=1, kind="stable")
        key = np.where(np.repeat(place < s["top_groups"], per, axis=1), key, -np.inf)
    idx = np.argsort(-key, axis=1, kind="stable")[:, : s["k"]]
    some = np.isfinite(np.take_along_axis(key, idx, 1))
    picked = np.where(some, np.take_along_axis(score, idx, 1), 0.0)
    total = np.maximum(picked.sum(1, keepdims=True), 1e-300) if s["renormalize"] else 1.0
    out = {"experts": np.where(some, idx, -1).astype(np.int32), "probs": s["scale"] * picked / total}
    if s["train"]:
        g = np.where(some, s["dprobs"].double().cpu().numpy(), 0.0)
        # dL/d(score_i), through the weights scale s_i / sum_j s_j: scale sum_j s_j (g_i - g_j) / total^2
        if s["renormalize"]:
            ds = s["scale"] * (picked[:, None, :] * (g[:, :, None] - g[:, None, :])).sum(2) / total / total
        else:
            ds = s["scale"] * g
        full = np.zeros((T, E))
        np.put_along_axis(full, idx, np.where(some, ds, 0.0), 1)
        if s["score"] == "sigmoid":
            out["dlogits"] = full * score * (1.0 - score)
        else:
            out["dlogits"] = score * (full - (full * score).sum(1, keepdims=True))
    return out


def _norm_exact(s):
    f = torch.float64
    H = s["H"]
    one = torch.ones(H, dtype=f, device="cuda")
    x, b = s["x"].to(f), s["branch"].to(f)
    wb = s["w_post"].to(f) if s["post"] else one
    g = (s["g"].to(f) if s["g"] is not None else torch.ones(1, dtype=f, device="cuda")) * s["scale"]
    vb = b.square().sum(1, keepdim=True) / H + _EPS if s["post"] else torch.ones((s["T"], 1), dtype=f, device="cuda")
    z = g * wb * b / vb.sqrt()
    y = x + z
    res = {"y": y}
    vy = y.square().sum(1, keepdim=True) / H + _EPS
    if s["pre"]:
        res["h"] = s["w_pre"].to(f) * y / vy.sqrt()
    if not s["train"]:
        return res
    d = s["dy"].to(f)
    if s["pre"]:
        dh = s["dh"].to(f)
        res["dw_pre"] = (dh * y / vy.sqrt()).sum(0)
        t = dh * s["w_pre"].to(f)
        d = d + t / vy.sqrt() - y * (t * y).sum(1, keepdim=True) / (H * vy ** 1.5)
    res["dx"] = d
    if s["g"] is not None:
        dg = d * s["scale"] * wb * b / vb.sqrt()
        res["dgate"] = dg.sum(0) if s["gate"] == "channel" else dg.sum(1, keepdim=True) if s["gate"] == "token" else dg
    if s["post"]:
        res["dw_post"] = (d * g * b / vb.sqrt()).sum(0)
        t = d * g * wb
        res["dbranch"] = t / vb.sqrt() - b * (t * b).sum(1, keepdim=True) / (H * vb ** 1.5)
    else:
        res["dbranch"] = d * g
    return res


def _w4_exact(s):
    f = torch.float64
    N, K = s["N"], s["K"]
    y = torch.zeros((s["M"], N), dtype=f, device="cuda")
    ends = np.cumsum(s["host_splits"])
    mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=f, device="cuda") / 2
    for g in range(s["G"]):
        rows = slice(int(ends[g]) - s["host_splits"][g], int(ends[g]))
        if rows.start == rows.stop:
            continue
        w = torch.empty((N, K), dtype=f, device="cuda")
        for half in (0, 1):
            c = (s["codes"][g].int() >> (4 * half)) & 15
            if s["kind"] == "nvfp4":
                w[:, half::2] = mag[(c & 7).long()] * (1 - 2 * (c >> 3))
            else:
                w[:, half::2] = c.to(f) - (s["zero"][g].to(f).repeat_interleave(s["group"] // 2, 1) if s["zeros"] else 8)
        if s["kind"] == "nvfp4":
            e = (s["scales"][g].int() >> 3) & 15                                     # E4M3: all of these are normal
            scale = torch.ldexp((8 + (s["scales"][g].int() & 7)).to(f), (e - 10).to(f))
            scale = scale * (s["amax"][g].to(f) / 2688)
        else:
            scale = s["scales"][g].to(f)
        w *= scale.repeat_interleave(s["group"], 1)
        y[rows] = s["x"][rows].to(f) @ w.t()
    return {"y": y}


def exact(case, seed):
    """run()'s outputs in 64 bits, written from the definitions."""
    s = prepare(case, seed)
    return {"route": _route_exact, "norm": _norm_exact, "w4": _w4_exact}[case["op"]](s)
