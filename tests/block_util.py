"""Plain 64-bit forms for the tests of the operators around the experts (CPU)."""
import math

import numpy as np
import torch


# ----------------------------------------------------------------------------- routing
def route_scores(row, score):
    """Scores of one row of logits in 64 bits; masked ones are 0."""
    live = [v != -math.inf for v in row]
    if score == "sigmoid":
        def f(v):
            if math.isnan(v):
                return v
            return 1.0 / (1.0 + math.exp(-v)) if v > -700 else math.exp(v) if v > -745 else 0.0
        return [f(v) if a else 0.0 for v, a in zip(row, live)]
    if any(math.isnan(v) or v == math.inf for v in row):
        return [math.nan if a else 0.0 for a in live]
    top = max((v for v in row), default=0.0)
    e = [math.exp(v - top) if a else 0.0 for v, a in zip(row, live)]
    s = sum(e)
    return [v / s if s else 0.0 for v in e]


def _key(v):
    """Ascending sort key: greater first, NaN before all numbers."""
    return (0, 0.0) if math.isnan(v) else (1, -v)


def plain_choice(row, k, score, bias, groups=1, top_groups=1, group_best=1):
    """The experts of one row, in order, -1 behind the last."""
    E = len(row)
    s = route_scores(row, score)
    c = [s[e] + bias[e] for e in range(E)] if bias is not None else list(s)
    live = [row[e] != -math.inf and c[e] != -math.inf for e in range(E)]
    order = c if bias is not None else row
    allowed = range(E)
    if groups > 1:
        per, value = E // groups, []
        by = c if bias is not None or group_best > 1 else row
        for g in range(groups):
            members = sorted((by[e] for e in range(g * per, (g + 1) * per) if live[e]), key=_key)[:group_best]
            value.append(math.nan if any(math.isnan(v) for v in members) else sum(members) if members else None)
        best = sorted((g for g in range(groups) if value[g] is not None), key=lambda g: (_key(value[g]), g))[:top_groups]
        allowed = [e for e in range(E) if e // per in best]
    got = sorted((e for e in allowed if live[e]), key=lambda e: (_key(order[e]), e))[:k]
    return got + [-1] * (k - len(got))


def plain_probs(row, chosen, score, renormalize, scale):
    """Probabilities of one row's chosen experts in 64 bits (ratios by logarithms where they are renormalized)."""
    live = [e for e in chosen if e >= 0]
    if not renormalize:
        s = route_scores(row, score)
        return [scale * s[e] if e >= 0 else 0.0 for e in chosen]
    if score == "softmax" and any(math.isnan(v) or v == math.inf for v in row) and \
            any(math.isnan(row[e]) or row[e] == math.inf for e in live):
        return [math.nan if e >= 0 else 0.0 for e in chosen]
    log = {e: row[e] if score == "softmax" else (min(row[e], 0.0) - math.log1p(math.exp(-abs(row[e])))
                                                 if not math.isnan(row[e]) else math.nan) for e in live}
    top = max(log.values(), default=0.0)
    w = {e: math.exp(log[e] - top) for e in live}
    total = sum(w[e] for e in live)
    return [scale * w[e] / total if e >= 0 else 0.0 for e in chosen]


def plain_dlogits(row, chosen, g, score, renormalize, scale):
    """Gradient of sum_j g_j probs_j for one row, and the sum of the magnitudes of what enters each element."""
    E = len(row)
    s = route_scores(row, score)
    d, mag = [0.0] * E, [0.0] * E
    slots = [(e, scale * gj) for e, gj in zip(chosen, g) if 0 <= e < E and row[e] != -math.inf]
    if renormalize:
        w = plain_probs(row, [e for e, _ in slots], score, True, 1.0)
        dot = sum(gj * wj for (_, gj), wj in zip(slots, w))
        for (e, gj), wj in zip(slots, w):
            f = 1.0 - s[e] if score == "sigmoid" else 1.0
            if score == "sigmoid":
                f = route_scores([-row[e]], "sigmoid")[0]
            d[e] += wj * (gj - dot) * f
            mag[e] += wj * (abs(gj) + sum(abs(h) * v for (_, h), v in zip(slots, w))) * f
    elif score == "sigmoid":
        for e, gj in slots:
            v = gj * s[e] * route_scores([-row[e]], "sigmoid")[0]
            d[e] += v
            mag[e] += abs(v)
    else:
        dot = sum(gj * s[e] for e, gj in slots)
        adot = sum(abs(gj) * s[e] for e, gj in slots)
        for e in range(E):
            if row[e] == -math.inf:
                continue
            at = [gj for f, gj in slots if f == e]
            d[e] = s[e] * (sum(at) - dot)
            mag[e] = s[e] * (sum(abs(v) for v in at) + adot)
    return d, mag


def route_tol(E, spread):
    """Relative error of a probability: the difference of two logits is rounded once, which exp turns into
    |difference| half steps (spread of them at most, twice: numerator and sum); exp itself and the two
    divisions are off by at most 2 steps each; the sum has at most E additions; one product with the scale."""
    return 2.0 ** -24 * (2 * spread + E + 16)


# ----------------------------------------------------------------------------- norms
def norm_forms(x, branch, weight, branch_weight, gate, scale, eps, dy=None, dh=None):
    """All results in 64 bits, and for each the sum of the magnitudes of what enters it: {name: (value, mag)}."""
    f = torch.float64
    x = x.to(f)
    T, H = x.shape
    out = {}
    n = an = bh = None
    if branch is not None:
        b = branch.to(f)
        rb = 1.0 / torch.sqrt((b * b).mean(1, keepdim=True) + eps) if branch_weight is not None else torch.ones((T, 1), dtype=f)
        wb = branch_weight.to(f) if branch_weight is not None else torch.ones(H, dtype=f)
        g = scale * (gate.to(f) if gate is not None else torch.ones(1, dtype=f))
        bh = b * rb
        n = bh * wb
        y = x + g * n
        ay = x.abs() + (g * n).abs()
        out["y"] = (y, ay)
    else:
        y, ay = x, x.abs()
    if weight is not None:
        w = weight.to(f)
        ry = 1.0 / torch.sqrt((y * y).mean(1, keepdim=True) + eps)
        # an error of y moves the root as well: by the rows' norms
        grow = 1.0 + torch.sqrt((ay * ay).mean(1, keepdim=True)) * ry
        yh, ayh = y * ry, ay * ry * grow
        out["h"] = (yh * w, ayh * w.abs())
    if dy is None and dh is None:
        return out
    d = dy.to(f) if dy is not None else torch.zeros((T, H), dtype=f)
    ad = d.abs()
    if dh is not None:
        u = dh.to(f) * w
        d = d + ry * (u - yh * (u * yh).mean(1, keepdim=True))
        ad = ad + ry * grow * (u.abs() + ayh * (u.abs() * ayh).mean(1, keepdim=True))
        out["dweight"] = ((dh.to(f) * yh).sum(0), (dh.to(f).abs() * ayh).sum(0))
    out["dx"] = (d, ad)
    if branch is not None:
        dg, adg = scale * d * n, abs(scale) * ad * n.abs()
        if gate is not None:
            if gate.dim() == 1:
                dg, adg = dg.sum(0), adg.sum(0)
            elif gate.shape[1] == 1 and H > 1 or tuple(gate.shape) == (T, 1):
                dg, adg = dg.sum(1, keepdim=True), adg.sum(1, keepdim=True)
            out["dgate"] = (dg, adg)
        q, aq = g * d, g.abs() * ad
        if branch_weight is not None:
            out["dbranch_weight"] = ((q * bh).sum(0), (aq * bh.abs()).sum(0))
            t, at = q * wb, aq * wb.abs()
            q = rb * (t - bh * (t * bh).mean(1, keepdim=True))
            aq = rb * (at + bh.abs() * (at * bh.abs()).mean(1, keepdim=True))
        out["dbranch"] = (q, aq)
    return out


def assert_norm(got, form, terms, what):
    """One rounding to got's type; `terms` fp32 roundings, each of at most a whole step 2^-23, of sums and products
    that are at most mag."""
    want, mag = form
    dt = got.dtype
    info = torch.finfo(dt)
    tol = info.eps / 2 * want.abs() * (1 + 2.0 ** -8) + terms * 2.0 ** -23 * mag + info.tiny * info.eps / 2
    bad = ~((got.detach().cpu().double() - want).abs() <= tol)
    if bad.any():
        i = tuple(int(v[0]) for v in bad.nonzero(as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: got {got.detach().cpu()[i]}, "
                             f"want {want[i]}, tolerance {tol[i]}")


# ----------------------------------------------------------------------------- weights of 4 bits
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def nibbles(codes):
    """uint8 [..., K / 2] -> int64 [..., K], the even element in the low four bits."""
    c = codes.long()
    return torch.stack([c & 15, c >> 4], -1).flatten(-2)


def int4_values(codes, scales, zeros):
    q = nibbles(codes).double()
    group = q.shape[-1] // scales.shape[-1]
    z = zeros.double().repeat_interleave(group, -1) if zeros is not None else 8.0
    return (q - z) * scales.double().repeat_interleave(group, -1)


def e4m3_value(b):
    s, e, m = b >> 7, (b >> 3) & 15, b & 7
    v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -v if s else v


def nvfp4_values(codes, scales, amax):
    q = torch.tensor(E2M1, dtype=torch.float64)[nibbles(codes)]
    table = torch.tensor([e4m3_value(b) for b in range(256)], dtype=torch.float64)
    s = table[scales.long()].repeat_interleave(16, -1)
    # S = fp32(2688 / amax), 1 for an amax of 0, clipped to the largest fp32
    g = [1.0 if a == 0 else float(min(np.float64(np.float32(2688.0 / np.float64(a))), float(np.finfo(np.float32).max))) for a in amax.tolist()]
    return q * s / torch.tensor(g, dtype=torch.float64)[:, None, None]
