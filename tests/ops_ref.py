"""Plain 64-bit references of the block operators, row by row from their definitions (tests only)."""
import math

import numpy as np
import torch


def half_step(dtype):
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


# ---- norms
def norm(v, kind, w, b, eps):
    if kind == "none":
        return v
    c = v - v.mean(1, keepdim=True) if kind == "layer" else v
    out = c / torch.sqrt((c * c).mean(1, keepdim=True) + eps) * w
    return out if b is None else out + b


def gate_rows(gate, rows_per_gate, T):
    return gate[torch.arange(T) // rows_per_gate]


def block(x, y, after, wa, ba, gate, rpg, alpha, beta, eps):
    z = norm(y, after, wa, ba, eps)
    if gate is not None:
        z = z * gate_rows(gate, rpg, x.shape[0])
    return alpha * x + beta * z


# ---- routing
def route(logits, k, score, bias, groups, top_groups, group_top, renorm, scale):
    """Every token by sorting Python tuples; returns numpy arrays and the closest call of each token."""
    T, E = logits.shape
    per = E // groups
    idx = np.full((T, k), -1, np.int64)
    gate = np.zeros((T, k))
    for t in range(T):
        l = logits[t].astype(np.float64)
        live = [e for e in range(E) if l[e] > -math.inf]
        s = np.zeros(E)
        if score == "sigmoid":
            for e in live:
                s[e] = 1 / (1 + math.exp(-l[e])) if l[e] > -700 else 0.0
        elif live:
            m = max(l[e] for e in live)
            z = {e: 1.0 if l[e] == m else math.exp(l[e] - m) for e in live}
            total = math.fsum(z.values())
            for e in live:
                s[e] = z[e] / total
        live = [e for e in live if bias is None or bias[e] > -math.inf]
        worth = {e: s[e] + (0.0 if bias is None else float(bias[e])) for e in live}
        rank = {e: float(l[e]) if bias is None else worth[e] for e in live}
        if groups > 1:
            of = []
            for g in range(groups):
                best = sorted((worth[e] for e in live if e // per == g), reverse=True)[:group_top]
                if bias is None and group_top == 1:
                    best = sorted((rank[e] for e in live if e // per == g), reverse=True)[:1]
                of.append((-(sum(best) if best else -math.inf), g))
            kept = {g for _, g in sorted(of)[:top_groups]}
            live = [e for e in live if e // per in kept]
        chosen = sorted(live, key=lambda e: (-rank[e], e))[:k]
        total = math.fsum(s[e] for e in chosen)
        for i, e in enumerate(chosen):
            idx[t, i] = e
            gate[t, i] = scale * (s[e] if not renorm else (s[e] / total if total > 0 else 0.0))
    counts = np.array([(idx == e).sum() for e in range(E)], np.int64)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    row_of = np.full((T, k), -1, np.int64)
    token = np.full(T * k, -1, np.int64)
    at = offsets[:-1].copy()
    for t in range(T):
        for i in range(k):
            e = idx[t, i]
            if e >= 0:
                row_of[t, i] = at[e]
                token[at[e]] = t
                at[e] += 1
    return dict(idx=idx, gate=gate, counts=counts, offsets=offsets, row_of=row_of, token_of_row=token)


def gates(logits, idx, score, renorm, scale):
    """Gates of a fixed choice as a differentiable 64-bit function of finite logits."""
    p = torch.sigmoid(logits) if score == "sigmoid" else torch.softmax(logits, 1)
    kept = idx >= 0
    g = p.gather(1, idx.clamp(min=0)) * kept
    if renorm:
        g = g / (g.sum(1, keepdim=True) + (~kept).all(1, keepdim=True))
    return scale * g


# ---- 8-bit experts
def quantize(x):
    """(q, scale) with numpy's IEEE single-precision quotients."""
    x = x.astype(np.float32)
    bad = ~np.isfinite(x).all(1)
    with np.errstate(all="ignore"):
        top = np.where(bad, np.float32(np.nan), np.abs(x).max(1, initial=np.float32(0))).astype(np.float32)
        scale = top / np.float32(127)
        q = np.where(scale[:, None] > 0, np.clip(np.rint(x / scale[:, None]), -127, 127), 0)
    return np.where(bad[:, None], 0, q).astype(np.int64), scale.astype(np.float32)


def int8_experts(x, w, ws, offsets, rows, w3=None, w3s=None):
    """(y, and what a sum in 32 bits may be off by) in 64 bits; rows past offsets[E] stay NaN."""
    E, N, K = w.shape
    q, scale = quantize(x)
    R = len(rows)
    y, slack = np.full((R, N), np.nan), np.zeros((R, N))
    for e in range(E):
        lo = min(max(int(offsets[e]), 0), R)
        hi = min(max(int(offsets[e + 1]), lo), R)
        for r in range(lo, hi):
            t = int(rows[r])
            real = 0 <= t < len(q)
            qt = q[t] if real else np.zeros(K, np.int64)
            sx = float(scale[t]) if real else 0.0

            def product(w, ws):
                v = (w[e].astype(np.int64) @ qt) * ws[e].astype(np.float64) * sx
                size = np.abs(w[e].astype(np.int64)) @ np.abs(qt)
                # whole numbers below 2^24 add exactly in fp32; above, one rounding (or truncation) for each
                # 16 products
                off = np.where(size < 2**24, 0.0, (K / 16 + 1) * 2.0**-23 * size) * np.abs(ws[e]) * abs(sx)
                return v, off + 4 * 2.0**-24 * np.abs(v)

            v, off = product(w, ws)
            if w3 is None:
                y[r], slack[r] = v, off
            else:
                u, off3 = product(w3, w3s)
                sig = 1 / (1 + np.exp(-np.clip(v, -700, None)))
                y[r] = v * sig * u
                # d silu / dv is at most 1.1; exp and the quotient add a few ulp, exp(-v) by its argument's
                slack[r] = 1.1 * off * np.abs(u) + off3 * np.abs(v * sig) + (4 + np.abs(v)) * 2.0**-22 * np.abs(y[r])
    return y, slack
