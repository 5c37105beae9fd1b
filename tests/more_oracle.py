"""Plain 64-bit definitions of the scored router and the 8-bit integer operators, on the CPU,
for the GPU tests.  Written from the definitions in include/swiglu.h; no library code.
Bounds as in ops_oracle: one step of fp32 (2^-24 relative) for every rounded operation."""
import numpy as np
import torch

from ops_oracle import F64, U32, sigmoid_gate


def route_scored(logits, bias, k, score, renorm, scale, groups, top, best):
    """(weights, experts, offsets, rows) of logits [T, E]; without a bias single scores are compared by
    their logits."""
    x = logits.to(F64).numpy()
    b = np.zeros(x.shape[1]) if bias is None else bias.to(F64).numpy()
    T, E = x.shape
    size = E // groups
    w, e = np.zeros((T, k)), np.full((T, k), -1, dtype=np.int64)
    for t in range(T):
        v = np.where(np.isnan(x[t]), -np.inf, x[t])
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "sigmoid":
                s = 1 / (1 + np.exp(-v))
            else:
                m = v.max()
                s = np.where(v == m, 1.0, np.exp(v - m)) if m > -np.inf else np.zeros(E)
                s = s / s.sum() if s.sum() > 0 else s
            c = s + b
        c = np.where((v > -np.inf) & ~np.isnan(c), c, -np.inf)
        if groups > 1:
            value = []
            for g in range(groups):
                part = sorted(c[g * size:(g + 1) * size], reverse=True)[:best]
                part = [p for p in part if p > -np.inf]
                value.append(sum(part) if part else -np.inf)
                if bias is None and best == 1:
                    value[-1] = v[g * size:(g + 1) * size].max()
            kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top]
            for g in range(groups):
                if g not in kept:
                    c[g * size:(g + 1) * size] = -np.inf
        by = v if bias is None else c
        order = sorted((j for j in range(E) if c[j] > -np.inf), key=lambda j: (-by[j], j))[:k]
        if not order:
            continue
        p = s[order]
        if renorm:
            p = p / p.sum() if p.sum() > 0 else np.zeros(len(order))
        w[t, :len(order)] = p * scale
        e[t, :len(order)] = order
    slots = [s for s in sorted(range(T * k), key=lambda s: (e.flat[s], s)) if e.flat[s] >= 0]
    rows = np.full(T * k, -1, dtype=np.int64)
    rows[:len(slots)] = slots
    offsets = np.zeros(E + 1, dtype=np.int64)
    offsets[1:] = np.cumsum([(e == j).sum() for j in range(E)])
    return w, e, offsets, rows


def quantize(x):
    """(codes int64 [rows, K], scales float64 [rows]) of bf16 values; whole numbers throughout:
    |x| = m 2^-133 with m < 2^261, so 127 m / a is compared with halves exactly."""
    v = x.to(F64).numpy()
    rows, K = v.shape
    q, s = np.zeros((rows, K), dtype=np.int64), np.zeros(rows)
    for r in range(rows):
        if not np.isfinite(v[r]).all():
            s[r] = np.nan
            continue
        a = np.abs(v[r]).max()
        s[r] = a / 127
        if a == 0:
            continue
        A = int(np.ldexp(a, 133))
        for i in range(K):
            n = 127 * int(np.ldexp(abs(v[r, i]), 133))
            d, left = divmod(n, A)
            d += 2 * left > A or (2 * left == A and d % 2 == 1)
            q[r, i] = -d if v[r, i] < 0 else d
    return q, s


def fragments(w):
    """Fragment order of int8 w [E, rows, K], written out index by index as the header has it."""
    E, rows, K = w.shape
    B, G = -(-rows // 32), -(-K // 128)
    full = np.zeros((E, B * 32, G * 128), dtype=np.int8)
    full[:, :rows, :K] = w
    out = np.zeros(E * B * G * 4096, dtype=np.int8)
    e, b, g, s, h, i, j = np.meshgrid(*(np.arange(n) for n in (E, B, G, 4, 2, 32, 16)), indexing="ij")
    out[((((e * B + b) * G + g) * 4 + s) * 2 + h) * 512 + 16 * i + j] = \
        full[e, 32 * b + i, 128 * g + 32 * s + 16 * h + j]
    return out


def products(q, sq, w, sw):
    """(p, slack) of codes q [M, K], w [C, K] and their scales: the exact sum is rounded to fp32 and
    multiplied twice."""
    p = (q.to(F64) @ w.to(F64).t().contiguous()) * sq.to(F64)[:, None] * sw.to(F64)
    return p, 4 * U32 * p.abs()


def gated(q, sq, w, sw):
    p, e = products(q, sq, w, sw)
    g, u, eg, eu = p[:, 0::2], p[:, 1::2], e[:, 0::2], e[:, 1::2]
    y = sigmoid_gate(g, u)
    silu = sigmoid_gate(g, torch.ones_like(g))
    # as ops_oracle.gated: |SiLU'| <= 1.1, the exp and the reciprocal within a few steps
    return y, 1.1 * u.abs() * eg + silu.abs() * eu + 1.1 * eg * eu + (16 + g.abs()) * U32 * y.abs()
