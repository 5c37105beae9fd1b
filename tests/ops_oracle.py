"""Plain 64-bit definitions of the mixture-of-experts and MXFP4 operators, on the
CPU, for the GPU tests.  Written from the definitions in include/swiglu.h; no
library code.  Error bounds next to the values: `slack` counts one fp32 step
(2^-24 relative) for every operation a sum of that length can make."""
import numpy as np
import torch

F64 = torch.float64
U32 = 2.0 ** -24          # half a step of fp32
HALF_BF16 = 2.0 ** -8     # torch.finfo(bfloat16).eps / 2
TINY = 2.0 ** -126        # below the normal range steps are absolute


def sigmoid_gate(g, u):
    return g / (1 + torch.exp(-g)) * u


def gated(a, w):
    """(y, slack) of SiLU(a G) * (a U), w [K, 2N] with G, U in alternate columns."""
    a, w = a.to(F64), w.to(F64)
    K = a.shape[-1]
    p, mag = a @ w, a.abs() @ w.abs()
    g, u = p[:, 0::2], p[:, 1::2]
    eg, eu = (K + 4) * U32 * mag[:, 0::2], (K + 4) * U32 * mag[:, 1::2]
    y = sigmoid_gate(g, u)
    silu = sigmoid_gate(g, torch.ones_like(g))
    # |SiLU'| <= 1.1; the hardware exp and reciprocal are within a few steps,
    # the exponent's argument within |g| steps
    slack = 1.1 * u.abs() * eg + silu.abs() * eu + 1.1 * eg * eu + (16 + g.abs()) * U32 * y.abs()
    return y, slack


def plain(a, w):
    a, w = a.to(F64), w.to(F64)
    return a @ w, (a.shape[-1] + 4) * U32 * (a.abs() @ w.abs())


def assert_close(got, want, slack, what, half=HALF_BF16):
    got = got.detach().cpu().to(F64)
    tol = slack + half * (want.abs() + slack) + TINY
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(int(x) for x in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first {i}: "
                             f"got {float(got[i])!r} want {float(want[i])!r} tol {float(tol[i]):.3g}")


def route(logits, k, renorm):
    """(weights, experts, offsets, rows) of logits [T, E] (any float dtype)."""
    x = logits.to(F64).numpy()
    T, E = x.shape
    w, e = np.zeros((T, k)), np.full((T, k), -1, dtype=np.int64)
    for t in range(T):
        v = np.where(np.isnan(x[t]), -np.inf, x[t])
        order = sorted((j for j in range(E) if v[j] > -np.inf), key=lambda j: (-v[j], j))[:k]
        if not order:
            continue
        m = v[order[0]]
        with np.errstate(invalid="ignore"):
            p = np.where(v == m, 1.0, np.exp(v - m))
        total = p[order].sum() if renorm else p.sum()
        w[t, :len(order)] = p[order] / total
        e[t, :len(order)] = order
    slots = [s for s in sorted(range(T * k), key=lambda s: (e.flat[s], s)) if e.flat[s] >= 0]
    rows = np.full(T * k, -1, dtype=np.int64)
    rows[:len(slots)] = slots
    offsets = np.zeros(E + 1, dtype=np.int64)
    offsets[1:] = np.cumsum([(e == j).sum() for j in range(E)])
    return w, e, offsets, rows


def combine_norm(B, w, e, S, X, post, gate, pre, scale, eps):
    """(x, h) and bounds; B [T, k, D]."""
    T, k, D = B.shape
    there = (e >= 0)[..., None]
    B = torch.where(there, B.to(F64), torch.zeros((), dtype=F64))
    terms = B * torch.where(there, w.to(F64)[..., None], torch.zeros((), dtype=F64))
    o, mag = terms.sum(1), terms.abs().sum(1)
    if S is not None:
        o, mag = o + S.to(F64), mag + S.to(F64).abs()
    eo = (k + 2) * U32 * mag
    # the mean of squares: D rounded terms in a tree, the square root, the division
    def norm(v, ev, g):
        ms = v.square().mean(-1, keepdim=True)
        r = 1 / (ms + eps).sqrt()
        dms = (2 * v.abs() * ev + ev.square()).mean(-1, keepdim=True) + (D / 8 + 32) * U32 * ms
        rel = 0.5 * dms / (ms + eps) + 8 * U32
        out = v * r * g
        return out, (r * g.abs() * ev + out.abs() * rel) * 1.01 + 4 * U32 * out.abs()
    if post is not None:
        o, eo = norm(o, eo, post.to(F64))
    if gate is not None:
        o, eo = o * gate.to(F64), eo * gate.to(F64).abs() + U32 * (o * gate.to(F64)).abs()
    x = X.to(F64) + scale * o
    ex = abs(scale) * eo + 2 * U32 * (X.to(F64).abs() + (scale * o).abs())
    h, eh = norm(x, ex, pre.to(F64))
    return x, ex, h, eh


# ---- MXFP4 -------------------------------------------------------------------------
GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


def quantize(x):
    """(codes [rows, K] uint8, scales [rows, K / 32] uint8) of bf16 values as float64."""
    rows, K = x.shape
    b = x.reshape(rows, K // 32, 32)
    a = np.abs(b)
    nan = np.isnan(b).any(-1)
    top = np.where(np.isnan(a), 0, a).max(-1)
    with np.errstate(divide="ignore"):
        e = np.where(np.isinf(top), 128, np.floor(np.log2(np.where(np.isinf(top), 1, top))))
    e = np.clip(np.where(top == 0, -127, e - 2), -127, 127)
    with np.errstate(invalid="ignore"):
        v = np.minimum(a * np.exp2(-e)[..., None], 6.0)
    v = np.where(np.isnan(v), 0, v)
    d = np.abs(v[..., None] - GRID)
    best = d.min(-1, keepdims=True)
    tie = d == best
    # the even code among the nearest
    code = np.where(tie, np.where(np.arange(8) % 2 == 0, 0, 1), 2).argmin(-1)
    code = code | (np.signbit(b).astype(np.int64) << 3)
    return (code.reshape(rows, K).astype(np.uint8),
            np.where(nan, 255, e + 127).astype(np.uint8))


def values(codes, scales):
    rows, K = codes.shape
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v.reshape(rows, K // 32, 32) * s[..., None]).reshape(rows, K)


def fragment_codes(codes):
    """Fragment order, written out index by index as the header has it."""
    rows, K = codes.shape
    rbs, G = -(-rows // 32), -(-K // 256)
    full = np.zeros((rbs * 32, G * 256), dtype=np.uint8)
    full[:rows, :K] = codes
    out = np.zeros(rbs * G * 4096, dtype=np.uint8)
    rb, g, s, h, i, b = np.meshgrid(*(np.arange(n) for n in (rbs, G, 4, 2, 32, 16)), indexing="ij")
    r, k = 32 * rb + i, 256 * g + 64 * s + 32 * h + 2 * b
    out[(((rb * G + g) * 4 + s) * 2 + h) * 512 + 16 * i + b] = full[r, k] | full[r, k + 1] << 4
    return out


def fragment_scales(scales):
    rows, n = scales.shape
    rbs, G = -(-rows // 32), -(-n // 8)
    full = np.full((rbs * 32, G * 8), 127, dtype=np.uint8)
    full[:rows, :n] = scales
    out = np.zeros(rbs * G * 256, dtype=np.uint8)
    rb, g, h, i, s = np.meshgrid(*(np.arange(n) for n in (rbs, G, 2, 32, 4)), indexing="ij")
    out[((rb * G + g) * 2 + h) * 128 + 4 * i + s] = full[32 * rb + i, 8 * g + 2 * s + h]
    return out
