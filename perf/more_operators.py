"""Cases of the scored router and the 8-bit integer operators, with their plain forms.

Six operators, two listed cases each (the smallest call in use and a prompt):
the router on sigmoid or softmax scores with a balancing bias and groups of
experts, the quantisation of activations to 8-bit integers with a scale for
each row, and the gated and plain products of such rows with 8-bit weights that
have a scale for each channel, for one weight set and grouped by expert.

`run` with `own` false is the plain form: elementary torch operations in 32
bits (the borders of a choice and of a rounding in 64), rounded once.  `exact`
is the definition in 64 bits, written apart.  Hidden sizes are those of this
repository's workloads (896, 1536, 3584, 18944) and expert widths are fractions
of theirs; the rest is generic.
"""
import math

import torch

own = False

BF16, F32, F64, I8, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int8, torch.int32
DEV = "cuda"
_handles = []


def _lib():
    """The library and a handle that a program keeps for its lifetime."""
    import gemm_epilogues_mlp_amd as sw
    if not _handles:
        _handles.append(sw.swiglu_create(0))
    return sw, _handles[0]


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one token decoded on its own: latency of the router, all of its steps in use
        {"name": "scored-token", "op": "route", "T": 1, "E": 256, "k": 8, "dtype": "f32",
         "score": "sigmoid", "bias": True, "groups": 8, "top": 4, "best": 2, "renorm": True,
         "scale": 2.5, "masked": 0.0},
        # a prompt: many tokens, bf16 logits, experts masked off, some tokens wholly
        {"name": "scored-prompt", "op": "route", "T": 8191, "E": 256, "k": 8, "dtype": "bf16",
         "score": "sigmoid", "bias": True, "groups": 8, "top": 4, "best": 2, "renorm": True,
         "scale": 2.5, "masked": 0.05},
        # activations of a small batch before the gated products, and of a prompt before the
        # down products
        {"name": "int8-quant-batch", "op": "quant", "rows": 16, "K": 3584},
        {"name": "int8-quant-prompt", "op": "quant", "rows": 8192, "K": 18944},
        # the 7B MLP's gated products at decode (the weights stream) and at a prompt
        {"name": "int8-up-decode", "op": "up", "M": 16, "N": 18944, "K": 3584},
        {"name": "int8-up-prompt", "op": "up", "M": 8192, "N": 18944, "K": 3584},
        # its down products
        {"name": "int8-down-decode", "op": "down", "M": 16, "N": 3584, "K": 18944},
        {"name": "int8-down-prompt", "op": "down", "M": 8192, "N": 3584, "K": 18944},
        # four sequences decoded together, 8 experts each: one row per expert
        {"name": "int8-experts-up-decode", "op": "gup", "R": 32, "E": 64, "k": 8, "K": 1536,
         "N": 1792, "skew": 0.0},
        # a prompt of 8190 tokens, 4 experts each, unevenly filled experts
        {"name": "int8-experts-up-prompt", "op": "gup", "R": 32760, "E": 32, "k": 4, "K": 3584,
         "N": 2368, "skew": 0.25},
        # the down products of the same two calls
        {"name": "int8-experts-down-decode", "op": "gdown", "R": 32, "E": 64, "K": 1792, "N": 1536,
         "skew": 0.0},
        {"name": "int8-experts-down-prompt", "op": "gdown", "R": 32760, "E": 32, "K": 2368,
         "N": 3584, "skew": 0.25},
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, -(-v // step) * step))


def draw(rng):
    op = rng.choice(["route", "quant", "up", "down", "gup", "gdown"])
    if op == "route":
        E = rng.choice([8, 16, 40, 60, 64, 72, 128, 160, 200, 256])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0])
        top = rng.randint(1, groups)
        best = rng.choice([1, 2]) if groups > 1 else 1
        return {"op": op, "T": _log(rng, 1, min(16384 * 64 // max(E, 64), 8191)), "E": E,
                "k": rng.randint(1, min(8, top * (E // groups))), "dtype": rng.choice(["f32", "bf16"]),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.7,
                "groups": groups, "top": top, "best": best, "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5]), "masked": rng.choice([0.0, 0.02, 0.2])}
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 8192), "K": _log(rng, 64, 18944, 16)}
    if op == "up":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 512, 18944, 8),
                "K": _log(rng, 512, 3584, 16)}
    if op == "down":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 512, 3584, 8),
                "K": _log(rng, 512, 18944, 16)}
    E = rng.choice([4, 8, 16, 24, 40, 64, 96])
    k = rng.randint(1, min(E, 8))
    K = _log(rng, 512, 3584, 16)
    # the expert stack stays under that of the listed prompt
    top = 32 * 3584 * 2368 // (E * K) // 8 * 8
    N = min(_log(rng, 384, 4864, 8), max(128, top))
    R = min(_log(rng, 1, 8190) * k, 32760 // k * k)
    c = {"op": op, "R": R, "E": E, "K": K, "N": N, "skew": rng.choice([0.0, 0.1, 0.25])}
    if op == "gup":
        c["k"] = k
    return c


# ------------------------------------------------------------------ the inputs
def _counts(case):
    """Rows of each expert rank: shares (rank + 1) ** -skew, largest remainders first."""
    E, R = case["E"], case["R"]
    share = [(e + 1.0) ** -case["skew"] for e in range(E)]
    total = sum(share)
    want = [R * s / total for s in share]
    n = [int(w) for w in want]
    for e in sorted(range(E), key=lambda e: (n[e] - want[e], e))[:R - sum(n)]:
        n[e] += 1
    return n


def _randn(g, *shape, std=1.0, dtype=F32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=F32).mul_(std).to(dtype)


def _activations(g, rows, K):
    """bf16 rows of different size, a few large channels."""
    x = torch.randn(rows, K, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=DEV))
    x *= torch.where(torch.rand(1, K, generator=g, device=DEV) < 0.01, 8.0, 1.0)
    return x.to(BF16)


def _quantize(x):
    """(codes [rows, K] int8, scales [rows]) of finite x; a code next to a half is settled in 64 bits."""
    top = x.abs().amax(-1, keepdim=True).float()
    q = torch.round(x.to(F64) * 127 / torch.where(top > 0, top, 1.0).to(F64))
    return q.to(I8), (top / 127)[:, 0]


def _blocks(w):
    """Fragment order of int8 rows: rows in blocks of 32, K in groups of 128, as [row block,
    group, step of 32, half, row, 16 bytes]; the padding is zero."""
    rows, K = w.shape
    rb, g = -(-rows // 32), -(-K // 128)
    p = torch.zeros(rb * 32, g * 128, device=w.device, dtype=I8)
    p[:rows, :K] = w
    return p.view(rb, 32, g, 4, 2, 16).permute(0, 2, 3, 4, 1, 5).contiguous().view(-1)


def _weights(g, E, rows, K):
    """Fragment-ordered codes of E matrices [rows, K] and their scales [E, rows]; the values have
    variance 1 / K."""
    size = -(-rows // 32) * -(-K // 128) * 4096
    P = torch.empty(E, size, device=DEV, dtype=I8)
    for e in range(E):
        P[e] = _blocks(_randn(g, rows, K, std=36.0).round_().clamp_(-127, 127).to(I8))
    S = torch.exp(_randn(g, E, rows, std=0.1)) * (K ** -0.5 / 36)
    return P, S


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        x = _randn(g, T, E, std=1.5)
        if case["masked"]:
            off = torch.rand(T, E, generator=g, device=DEV) < case["masked"]
            off |= torch.rand(T, 1, generator=g, device=DEV) < case["masked"] / 4
            x = torch.where(off, float("-inf"), x)
        i32 = dict(device=DEV, dtype=I32)
        return {"case": case, "logits": x.to(BF16 if case["dtype"] == "bf16" else F32),
                "bias": _randn(g, E, std=0.05) if case["bias"] else None,
                "weights": torch.empty(T, k, device=DEV), "experts": torch.empty(T, k, **i32),
                "offsets": torch.empty(E + 1, **i32), "rows": torch.empty(T * k, **i32)}
    if op == "quant":
        rows, K = case["rows"], case["K"]
        return {"case": case, "X": _activations(g, rows, K),
                "Q": torch.empty(rows, K, device=DEV, dtype=I8), "SQ": torch.empty(rows, device=DEV)}
    if op in ("up", "down"):
        M, N, K = case["M"], case["N"], case["K"]
        Q, SQ = _quantize(_activations(g, M, K))
        P, SW = _weights(g, 1, N * (2 if op == "up" else 1), K)
        return {"case": case, "Q": Q, "SQ": SQ, "P": P, "SW": SW,
                "Y": torch.empty(M, N, device=DEV, dtype=BF16)}
    R, E, K, N = case["R"], case["E"], case["K"], case["N"]
    n = torch.tensor(_counts(case), device=DEV)[torch.randperm(E, generator=g, device=DEV)]
    offsets = torch.zeros(E + 1, device=DEV, dtype=I32)
    offsets[1:] = n.cumsum(0)
    # slots in random order over the experts, ascending within each
    expert = torch.repeat_interleave(torch.arange(E, device=DEV), n, output_size=R)
    rows = torch.randperm(R, generator=g, device=DEV)
    rows = rows[torch.argsort(expert * R + rows)].int()
    Q, SQ = _quantize(_activations(g, R // case["k"] if op == "gup" else R, K))
    P, SW = _weights(g, E, N * (2 if op == "gup" else 1), K)
    return {"case": case, "offsets": offsets, "rows": rows, "most": max(_counts(case)), "Q": Q,
            "SQ": SQ, "P": P, "SW": SW, "Y": torch.empty(R, N, device=DEV, dtype=BF16)}


# -------------------------------------------------------------- the operators
def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_route(s):
    sw, h = _lib()
    c = s["case"]
    if "ws" not in s:
        s["ws"] = torch.empty(sw.swiglu_route_workspace_bytes(c["T"], c["E"], c["k"]),
                              device=DEV, dtype=torch.uint8)
    sw.swiglu_route_scored(h, s["logits"], s["bias"], s["weights"], s["experts"], s["offsets"],
                           s["rows"], s["ws"], c["T"], c["E"], c["k"],
                           score=sw.SCORE_SIGMOID if c["score"] == "sigmoid" else sw.SCORE_SOFTMAX,
                           renormalize=c["renorm"], scale=c["scale"], groups=c["groups"],
                           top_groups=c["top"], group_best=c["best"],
                           dtype=sw.DTYPE_BF16 if c["dtype"] == "bf16" else sw.DTYPE_F32)
    return s["weights"], s["experts"], s["offsets"], s["rows"]


def _own_quant(s):
    sw, h = _lib()
    c = s["case"]
    sw.swiglu_quantize_int8(h, s["X"], s["Q"], s["SQ"], c["rows"], c["K"])
    return s["Q"], s["SQ"]


def _own_up(s):
    sw, h = _lib()
    c = s["case"]
    sw.swiglu_forward_int8(h, s["Q"], s["SQ"], s["P"], s["SW"], s["Y"], c["M"], c["N"], c["K"])
    return s["Y"]


def _own_down(s):
    sw, h = _lib()
    c = s["case"]
    sw.swiglu_matmul_int8(h, s["Q"], s["SQ"], s["P"], s["SW"], s["Y"], c["M"], c["N"], c["K"])
    return s["Y"]


def _own_gup(s):
    sw, h = _lib()
    c = s["case"]
    sw.swiglu_grouped_forward_int8(h, s["Q"], s["SQ"], s["rows"], s["offsets"], s["P"], s["SW"],
                                   s["Y"], c["R"] // c["k"], c["R"], c["N"], c["K"], c["E"],
                                   k=c["k"])
    return s["Y"]


def _own_gdown(s):
    sw, h = _lib()
    c = s["case"]
    sw.swiglu_grouped_matmul_int8(h, s["Q"], s["SQ"], s["rows"], s["offsets"], s["P"], s["SW"],
                                  s["Y"], c["R"], c["N"], c["K"], c["E"])
    return s["Y"]


# --------------------------------------------------------------- plain forms
def _plain_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    x = s["logits"].to(F64)
    there = x > float("-inf")
    if c["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-x))
    else:
        top = x.amax(-1, keepdim=True)
        p = torch.where(there, torch.exp(x - torch.where(top > float("-inf"), top, 0.0)), 0.0)
        total = p.sum(-1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
    v = torch.where(there, p + s["bias"].to(F64) if c["bias"] else p, float("-inf"))
    if G > 1:
        best = torch.sort(v.view(T, G, E // G), dim=-1, descending=True).values[..., :c["best"]]
        best = torch.where(best[..., :1] > float("-inf"),
                           torch.where(best > float("-inf"), best, 0.0), best).sum(-1)
        first = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :c["top"]]
        kept = (first[..., None] == torch.arange(G, device=x.device)).any(1)
        v = torch.where(kept.repeat_interleave(E // G, 1), v, float("-inf"))
    v, e = torch.sort(v, dim=-1, descending=True, stable=True)
    v, e = v[:, :k], e[:, :k]
    there = v > float("-inf")
    w = torch.where(there, p.gather(1, e), 0.0)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    e = torch.where(there, e, -1)
    key = torch.where(there, e, E).view(-1)
    rows = torch.argsort(key, stable=True)
    n = (key[:, None] == torch.arange(E, device=x.device)).sum(0)
    offsets = torch.zeros(E + 1, device=x.device, dtype=I32)
    offsets[1:] = n.cumsum(0)
    rows = torch.where(torch.arange(T * k, device=x.device) < offsets[E], rows, -1)
    return (w * c["scale"]).float(), e.int(), offsets, rows.int()


def _plain_quant(s):
    return _quantize(s["X"])


def _unblock(P, rows, K):
    """Codes [E, rows, K] of fragment-ordered ones."""
    rb, g = -(-rows // 32), -(-K // 128)
    w = P.view(-1, rb, g, 4, 2, 32, 16).permute(0, 1, 5, 2, 3, 4, 6).reshape(-1, rb * 32, g * 128)
    return w[:, :rows, :K]


def _gate(p):
    g, u = p[:, 0::2], p[:, 1::2]
    return g / (1 + torch.exp(-g)) * u


def _plain_dense(s, rows):
    """fp32 values [M, rows] of the products."""
    w = _unblock(s["P"], rows, s["case"]["K"])[0].float()
    return (s["Q"].float() @ w.t()) * s["SQ"][:, None] * s["SW"][0]


def _plain_up(s):
    return _gate(_plain_dense(s, 2 * s["case"]["N"])).to(BF16)


def _plain_down(s):
    return _plain_dense(s, s["case"]["N"]).to(BF16)


def _plain_grouped(s, Q, SQ, C):
    """fp32 values [R, C] of the sorted rows Q [R, K] with their experts' weights."""
    c = s["case"]
    R, E, off = c["R"], c["E"], s["offsets"].long()
    i = torch.arange(R, device=Q.device)
    e = torch.searchsorted(off[1:], i, right=True)
    w = _unblock(s["P"], C, c["K"])
    if R <= E:  # few rows: each with a copy of its expert's weights
        p = torch.bmm(w[e].float(), Q.float()[:, :, None])[:, :, 0]
    else:
        at = off[:-1, None] + torch.arange(s["most"], device=Q.device)
        held = Q.float()[at.clamp(max=R - 1)]
        p = torch.bmm(held, w.float().transpose(1, 2).contiguous())[e, i - off[e]]
    return p * SQ[:, None] * s["SW"][e]


def _plain_gup(s):
    c = s["case"]
    t = s["rows"].long() // c["k"]
    return _gate(_plain_grouped(s, s["Q"][t], s["SQ"][t], 2 * c["N"])).to(BF16)


def _plain_gdown(s):
    y = torch.empty_like(s["Y"])
    y[s["rows"].long()] = _plain_grouped(s, s["Q"], s["SQ"], s["case"]["N"]).to(BF16)
    return y


_OWN = {"route": _own_route, "quant": _own_quant, "up": _own_up, "down": _own_down, "gup": _own_gup,
        "gdown": _own_gdown}
_PLAIN = {"route": _plain_route, "quant": _plain_quant, "up": _plain_up, "down": _plain_down,
          "gup": _plain_gup, "gdown": _plain_gdown}


# ---------------------------------------------------------------- what it costs
def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        b = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * E * b + 12 * T * k + 4 * (E + 1) + 4 * E * case["bias"],
                "flops": 6 * T * E}
    if op == "quant":
        n = case["rows"] * case["K"]
        return {"bytes": 3 * n + 4 * case["rows"], "flops": 4 * n}
    K, N = case["K"], case["N"]
    m = 2 if op in ("up", "gup") else 1
    if op in ("up", "down"):
        M = case["M"]
        return {"bytes": M * (K + 4) + m * N * (K + 4) + 2 * M * N, "flops": 2 * m * M * N * K}
    R = case["R"]
    active = sum(n > 0 for n in _counts(case))
    a = (K + 4) * (R // case["k"] if op == "gup" else R)
    return {"bytes": a + m * N * (K + 4) * active + 2 * R * N + 4 * R + 4 * (case["E"] + 1),
            "flops": 2 * m * R * K * N}


# ------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_weights(s), None, None, None
    if op == "quant":
        return None, s["X"].abs().max(-1).values.to(F64) / 127
    K, N = case["K"], case["N"]
    if op in ("up", "down"):
        return _exact_products(s["Q"], s["SQ"], s["P"][0], s["SW"][0], op == "up", N, K)
    off = s["offsets"].tolist()
    y = torch.empty(case["R"], N, device=DEV, dtype=F64)
    for e in range(case["E"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        slots = s["rows"][a:b].long()
        if op == "gup":
            t = slots // case["k"]
            y[a:b] = _exact_products(s["Q"][t], s["SQ"][t], s["P"][e], s["SW"][e], True, N, K)
        else:
            y[slots] = _exact_products(s["Q"][a:b], s["SQ"][a:b], s["P"][e], s["SW"][e], False, N, K)
    return y


def _exact_products(Q, SQ, P, SW, gated, N, K):
    C = 2 * N if gated else N
    # row, k -> place in fragment order
    r, k = torch.arange(C, device=DEV), torch.arange(K, device=DEV)
    groups = -(-K // 128)
    at = (r // 32 * groups * 4096 + r % 32 * 16)[:, None] + \
        (k // 128 * 4096 + k % 128 // 32 * 1024 + k % 32 // 16 * 512 + k % 16)[None]
    w = P[at].to(F64) * SW.to(F64)[:, None]
    a = Q.to(F64) * SQ.to(F64)[:, None]
    if not gated:
        return a @ w.t()
    g, u = a @ w[0::2].t(), a @ w[1::2].t()
    return g * torch.sigmoid(g) * u


def _exact_weights(s):
    """The chosen experts' weights, one choice after another."""
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    low = float("-inf")
    x = s["logits"].to(F64)
    shut = torch.isneginf(x)
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1).nan_to_num(0.0)
    v = p if s["bias"] is None else p + s["bias"].to(F64)
    v = v.masked_fill(shut, low)
    if G > 1:
        parts = v.view(T, G, E // G)
        total = torch.topk(parts, min(c["best"], E // G), dim=-1).values
        total = total.masked_fill(torch.isneginf(total) & (parts > low).any(-1, keepdim=True), 0.0)
        total = total.sum(-1)
        kept = torch.zeros(T, G, device=DEV, dtype=torch.bool)
        for _ in range(c["top"]):
            kept.scatter_(1, total.masked_fill(kept, low).max(-1, keepdim=True).indices, True)
        v = v.masked_fill(~kept.repeat_interleave(E // G, 1), low)
    w = torch.zeros(T, k, device=DEV, dtype=F64)
    for i in range(k):
        best, at = v.max(-1, keepdim=True)
        w[:, i:i + 1] = p.gather(1, at).masked_fill(torch.isneginf(best), 0.0)
        v = v.scatter(1, at, low)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp_min(1e-300)
    return w * c["scale"]
