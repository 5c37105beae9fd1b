"""Cases of the mixture-of-experts and MXFP4 operators, with their plain forms.

Six operators, two listed cases each (the smallest call in use and a prompt):
the router, the gated and the down products grouped by expert, the weighted
sum and norms that close the block, MXFP4 quantisation (there and back), and
the gated MLP on MXFP4 activations and weights.

`run` with `own` false is the plain form: elementary torch operations in 32
bits, rounded once.  `exact` is the definition in 64 bits, written apart.
Hidden sizes are those of this repository's workloads (896, 1536, 3584) and
expert widths are fractions of theirs; the rest is generic.
"""
import functools
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
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
        # one token decoded on its own: latency of the router
        {"name": "route-token", "op": "route", "T": 1, "E": 64, "k": 6, "dtype": "f32",
         "renorm": True, "masked": 0.0},
        # a prompt: many tokens, bf16 logits with ties, experts masked off, some tokens wholly
        {"name": "route-prompt", "op": "route", "T": 8191, "E": 128, "k": 8, "dtype": "bf16",
         "renorm": False, "masked": 0.05},
        # four sequences decoded together, 8 experts each: one row per expert, weights stream
        {"name": "up-decode", "op": "up", "R": 32, "E": 64, "k": 8, "K": 1536, "N": 1792,
         "skew": 0.0},
        # a prompt of 8190 tokens, 4 experts each, unevenly filled experts
        {"name": "up-prompt", "op": "up", "R": 32760, "E": 32, "k": 4, "K": 3584, "N": 2368,
         "skew": 0.25},
        # the down products of the same two calls
        {"name": "down-decode", "op": "down", "R": 32, "E": 64, "K": 1792, "N": 1536,
         "skew": 0.0},
        {"name": "down-prompt", "op": "down", "R": 32760, "E": 32, "K": 2368, "N": 3584,
         "skew": 0.25},
        # the end of the block for one token, and for a prompt with the stream kept in fp32
        {"name": "norm-token", "op": "norm", "T": 1, "k": 6, "D": 3584, "dtype": "bf16",
         "shared": True, "post": True, "gate": "row", "dropped": 0.0},
        {"name": "norm-prompt", "op": "norm", "T": 8191, "k": 8, "D": 1536, "dtype": "f32",
         "shared": False, "post": True, "gate": "each", "dropped": 0.03},
        # activations of a small batch and of a prompt to 4 bits and back
        {"name": "fp4-quant-batch", "op": "quant", "rows": 128, "K": 896},
        {"name": "fp4-quant-prompt", "op": "quant", "rows": 8192, "K": 3584},
        # the 7B MLP at decode and at a prompt: activations quantised on the way
        {"name": "fp4-mlp-decode", "op": "fp4", "M": 16, "N": 18944, "K": 3584},
        {"name": "fp4-mlp-prompt", "op": "fp4", "M": 8192, "N": 18944, "K": 3584},
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = max(lo, min(hi, -(-v // step) * step))
    return v if v != 3072 else 3104


def draw(rng):
    op = rng.choice(["route", "up", "down", "norm", "quant", "fp4"])
    if op == "route":
        E = rng.choice([8, 16, 40, 60, 64, 72, 128, 160, 200, 256])
        return {"op": op, "T": _log(rng, 1, 16384 * 64 // max(E, 64)), "E": E,
                "k": rng.randint(1, 8), "dtype": rng.choice(["f32", "bf16"]),
                "renorm": rng.random() < 0.5, "masked": rng.choice([0.0, 0.02, 0.2])}
    if op in ("up", "down"):
        E = rng.choice([4, 8, 16, 24, 40, 64, 96])
        k = rng.randint(1, min(E, 8))
        K = _log(rng, 512, 3584, 8)
        # the expert stack stays under that of the listed prompt
        top = 32 * 3584 * 2368 // (E * K) // 8 * 8
        N = min(_log(rng, 384, 4864, 8), max(128, top))
        R = _log(rng, 1, 8190) * k
        c = {"op": op, "R": min(R, 32760 // k * k), "E": E, "K": K, "N": N,
             "skew": rng.choice([0.0, 0.1, 0.25])}
        if op == "up":
            c["k"] = k
        return c
    if op == "norm":
        D = _log(rng, 512, 8192, 8)
        k = rng.randint(1, 8)
        T = _log(rng, 1, max(1, 8191 * 8 * 1536 // (k * D)))
        return {"op": op, "T": min(T, 12000), "k": k, "D": D, "dtype": rng.choice(["bf16", "f32"]),
                "shared": rng.random() < 0.5, "post": rng.random() < 0.7,
                "gate": rng.choice(["none", "row", "each"]), "dropped": rng.choice([0.0, 0.1])}
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 8192), "K": _log(rng, 64, 3584, 32)}
    return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 512, 18944, 8),
            "K": _log(rng, 512, 3584, 32)}


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


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, std=1.0, dtype=BF16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=F32).mul_(std).to(dtype)


def _weights(g, E, K, C):
    """[E, K, C] bf16 of variance 1 / K, made an expert at a time."""
    w = torch.empty(E, K, C, device=DEV, dtype=BF16)
    for e in range(E):
        w[e] = _randn(g, K, C, std=K ** -0.5)
    return w


def _blocks(x):
    """Fragment order of 4-bit codes: rows in blocks of 32, K in groups of 256, as
    [row block, group, step of 64, half, row, 16 bytes]; the padding is zero codes."""
    rows, kb = x.shape
    rb, g = -(-rows // 32), -(-kb // 128)
    p = torch.zeros(rb * 32, g * 128, device=x.device, dtype=torch.uint8)
    p[:rows, :kb] = x
    return p.view(rb, 32, g, 4, 2, 16).permute(0, 2, 3, 4, 1, 5).contiguous().view(-1)


def _scale_blocks(s):
    """Fragment order of the scale bytes: [row block, group, half, row, step]; the padding is 2^0."""
    rows, n = s.shape
    rb, g = -(-rows // 32), -(-n // 8)
    p = torch.full((rb * 32, g * 8), 127, device=s.device, dtype=torch.uint8)
    p[:rows, :n] = s
    return p.view(rb, 32, g, 4, 2).permute(0, 2, 4, 1, 3).contiguous().view(-1)


def _quantize(x):
    """(codes [rows, K / 2] low nibble first, scale bytes [rows, K / 32]) of finite x."""
    rows, K = x.shape
    b = x.float().view(rows, K // 32, 32)
    top = b.abs().amax(-1)
    _, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1)
    e = torch.where(top > 0, (e - 3).clamp(-127, 127), -127)
    v = b * torch.exp2(-e.float())[..., None]
    a = v.abs()
    code = torch.where(a < 2, (a * 2).round(),
                       torch.where(a < 4, a.round() + 2, ((a / 2).round() + 4).clamp(max=7)))
    code = (code.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)).view(rows, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        x = _randn(g, T, E, std=1.5, dtype=F32)
        if case["masked"]:
            off = torch.rand(T, E, generator=g, device=DEV) < case["masked"]
            off |= torch.rand(T, 1, generator=g, device=DEV) < case["masked"] / 4
            x = torch.where(off, float("-inf"), x)
        i32 = dict(device=DEV, dtype=torch.int32)
        return {"case": case, "logits": x.to(BF16 if case["dtype"] == "bf16" else F32),
                "weights": torch.empty(T, k, device=DEV), "experts": torch.empty(T, k, **i32),
                "offsets": torch.empty(E + 1, **i32), "rows": torch.empty(T * k, **i32)}
    if op in ("up", "down"):
        R, E, K, N = case["R"], case["E"], case["K"], case["N"]
        n = torch.tensor(_counts(case), device=DEV)[torch.randperm(E, generator=g, device=DEV)]
        offsets = torch.zeros(E + 1, device=DEV, dtype=torch.int32)
        offsets[1:] = n.cumsum(0)
        # slots in random order over the experts, ascending within each
        expert = torch.repeat_interleave(torch.arange(E, device=DEV), n, output_size=R)
        rows = torch.randperm(R, generator=g, device=DEV)
        rows = rows[torch.argsort(expert * R + rows)].int()
        s = {"case": case, "offsets": offsets, "rows": rows, "most": max(_counts(case)),
             "Y": torch.empty(R, N, device=DEV, dtype=BF16)}
        if op == "up":
            s["A"] = _randn(g, R // case["k"], K)
            s["W"] = _weights(g, E, K, 2 * N)
        else:
            s["A"] = _randn(g, R, K, std=0.35)
            s["W"] = _weights(g, E, K, N)
        return s
    if op == "norm":
        T, k, D = case["T"], case["k"], case["D"]
        xt = BF16 if case["dtype"] == "bf16" else F32
        w = torch.softmax(_randn(g, T, k, dtype=F32), -1)
        e = torch.randint(0, 64, (T, k), generator=g, device=DEV, dtype=torch.int32)
        if case["dropped"]:
            lost = torch.rand(T, k, generator=g, device=DEV) < case["dropped"]
            e, w = torch.where(lost, -1, e), torch.where(lost, 0.0, w)
        B = _randn(g, T * k, D, std=0.5)
        B[(e < 0).view(-1)] = float("nan")  # rows that no product wrote
        return {"case": case, "B": B, "w": w, "e": e, "X": _randn(g, T, D, std=2.0, dtype=xt),
                "S": _randn(g, T, D, std=0.5) if case["shared"] else None,
                "post": _randn(g, D, std=0.2).add_(1) if case["post"] else None,
                "gate": {"none": None, "row": _randn(g, D, std=0.3).add_(1),
                         "each": _randn(g, T, D, std=0.5)}[case["gate"]],
                "pre": _randn(g, D, std=0.2).add_(1),
                "X_out": torch.empty(T, D, device=DEV, dtype=xt),
                "H": torch.empty(T, D, device=DEV, dtype=BF16)}
    if op == "quant":
        rows, K = case["rows"], case["K"]
        # activations: rows of different size, a few large channels
        x = torch.randn(rows, K, generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=DEV))
        x *= torch.where(torch.rand(1, K, generator=g, device=DEV) < 0.01, 20.0, 1.0)
        return {"case": case, "X": x.to(BF16), "out": torch.empty(rows, K, device=DEV, dtype=BF16),
                **_room(rows, K)}
    M, N, K = case["M"], case["N"], case["K"]
    q, s = _quantize(_randn(g, 2 * N, K, std=K ** -0.5))
    return {"case": case, "X": _randn(g, M, K), "W": _blocks(q), "SW": _scale_blocks(s),
            "Y": torch.empty(M, N, device=DEV, dtype=BF16), **_room(M, K)}


def _room(rows, K):
    n = -(-rows // 32) * -(-K // 256)
    return {"Q": torch.empty(n * 4096, device=DEV, dtype=torch.uint8),
            "SQ": torch.empty(n * 256, device=DEV, dtype=torch.uint8)}


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
    sw.swiglu_route(h, s["logits"], s["weights"], s["experts"], s["offsets"], s["rows"], s["ws"],
                    c["T"], c["E"], c["k"], renormalize=c["renorm"],
                    dtype=sw.DTYPE_BF16 if c["dtype"] == "bf16" else sw.DTYPE_F32)
    return s["weights"], s["experts"], s["offsets"], s["rows"]


def _own_up(s):
    sw, h = _lib()
    c = s["case"]
    sw.swiglu_grouped_forward(h, s["A"], s["rows"], s["offsets"], s["W"], s["Y"],
                              c["R"] // c["k"], c["R"], c["N"], c["K"], c["E"], k=c["k"])
    return s["Y"]


def _own_down(s):
    sw, h = _lib()
    c = s["case"]
    sw.swiglu_grouped_matmul(h, s["A"], s["rows"], s["offsets"], s["W"], s["Y"], c["R"], c["N"],
                             c["K"], c["E"])
    return s["Y"]


def _own_norm(s):
    sw, h = _lib()
    c = s["case"]
    sw.swiglu_combine_norm(h, s["B"], s["w"], s["e"], s["S"], s["X"], s["post"], s["gate"],
                           s["pre"], s["X_out"], s["H"], c["T"], c["D"], k=c["k"], scale=0.5,
                           eps=1e-6, gate_ld=c["D"] if c["gate"] == "each" else 0,
                           dtype=sw.DTYPE_BF16 if c["dtype"] == "bf16" else sw.DTYPE_F32)
    return s["X_out"], s["H"]


def _own_quant(s):
    sw, h = _lib()
    c = s["case"]
    sw.swiglu_quantize_mxfp4(h, s["X"], s["Q"], s["SQ"], c["rows"], c["K"])
    sw.swiglu_dequantize_mxfp4(h, s["Q"], s["SQ"], s["out"], c["rows"], c["K"])
    return s["out"]


def _own_fp4(s):
    sw, h = _lib()
    c = s["case"]
    sw.swiglu_quantize_mxfp4(h, s["X"], s["Q"], s["SQ"], c["M"], c["K"])
    sw.swiglu_forward_mxfp4(h, s["Q"], s["SQ"], s["W"], s["SW"], s["Y"], c["M"], c["N"], c["K"])
    return s["Y"]


# --------------------------------------------------------------- plain forms
def _plain_route(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = s["logits"].float()
    v, e = torch.sort(x, dim=-1, descending=True, stable=True)
    v, e = v[:, :k], e[:, :k]
    there = v > float("-inf")
    top = torch.where(there[:, :1], v[:, :1], 0.0)
    p = torch.where(there, torch.exp(v - top), 0.0)
    total = p.sum(-1, keepdim=True) if c["renorm"] else torch.exp(x - top).sum(-1, keepdim=True)
    w = torch.where(there, p / torch.where(total > 0, total, 1.0), 0.0)
    e = torch.where(there, e, -1)
    key = torch.where(there, e, E).view(-1)
    rows = torch.argsort(key, stable=True)
    n = (key[:, None] == torch.arange(E, device=x.device)).sum(0)
    offsets = torch.zeros(E + 1, device=x.device, dtype=torch.int32)
    offsets[1:] = n.cumsum(0)
    rows = torch.where(torch.arange(T * k, device=x.device) < offsets[E], rows, -1)
    return w, e.int(), offsets, rows.int()


def _plain_products(s, A, C):
    """fp32 products [R, C] of the gathered rows A [R, K] (bf16) with their experts' weights."""
    c = s["case"]
    R, E, off = c["R"], c["E"], s["offsets"].long()
    i = torch.arange(R, device=A.device)
    e = torch.searchsorted(off[1:], i, right=True)
    if R <= E:  # few rows: each with a copy of its expert's weights
        return torch.bmm(A.float()[:, None], s["W"][e].float())[:, 0]
    at = off[:-1, None] + torch.arange(s["most"], device=A.device)
    held = A.float()[at.clamp(max=R - 1)]
    return torch.bmm(held, s["W"].float())[e, i - off[e]]


def _plain_up(s):
    c = s["case"]
    p = _plain_products(s, s["A"][s["rows"].long() // c["k"]], 2 * c["N"])
    g, u = p[:, 0::2], p[:, 1::2]
    return (g / (1 + torch.exp(-g)) * u).to(BF16)


def _plain_down(s):
    y = torch.empty_like(s["Y"])
    y[s["rows"].long()] = _plain_products(s, s["A"], s["case"]["N"]).to(BF16)
    return y


def _plain_norm(s):
    c = s["case"]
    T, k, D = c["T"], c["k"], c["D"]
    there = s["e"] >= 0
    B = torch.where(there[..., None], s["B"].float().view(T, k, D), 0.0)
    o = (B * s["w"][..., None]).sum(1)
    if s["S"] is not None:
        o = o + s["S"].float()
    if s["post"] is not None:
        o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + 1e-6) * s["post"].float()
    if s["gate"] is not None:
        o = o * s["gate"].float()
    x = s["X"].float() + 0.5 * o
    h = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s["pre"].float()
    return x.to(s["X"].dtype), h.to(BF16)


@functools.lru_cache(maxsize=None)
def _table():
    """Values of the E2M1 codes 0 to 15."""
    return torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                        device=DEV)


def _grid(code):
    return _table()[code.int()]


def _values(q, s):
    """Values [rows, K] of row-major codes and scale bytes."""
    rows, kb = q.shape
    v = torch.stack([_grid(q & 15), _grid(q >> 4)], -1).view(rows, kb // 16, 32)
    return (v * torch.exp2(s.float() - 127)[..., None]).view(rows, kb * 2)


def _plain_quant(s):
    return _values(*_quantize(s["X"])).to(BF16)


def _unblock(p, s, rows, K):
    """Row-major codes and scale bytes of a fragment-ordered tensor."""
    rb, g = -(-rows // 32), -(-K // 256)
    q = p.view(rb, g, 4, 2, 32, 16).permute(0, 4, 1, 2, 3, 5).reshape(rb * 32, g * 128)
    e = s.view(rb, g, 2, 32, 4).permute(0, 3, 1, 4, 2).reshape(rb * 32, g * 8)
    return q[:rows, :K // 2], e[:rows, :K // 32]


def _plain_fp4(s):
    c = s["case"]
    a = _values(*_quantize(s["X"]))
    w = _values(*_unblock(s["W"], s["SW"], 2 * c["N"], c["K"]))
    p = a @ w.t()
    g, u = p[:, 0::2], p[:, 1::2]
    return (g / (1 + torch.exp(-g)) * u).to(BF16)


_OWN = {"route": _own_route, "up": _own_up, "down": _own_down, "norm": _own_norm,
        "quant": _own_quant, "fp4": _own_fp4}
_PLAIN = {"route": _plain_route, "up": _plain_up, "down": _plain_down, "norm": _plain_norm,
          "quant": _plain_quant, "fp4": _plain_fp4}


# ---------------------------------------------------------------- what it costs
def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        b = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * E * b + 12 * T * k + 4 * (E + 1), "flops": 4 * T * E}
    if op in ("up", "down"):
        R, K, N = case["R"], case["K"], case["N"]
        active = sum(n > 0 for n in _counts(case))
        m = 2 if op == "up" else 1
        a = 2 * K * (R // case["k"] if op == "up" else R)
        return {"bytes": a + 2 * m * K * N * active + 2 * R * N + 4 * R,
                "flops": 2 * m * R * K * N}
    if op == "norm":
        T, k, D = case["T"], case["k"], case["D"]
        b = 2 if case["dtype"] == "bf16" else 4
        n = 2 * T * k * D + 2 * b * T * D + 2 * T * D + 8 * T * k + 2 * D
        n += 2 * T * D * case["shared"] + 2 * D * case["post"]
        n += {"none": 0, "row": 2 * D, "each": 2 * T * D}[case["gate"]]
        return {"bytes": n, "flops": T * D * (2 * k + 10)}
    if op == "quant":
        n = case["rows"] * case["K"]
        return {"bytes": 4 * n + 2 * (n // 2 + n // 32), "flops": 4 * n}
    M, N, K = case["M"], case["N"], case["K"]
    codes = K // 2 + K // 32
    return {"bytes": 2 * M * K + 2 * M * codes + 2 * N * codes + 2 * M * N,
            "flops": 4 * M * N * K}


# ------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        x = s["logits"].to(F64)
        T, E, k = case["T"], case["E"], case["k"]
        p = torch.softmax(x, -1)  # all NaN where everything is masked
        p = torch.where(torch.isnan(p), 0.0, p)
        w = torch.topk(p, k, dim=-1).values
        if case["renorm"]:
            w = w / w.sum(-1, keepdim=True).clamp_min(1e-300)
        return w, None, None, None
    if op in ("up", "down"):
        R = case["R"]
        off = s["offsets"].tolist()
        y = torch.empty(R, case["N"], device=DEV, dtype=F64)
        for e in range(case["E"]):
            rows = s["rows"][off[e]:off[e + 1]].long()
            if not rows.numel():
                continue
            w = s["W"][e].to(F64)
            if op == "up":
                a = s["A"][rows // case["k"]].to(F64)
                g, u = a @ w[:, 0::2].contiguous(), a @ w[:, 1::2].contiguous()
                y[off[e]:off[e + 1]] = g * torch.sigmoid(g) * u
            else:
                y[rows] = s["A"][off[e]:off[e + 1]].to(F64) @ w
        return y
    if op == "norm":
        T, k, D = case["T"], case["k"], case["D"]
        o = torch.zeros(T, D, device=DEV, dtype=F64)
        B, w = s["B"].view(T, k, D), s["w"].to(F64)
        for j in range(k):
            part = w[:, j, None] * B[:, j].to(F64)
            o += torch.where(s["e"][:, j, None] >= 0, part, torch.zeros_like(part))
        if s["S"] is not None:
            o += s["S"].to(F64)
        if s["post"] is not None:
            o = o / (o.square().mean(-1, keepdim=True) + 1e-6).sqrt() * s["post"].to(F64)
        if s["gate"] is not None:
            o = o * s["gate"].to(F64)
        x = s["X"].to(F64) + o / 2
        h = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * s["pre"].to(F64)
        return x, h
    if op == "quant":
        return _nearest(s["X"])
    a = _nearest(s["X"])
    q, e = _unblock(s["W"], s["SW"], 2 * case["N"], case["K"])
    w = _values(q, e).to(F64)  # exact: at most two significant bits
    g, u = a @ w[0::2].t().contiguous(), a @ w[1::2].t().contiguous()
    return g * torch.sigmoid(g) * u


def _nearest(x):
    """Each block of 32 to the nearest of the 4-bit values at its scale, even codes at ties."""
    rows, K = x.shape
    b = x.to(F64).view(-1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(top.clamp_min(2.0 ** -140))) - 2
    scale = torch.exp2(e.clamp(-127, 127))
    a = (b / scale).abs()
    best, out = torch.full_like(a, float("inf")), torch.zeros_like(a)
    for v in (0., 1., 2., 4., .5, 1.5, 3., 6.):  # even codes first: they keep a tie
        d = (a - v).abs()
        out = torch.where(d < best, v, out)
        best = torch.minimum(best, d)
    return (torch.copysign(out, b) * scale).view(rows, K)
