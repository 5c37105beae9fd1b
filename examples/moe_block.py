"""A mixture-of-experts block on the library's operators, end to end.

    python examples/moe_block.py [--tokens 1 --experts 64 --top 6 --width 1536 --expert-width 896
                                  --shared-width 1792 --blocks 2 --int8 --check]

Every block takes the residual stream X and its normed form H:

    logits         = H Wr                                       torch, fp32
    e, w, spans    = swiglu_route(logits)
    up             = swiglu_grouped_forward(H, ...)             experts, gated
    down           = swiglu_grouped_matmul(up, ...)
    S              = swiglu_forward_mxfp4(quantised H) Ws       the shared expert, 4 bits
    X, H           = swiglu_combine_norm(down, w, e, S, X, ...)

With --int8 the experts' weights and inputs are 8-bit integers, and the router scores by sigmoid
with a bias for balance over four groups of experts, of which two are open to a token:

    e, w, spans    = swiglu_route_scored(logits, bias)
    up             = swiglu_grouped_forward_int8(quantised H, ...)
    down           = swiglu_grouped_matmul_int8(quantised up, ...)

H of a block is the input of the next one.  The step is captured in a HIP graph
and replayed, as a serving loop would; --check compares it with the same block
in plain torch operations.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_epilogues_mlp_amd as sw  # noqa: E402

BF16, DEV = torch.bfloat16, "cuda"


class Block:
    """One block's weights, laid out once, and its workspaces for T tokens."""

    groups, top_groups, scale = 4, 2, 1.5      # of the scored router

    def __init__(self, handle, T, E, k, D, N, NS, seed, int8=False):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def randn(*shape, std):
            return torch.randn(*shape, generator=g, device=DEV).mul_(std).to(BF16)
        self.h, self.size, self.int8 = handle, (T, E, k, D, N, NS), int8
        self.router = randn(D, E, std=D ** -0.5).float()
        self.up, self.down = randn(E, D, 2 * N, std=D ** -0.5), randn(E, N, D, std=N ** -0.5)
        self.post, self.pre = randn(D, std=0.1).add_(1), randn(D, std=0.1).add_(1)
        self.shared_down = randn(NS, D, std=NS ** -0.5)
        # the shared expert's Gate and Up weights: paired rows, then 4 bits
        w1, w2 = randn(D, NS, std=D ** -0.5), randn(D, NS, std=D ** -0.5)
        paired = torch.empty(2 * NS, D, dtype=BF16, device=DEV)
        sw.swiglu_pack_kmajor(handle, w1, w2, paired, D, NS)
        self.w4, self.sw4 = self._codes(2 * NS, D)
        sw.swiglu_quantize_mxfp4(handle, paired, self.w4, self.sw4, 2 * NS, D)

        i32 = dict(device=DEV, dtype=torch.int32)
        self.w, self.e = torch.empty(T, k, device=DEV), torch.empty(T, k, **i32)
        self.offsets, self.rows = torch.empty(E + 1, **i32), torch.empty(T * k, **i32)
        need = sw.swiglu_route_workspace_bytes(T, E, k)
        self.ws = torch.empty(need, device=DEV, dtype=torch.uint8) if need else None
        self.gated = torch.empty(T * k, N, device=DEV, dtype=BF16)
        self.out = torch.empty(T * k, D, device=DEV, dtype=BF16)
        self.q, self.sq = self._codes(T, D)
        self.shared = torch.empty(T, NS, device=DEV, dtype=BF16)
        self.H = torch.empty(T, D, device=DEV, dtype=BF16)
        if int8:
            self.bias = 0.1 * torch.randn(E, generator=g, device=DEV)
            self.up, self.down = self._int8_weights(self.up), self._int8_weights(self.down)
            self.q8, self.s8 = self._int8_rows(T, D)
            self.q8_up, self.s8_up = self._int8_rows(T * k, N)

    def _int8_weights(self, w):
        """w [E, K, rows] as fragments, with the scales of its output channels, and as plain codes."""
        E, K, rows = w.shape
        codes, scales = self._int8_rows(E * rows, K)
        sw.swiglu_quantize_int8(self.h, w.transpose(1, 2).contiguous(), codes, scales, E * rows, K)
        packed = torch.empty(E * sw.swiglu_int8_packed_bytes(rows, K), device=DEV, dtype=torch.uint8)
        sw.swiglu_pack_int8_fragments(self.h, codes, packed, E, rows, K)
        return packed, scales, codes.view(E, rows, K)

    @staticmethod
    def _int8_rows(rows, K):
        return (torch.empty(rows, K, device=DEV, dtype=torch.int8), torch.empty(rows, device=DEV))

    @staticmethod
    def _codes(rows, K):
        return (torch.empty(sw.swiglu_mxfp4_bytes(rows, K), device=DEV, dtype=torch.uint8),
                torch.empty(sw.swiglu_mxfp4_scale_bytes(rows, K), device=DEV, dtype=torch.uint8))

    def __call__(self, X, H):
        """X is updated in place; returns the next block's H."""
        h, (T, E, k, D, N, NS) = self.h, self.size
        if self.int8:
            self._experts_int8(H)
        else:
            sw.swiglu_route(h, H.float() @ self.router, self.w, self.e, self.offsets, self.rows,
                            self.ws, T, E, k)
            sw.swiglu_grouped_forward(h, H, self.rows, self.offsets, self.up, self.gated, T, T * k, N,
                                      D, E, k=k)
            sw.swiglu_grouped_matmul(h, self.gated, self.rows, self.offsets, self.down, self.out,
                                     T * k, D, N, E)
        sw.swiglu_quantize_mxfp4(h, H, self.q, self.sq, T, D)
        sw.swiglu_forward_mxfp4(h, self.q, self.sq, self.w4, self.sw4, self.shared, T, NS, D)
        sw.swiglu_combine_norm(h, self.out, self.w, self.e, self.shared @ self.shared_down, X,
                               self.post, None, self.pre, X, self.H, T, D, k=k,
                               dtype=sw.DTYPE_F32)
        return self.H

    def _experts_int8(self, H):
        h, (T, E, k, D, N, _) = self.h, self.size
        sw.swiglu_route_scored(h, H.float() @ self.router, self.bias, self.w, self.e, self.offsets,
                               self.rows, self.ws, T, E, k, score=sw.SCORE_SIGMOID, scale=self.scale,
                               groups=self.groups, top_groups=self.top_groups,
                               group_best=min(2, E // self.groups))
        sw.swiglu_quantize_int8(h, H, self.q8, self.s8, T, D)
        sw.swiglu_grouped_forward_int8(h, self.q8, self.s8, self.rows, self.offsets, *self.up[:2],
                                       self.gated, T, T * k, N, D, E, k=k)
        sw.swiglu_quantize_int8(h, self.gated, self.q8_up, self.s8_up, T * k, N)
        sw.swiglu_grouped_matmul_int8(h, self.q8_up, self.s8_up, self.rows, self.offsets,
                                      *self.down[:2], self.out, T * k, D, N, E)

    @staticmethod
    def _rows_int8(a):
        """Rows a as their 8-bit codes times their scales: s = max|a| / 127, codes by rounding."""
        s = a.abs().amax(-1, keepdim=True) / 127
        return torch.round(a / s.clamp_min(1e-38)) * s

    def _weights(self, x):
        """Expert x's up and down weights in fp32, [K, rows]."""
        if not self.int8:
            return self.up[x].float(), self.down[x].float()
        return tuple((codes[x].float() * scales.view(len(codes), -1, 1)[x]).t()
                     for _, scales, codes in (self.up, self.down))

    def plain(self, X, H):
        """The same block in torch operations; experts as the library chose them."""
        T, E, k, D, N, NS = self.size
        logits, rows = H.float() @ self.router, H.float()
        scores = torch.sigmoid(logits) if self.int8 else torch.softmax(logits, -1)
        p = scores.gather(1, self.e.long())
        p = p / p.sum(-1, keepdim=True)
        if self.int8:
            p, rows = p * self.scale, self._rows_int8(rows)
        o = torch.zeros(T, D, device=DEV)
        for x in range(E):
            t, j = torch.nonzero(self.e == x, as_tuple=True)
            if t.numel():
                up, down = self._weights(x)
                a = rows[t] @ up
                a = (torch.nn.functional.silu(a[:, 0::2]) * a[:, 1::2]).to(BF16).float()
                a = self._rows_int8(a) if self.int8 else a
                o.index_add_(0, t, p[t, j, None] * (a @ down).to(BF16).float())
        a, w = torch.empty(T, D, device=DEV, dtype=BF16), torch.empty(2 * NS, D, device=DEV, dtype=BF16)
        sw.swiglu_dequantize_mxfp4(self.h, self.q, self.sq, a, T, D)
        sw.swiglu_dequantize_mxfp4(self.h, self.w4, self.sw4, w, 2 * NS, D)
        a = a.float() @ w.float().t()
        a = (torch.nn.functional.silu(a[:, 0::2]) * a[:, 1::2]).to(BF16)
        o = o + (a @ self.shared_down).float()
        x = X + torch.nn.functional.rms_norm(o, (D,), self.post.float(), 1e-6)
        return x, torch.nn.functional.rms_norm(x, (D,), self.pre.float(), 1e-6).to(BF16)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 1), ("experts", 64), ("top", 6), ("width", 1536),
                        ("expert-width", 896), ("shared-width", 1792), ("blocks", 2), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--int8", action="store_true", help="experts on 8-bit integers, scored router")
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    handle = sw.swiglu_create(0)
    try:
        blocks = [Block(handle, a.tokens, a.experts, a.top, a.width, a.expert_width, a.shared_width,
                        seed, a.int8) for seed in range(a.blocks)]
        g = torch.Generator(device=DEV).manual_seed(99)
        X0 = torch.randn(a.tokens, a.width, generator=g, device=DEV)
        H0 = torch.nn.functional.rms_norm(X0, (a.width,), eps=1e-6).to(BF16)
        X = X0.clone()

        def step():
            X.copy_(X0)
            H = H0
            for b in blocks:
                H = b(X, H)
            return H
        worst = 0.0
        if a.check:
            H = H0
            for b in blocks:
                before, out = X.clone(), b(X, H)
                x, want = b.plain(before, H)
                worst = max(worst, float((X - x).norm() / (x - before).norm()),
                            float((out.float() - want.float()).norm() / want.float().norm()))
                H = out
            print(f"against plain operations: relative error {worst:.2e}", flush=True)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        eager = X.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graph.replay()
        torch.cuda.synchronize()
        same = bool(torch.equal(X, eager))
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(a.steps):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"{a.tokens} tokens, {a.blocks} blocks of {a.experts} experts (top {a.top}), width "
              f"{a.width}: {start.elapsed_time(end) / a.steps * 1e3:.1f} us a step; replay equals "
              f"the eager step: {same}", flush=True)
        return {"error": worst, "same": same}
    finally:
        torch.cuda.synchronize()
        sw.swiglu_destroy(handle)


if __name__ == "__main__":
    main()
