"""A mixture-of-experts block on the library's operators, end to end.

    python examples/moe_block.py [--tokens 1 --experts 64 --top 6 --width 1536 --expert-width 896
                                  --shared-width 1792 --blocks 2 --check]

Every block takes the residual stream X and its normed form H:

    logits         = H Wr                                       torch, fp32
    e, w, spans    = swiglu_route(logits)
    up             = swiglu_grouped_forward(H, ...)             experts, gated
    down           = swiglu_grouped_matmul(up, ...)
    S              = swiglu_forward_mxfp4(quantised H) Ws       the shared expert, 4 bits
    X, H           = swiglu_combine_norm(down, w, e, S, X, ...)

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

    def __init__(self, handle, T, E, k, D, N, NS, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def randn(*shape, std):
            return torch.randn(*shape, generator=g, device=DEV).mul_(std).to(BF16)
        self.h, self.size = handle, (T, E, k, D, N, NS)
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

    @staticmethod
    def _codes(rows, K):
        return (torch.empty(sw.swiglu_mxfp4_bytes(rows, K), device=DEV, dtype=torch.uint8),
                torch.empty(sw.swiglu_mxfp4_scale_bytes(rows, K), device=DEV, dtype=torch.uint8))

    def __call__(self, X, H):
        """X is updated in place; returns the next block's H."""
        h, (T, E, k, D, N, NS) = self.h, self.size
        sw.swiglu_route(h, H.float() @ self.router, self.w, self.e, self.offsets, self.rows,
                        self.ws, T, E, k)
        sw.swiglu_grouped_forward(h, H, self.rows, self.offsets, self.up, self.gated, T, T * k, N,
                                  D, E, k=k)
        sw.swiglu_grouped_matmul(h, self.gated, self.rows, self.offsets, self.down, self.out, T * k,
                                 D, N, E)
        sw.swiglu_quantize_mxfp4(h, H, self.q, self.sq, T, D)
        sw.swiglu_forward_mxfp4(h, self.q, self.sq, self.w4, self.sw4, self.shared, T, NS, D)
        sw.swiglu_combine_norm(h, self.out, self.w, self.e, self.shared @ self.shared_down, X,
                               self.post, None, self.pre, X, self.H, T, D, k=k,
                               dtype=sw.DTYPE_F32)
        return self.H

    def plain(self, X, H):
        """The same block in torch operations; experts as the library chose them."""
        T, E, k, D, N, NS = self.size
        p = torch.softmax(H.float() @ self.router, -1).gather(1, self.e.long())
        p = p / p.sum(-1, keepdim=True)
        o = torch.zeros(T, D, device=DEV)
        for x in range(E):
            t, j = torch.nonzero(self.e == x, as_tuple=True)
            if t.numel():
                a = H[t].float() @ self.up[x].float()
                a = (torch.nn.functional.silu(a[:, 0::2]) * a[:, 1::2]).to(BF16).float()
                o.index_add_(0, t, p[t, j, None] * (a @ self.down[x].float()).to(BF16).float())
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
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    handle = sw.swiglu_create(0)
    try:
        blocks = [Block(handle, a.tokens, a.experts, a.top, a.width, a.expert_width, a.shared_width,
                        seed) for seed in range(a.blocks)]
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
