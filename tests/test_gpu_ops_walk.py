"""Mixture-of-experts and MXFP4 launches in which one workgroup does several pieces of
work in turn: units of the grouped tiles (the stage ring refilled behind a unit's rows of
Y), tiles of the MXFP4 product (its ring runs on from tile to tile, an odd number of K
groups changing its halves' places), rounds of 64 slots a wave in the router's placing
launch; and what bad offsets and a replayed graph leave, every row of it."""
import numpy as np
import pytest
import torch

import gemm_epilogues_mlp_amd as sw
import ops_oracle as O
from test_gpu_moe import randn, run_route, spans
from test_gpu_mxfp4 import product

BF = torch.bfloat16


@pytest.fixture(scope="module")
def handle():
    h = sw.swiglu_create(0)
    yield h
    sw.swiglu_destroy(h)


# ------------------------------------------------------------------ grouped products
def units_a_workgroup(counts, ldw, bm, bnw, parts):
    """The most units that a workgroup of the tile kernel takes: the launch's arithmetic."""
    R, E, ntn = sum(counts), len(counts), -(-ldw // bnw)
    most = min(R, (R + min(R, E) * (bm - 1)) // bm) * ntn
    grid = -(-most * (2 if parts > 1 and most < 1024 else 1) // 8) * 8

    def work(n):
        left = -(-(n % bm) // (bm // parts))
        return n // bm * (2 * parts + 3) + (2 * left + 3 if left else 0)
    p = [work(n) * ntn for n in counts]
    t = [-(-n // bm) * ntn for n in counts]
    cuts = []
    for x in range(8):
        at, before, units, cut = sum(p) * x // 8, 0, 0, sum(t)
        for pe, te in zip(p, t):
            if before + pe > at:
                cut = units + (at - before) * te // pe
                break
            before, units = before + pe, units + te
        cuts.append(cut)
    cuts.append(sum(t))
    return max(-(-(b - a) // (grid // 8)) for a, b in zip(cuts, cuts[1:]))


# Few experts with whole tiles and one row more, many with a single row: the bound that the
# grid comes from is met, and an XCD whose share is short tiles has more than an eighth
WALKS = [(2, 128, 128, 2, [513] * 8 + [1] * 60, 2048), (3, 256, 256, 4, [1025] * 8 + [1] * 40, 4080)]


def test_the_walks_are_walks():
    for _, bm, bnw, parts, counts, ldw in WALKS:
        assert units_a_workgroup(counts, ldw, bm, bnw, parts) > 1
    assert units_a_workgroup([130, 1, 0, 257, 40], 528, 128, 128, 2) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("K", [32, 72, 200])
@pytest.mark.parametrize("case", WALKS, ids=lambda c: f"variant{c[0]}")
def test_grouped_workgroups_take_several_units(handle, case, K):
    variant, _, _, _, counts, ldw = case
    # short and whole tiles mixed along the sorted rows
    counts = [counts[i] for i in torch.randperm(len(counts), generator=torch.Generator().manual_seed(1))]
    R, off, rows = spans(counts, K)
    E, N, n = len(counts), ldw // 2, sum(counts)
    print(f"walk variant {variant} K={K}: {R} rows, {E} experts", flush=True)
    A, W = randn(1, R, K), randn(2, E, K, ldw, std=K ** -0.5)
    Y = torch.full((R + 1, N), -7.0, dtype=BF, device="cuda")
    sw.swiglu_grouped_forward(handle, A.cuda(), rows.cuda(), off.cuda(), W.cuda(), Y, R, R, N, K, E,
                              variant=variant)
    D = torch.full((R + 1, ldw), -7.0, dtype=BF, device="cuda")
    sw.swiglu_grouped_matmul(handle, A.cuda(), rows.cuda(), off.cuda(), W.cuda(), D, R, ldw, K, E,
                             variant=variant)
    torch.cuda.synchronize()
    assert bool((Y[n:] == -7.0).all()) and bool((D[n:] == -7.0).all())
    Y, D = Y.cpu(), D.cpu()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        O.assert_close(Y[r], *O.gated(A[rows[r].long()], W[e]), f"up expert {e}")
        O.assert_close(D[rows[r].long()], *O.plain(A[r], W[e]), f"down expert {e}")


@pytest.mark.gpu
@pytest.mark.parametrize("variant", range(5))
def test_bad_offsets_leave_whole_spans(handle, variant):
    """An offset below an earlier one counts as that one: [-5, 20, 10, 90] over 50 rows is
    [0, 20), none, [20, 50), every row with its own expert's weights."""
    R, N, K = 50, 72, 40
    off = torch.tensor([-5, 20, 10, 90], dtype=torch.int32)
    rows = torch.arange(R, dtype=torch.int32)
    A, W = randn(1, R, K), randn(2, 3, K, 2 * N, std=K ** -0.5)
    Y = torch.full((R + 8, N), -7.0, dtype=BF, device="cuda")
    sw.swiglu_grouped_forward(handle, A.cuda(), rows.cuda(), off.cuda(), W.cuda(), Y, R, R, N, K, 3,
                              variant=variant)
    torch.cuda.synchronize()
    assert bool((Y[R:] == -7.0).all())
    O.assert_close(Y[:20], *O.gated(A[:20], W[0]), "expert 0")
    O.assert_close(Y[20:R], *O.gated(A[20:], W[2]), "expert 2")


# ----------------------------------------------------------------------------- MXFP4
@pytest.mark.gpu
@pytest.mark.parametrize("K", [32, 288, 768])  # 1 group of K, 2, and 3
@pytest.mark.parametrize("variant,bm,bn,places", [(2, 128, 64, 2), (3, 256, 128, 1)])
def test_mxfp4_ring_runs_on_from_tile_to_tile(handle, variant, bm, bn, places, K):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    M = 2000
    N = bn * -(-(cus * places * 5 // 4) // -(-M // bm)) + 8
    assert -(-M // bm) * -(-N // bn) > cus * places
    print(f"mxfp4 walk {M}x{N}x{K} variant {variant}", flush=True)
    y, (want, slack) = product(handle, M, N, K, variant, 21)
    O.assert_close(y, want, slack, f"{M}x{N}x{K} variant {variant}")


# ---------------------------------------------------------------------------- router
def route_many(logits, k, renorm):
    """ops_oracle.route for many tokens: sorts in place of its loops."""
    x = logits.to(torch.float64).numpy()
    T, E = x.shape
    v = np.where(np.isnan(x), -np.inf, x)
    e = np.argsort(-v, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(v, e, 1)
    there = top > -np.inf
    m = np.where(there[:, :1], top[:, :1], 0.0)
    p = np.where(there, np.exp(np.where(there, top, 0.0) - m), 0.0)
    total = p.sum(1, keepdims=True) if renorm else np.exp(v - m).sum(1, keepdims=True)
    w = np.where(there, p / np.where(total > 0, total, 1.0), 0.0)
    e = np.where(there, e, -1)
    key = np.where(there, e, E).reshape(-1)
    rows = np.argsort(key, kind="stable")
    offsets = np.zeros(E + 1, dtype=np.int64)
    offsets[1:] = np.cumsum(np.bincount(key, minlength=E + 1)[:E])
    rows[offsets[E]:] = -1
    return w, e, offsets, rows


def masked_logits(T, E, k, dtype):
    g = torch.Generator().manual_seed(T + E + k)
    x = torch.randn(T, E, generator=g) * 1.5
    off = (torch.rand(T, E, generator=g) < 0.1) | (torch.rand(T, 1, generator=g) < 0.1)
    return torch.where(off, float("-inf"), x).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["f32", "bf16"])
def test_route_many_is_the_definition(dtype):
    for T, E, k in ((60, 12, 5), (40, 70, 3), (9, 4, 4)):
        x = masked_logits(T, E, k, dtype)
        for renorm in (False, True):
            for a, b in zip(route_many(x, k, renorm), O.route(x, k, renorm)):
                assert np.allclose(a, b, rtol=1e-14, atol=0)


# 2192 slots a workgroup of 16 waves; more than 64 and 32 workgroups of tokens with 500 and
# 1000 experts, whose counts a workgroup adds up 64 and 32 at a time
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(70000, 64, 8), (40001, 250, 30), (5000, 500, 3), (3001, 1000, 40)])
def test_route_many_slots(handle, T, E, k, dtype):
    x = masked_logits(T, E, k, dtype)
    for renorm in (False, True):
        print(f"route {T}x{E} k={k} {dtype} renorm={renorm}", flush=True)
        w, e, off, rows = run_route(handle, x, k, renorm)
        W, X, OFF, ROWS = route_many(x, k, renorm)
        assert np.array_equal(e.numpy(), X)
        assert np.array_equal(off.numpy(), OFF)
        assert np.array_equal(rows.numpy(), ROWS)
        # terms within |x - m| + 2 steps of exp, a sum of E of them, a division
        most = float(x[torch.isfinite(x)].abs().max())
        want = torch.from_numpy(W)
        O.assert_close(w, want, (2 * most + E + 8) * O.U32 * want, "weights", half=O.U32)


# ----------------------------------------------------------------------------- graph
@pytest.mark.gpu
def test_a_replay_runs_every_operator(handle):
    """Every output of the block poisoned before a replay, the router's among them."""
    T, E, k, D, N = 600, 6, 2, 72, 40
    x, X = randn(1, T, E, dtype=torch.float32).cuda(), randn(2, T, D).cuda()
    Wu, Wd = randn(3, E, D, 2 * N, std=0.1).cuda(), randn(4, E, N, D, std=0.1).cuda()
    pre = torch.ones(D, dtype=BF, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    w, e = torch.empty(T, k, device="cuda"), torch.empty(T, k, **i32)
    off, rows = torch.empty(E + 1, **i32), torch.empty(T * k, **i32)
    ws = torch.empty(sw.swiglu_route_workspace_bytes(T, E, k), dtype=torch.uint8, device="cuda")
    up, down = torch.empty(T * k, N, dtype=BF, device="cuda"), torch.empty(T * k, D, dtype=BF, device="cuda")
    out, H = torch.empty_like(X), torch.empty_like(X)
    results = (w, e, off, rows, up, down, out, H)

    def step():
        sw.swiglu_route(handle, x, w, e, off, rows, ws, T, E, k)
        sw.swiglu_grouped_forward(handle, X, rows, off, Wu, up, T, T * k, N, D, E, k=k)
        sw.swiglu_grouped_matmul(handle, up, rows, off, Wd, down, T * k, D, N, E)
        sw.swiglu_combine_norm(handle, down, w, e, None, X, None, None, pre, out, H, T, D, k=k)

    def poison():
        for t in results:
            t.fill_(float("nan") if t.is_floating_point() else -9)
        ws.fill_(0xEE)
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    eager = [t.clone() for t in results]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(4):
        poison()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, results))
