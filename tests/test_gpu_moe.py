"""The mixture-of-experts operators on the GPU against their 64-bit definitions:
routing, products grouped by expert (every kernel variant), the combining norm;
masks that leave nothing, empty and single-row experts, odd sizes, dropped
slots, bad offsets and slots, refusals, streams and graphs."""
import numpy as np
import pytest
import torch

import gemm_epilogues_mlp_amd as sw
import ops_oracle as O

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def handle():
    h = sw.swiglu_create(0)
    yield h
    sw.swiglu_destroy(h)


def randn(seed, *shape, std=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


# ------------------------------------------------------------------------------ router
def run_route(handle, x, k, renorm, stream=None):
    T, E = x.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    e, off, rows = torch.full((T, k), -9, **i32), torch.full((E + 1,), -9, **i32), \
        torch.full((T * k,), -9, **i32)
    ws = torch.randint(0, 255, (sw.swiglu_route_workspace_bytes(T, E, k),), dtype=torch.uint8,
                       device="cuda")
    sw.swiglu_route(handle, x.cuda(), w, e, off, rows, ws, T, E, k, renormalize=renorm,
                    dtype=sw.DTYPE_F32 if x.dtype == torch.float32 else sw.DTYPE_BF16)
    torch.cuda.synchronize()
    return w.cpu(), e.cpu(), off.cpu(), rows.cpu()


def check_route(handle, x, k, renorm, what):
    w, e, off, rows = run_route(handle, x, k, renorm)
    W, X, OFF, ROWS = O.route(x, k, renorm)
    assert np.array_equal(e.numpy(), X), what
    assert np.array_equal(off.numpy(), OFF), what
    assert np.array_equal(rows.numpy(), ROWS), what
    # terms within |x - m| + 2 steps of exp, a sum of E of them, a division
    want = torch.from_numpy(W)
    fin = x.to(torch.float64)
    fin = torch.where(torch.isfinite(fin), fin, torch.zeros(())).abs().amax().item() if x.numel() else 0
    slack = (min(2 * fin, 200.0) + x.shape[1] + 8) * O.U32 * want
    O.assert_close(w, want, slack, what, half=O.U32)


@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 6), (3, 5, 5), (17, 8, 1), (64, 60, 8),
                                   (65, 64, 8), (200, 72, 4), (513, 128, 8), (1000, 200, 3),
                                   (333, 256, 8), (130, 500, 17), (90, 1000, 64), (5000, 160, 2),
                                   (128, 100, 32)])
def test_route(handle, T, E, k, dtype):
    for renorm in (False, True):
        print(f"route {T}x{E} k={k} {dtype} renorm={renorm}", flush=True)
        x = randn(T + E + k, T, E, std=1.5, dtype=torch.float32)
        off = torch.rand(T, E, generator=torch.Generator().manual_seed(T)) < 0.1
        off |= torch.rand(T, 1, generator=torch.Generator().manual_seed(E)) < 0.1
        x = torch.where(off, float("-inf"), x).to(dtype)
        check_route(handle, x, k, renorm, f"{T}x{E} k={k} {dtype} renorm={renorm}")


def test_route_unaligned_rows(handle):
    x = randn(2, 40 * 64 + 1, dtype=torch.float32)
    flat = x.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    w, e = torch.empty(40, 4, device="cuda"), torch.empty(40, 4, **i32)
    off, rows = torch.empty(65, **i32), torch.empty(160, **i32)
    sw.swiglu_route(handle, flat[1:], w, e, off, rows, None, 40, 64, 4)
    torch.cuda.synchronize()
    assert np.array_equal(e.cpu().numpy(), O.route(x[1:].view(40, 64), 4, True)[1])


def test_route_special_logits(handle):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(BF).min
    rows = [[-inf] * 6, [nan] * 6, [nan, 1, -inf, 2, nan, 0], [inf, 1, inf, 2, 0, -inf],
            [low] * 6, [low, -inf, low, nan, -inf, -inf], [0.0, -0.0, 0.0, -0.0, 0.0, 0.0],
            [3, 3, 3, 1, 3, 3], [100, -100, 0, 100, -100, 0]]
    for dtype in (torch.float32, BF):
        x = torch.tensor(rows, dtype=dtype)
        for renorm in (False, True):
            for k in (1, 3, 6):
                check_route(handle, x, k, renorm, f"{dtype} {renorm} {k}")


def test_route_no_tokens(handle):
    _, _, off, _ = run_route(handle, torch.zeros(0, 12), 2, True)
    assert bool((off == 0).all())


def test_route_repeats(handle):
    x = randn(9, 4000, 64, dtype=BF)
    first = run_route(handle, x, 6, True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, run_route(handle, x, 6, True)))


# ---------------------------------------------------------------------- grouped products
def spans(counts, seed, drop=0):
    """offsets and rows of experts with these counts over R = sum + drop slots."""
    R = sum(counts) + drop
    perm = torch.randperm(R, generator=torch.Generator().manual_seed(seed))
    rows, at = torch.full((R,), -1, dtype=torch.int32), 0
    for n in counts:
        rows[at:at + n] = perm[at:at + n].sort().values.int()
        at += n
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    return R, off, rows


COUNTS = {"ones": [1, 1, 1], "empty": [0, 3, 0, 0, 17, 0], "tile": [16, 64, 0, 33],
          "ragged": [130, 1, 0, 257, 40], "none": [0, 0], "half": [384, 129],
          "many": [2] * 70 + [0] * 5 + [1, 5]}
UP_SHAPES = [(8, 8), (72, 40), (136, 200), (264, 520)]


@pytest.mark.parametrize("variant", [-1, 0, 1, 2, 3, 4])
@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("N,K", UP_SHAPES)
def test_grouped(handle, N, K, name, variant):
    counts, k = COUNTS[name], 3
    print(f"grouped {name} N={N} K={K} variant {variant}", flush=True)
    R, off, rows = spans(counts, N + K, drop=5)
    E, T = len(counts), -(-R // k)
    # up
    A, W = randn(1, T, K), randn(2, E, K, 2 * N, std=K ** -0.5)
    Y = torch.full((R + 1, N), -7.0, dtype=BF, device="cuda")
    sw.swiglu_grouped_forward(handle, A.cuda(), rows.cuda(), off.cuda(), W.cuda(), Y, T, R, N, K,
                              E, k=k, variant=variant)
    torch.cuda.synchronize()
    n = sum(counts)
    assert bool((Y[n:] == -7.0).all()), "wrote past the spans"
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if counts[e]:
            want, slack = O.gated(A[rows[r].long() // k], W[e])
            O.assert_close(Y[r], want, slack, f"up expert {e}")
    # down
    A, W = randn(3, R, K), randn(4, E, K, N, std=K ** -0.5)
    Y = torch.full((R, N), -7.0, dtype=BF, device="cuda")
    sw.swiglu_grouped_matmul(handle, A.cuda(), rows.cuda(), off.cuda(), W.cuda(), Y, R, N, K, E,
                             variant=variant)
    torch.cuda.synchronize()
    seen = torch.zeros(R, dtype=torch.bool)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if counts[e]:
            want, slack = O.plain(A[r], W[e])
            O.assert_close(Y[rows[r].long().cuda()], want, slack, f"down expert {e}")
            seen[rows[r].long()] = True
    assert bool((Y.cpu()[~seen] == -7.0).all()), "wrote a slot of no span"


@pytest.mark.parametrize("variant", range(5))
def test_rows_of_other_experts_do_not_leak(handle, variant):
    """NaN everywhere but in the rows and weights of one expert."""
    R, off, rows = spans([40, 70, 30], 3)
    N, K = 136, 72
    A, W = randn(1, R, K), randn(2, 3, K, 2 * N, std=K ** -0.5)
    A[rows[:40].long()] = float("nan")
    A[rows[110:].long()] = float("nan")
    W[0] = W[2] = float("nan")
    Y = torch.zeros(R, N, dtype=BF, device="cuda")
    sw.swiglu_grouped_forward(handle, A.cuda(), rows.cuda(), off.cuda(), W.cuda(), Y, R, R, N, K, 3,
                              variant=variant)
    torch.cuda.synchronize()
    want, slack = O.gated(A[rows[40:110].long()], W[1])
    O.assert_close(Y[40:110], want, slack, "leak")


@pytest.mark.parametrize("variant", range(5))
def test_bad_offsets_and_slots_stay_inside(handle, variant):
    """Offsets past R are held to it, slots that name no row give zeros (up) or are not
    written (down)."""
    R, N, K = 50, 72, 40
    off = torch.tensor([-5, 20, 10, 90], dtype=torch.int32)  # spans [0,20), none, [10,50)
    rows = torch.arange(R, dtype=torch.int32)
    rows[30], rows[31], rows[32] = -1, R, 2 ** 31 - 1
    A, W = randn(1, R, K), randn(2, 3, K, 2 * N, std=K ** -0.5)
    Y = torch.full((R + 8, N), -7.0, dtype=BF, device="cuda")
    sw.swiglu_grouped_forward(handle, A.cuda(), rows.cuda(), off.cuda(), W.cuda(), Y, R, R, N, K, 3,
                              variant=variant)
    torch.cuda.synchronize()
    assert bool((Y[R:] == -7.0).all()) and bool((Y[30:33] == 0).all())
    want, slack = O.gated(A[33:], W[2])
    O.assert_close(Y[33:R], want, slack, "after the bad slots")
    off = torch.tensor([0, 20, 20, 90], dtype=torch.int32)
    W = randn(2, 3, K, N, std=K ** -0.5)
    Y = torch.full((R + 8, N), -7.0, dtype=BF, device="cuda")
    sw.swiglu_grouped_matmul(handle, A.cuda(), rows.cuda(), off.cuda(), W.cuda(), Y, R, N, K, 3,
                             variant=variant)
    torch.cuda.synchronize()
    assert bool((Y[R:] == -7.0).all()) and bool((Y[30:33] == -7.0).all())
    want, slack = O.plain(A[33:], W[2])
    O.assert_close(Y[33:R], want, slack, "down")


@pytest.mark.parametrize("variant", range(5))
def test_overlapping_offsets_count_once(handle, variant):
    """An offset below an earlier one counts as that one: every row has one expert, and the
    units never exceed those of R rows."""
    R, N, K, E = 300, 72, 40, 100
    off = torch.full((E + 1,), R, dtype=torch.int32)
    off[0::2] = 0                              # taken as they are: 50 spans of all rows
    off[:4] = torch.tensor([0, 40, 10, 30])
    off[4] = 170
    ends = np.maximum.accumulate(np.clip(off.numpy(), 0, R))
    rows = torch.arange(R, dtype=torch.int32)
    A, W = randn(1, R, K), randn(2, E, K, 2 * N, std=K ** -0.5)
    Y = torch.full((R, N), -7.0, dtype=BF, device="cuda")
    sw.swiglu_grouped_forward(handle, A.cuda(), rows.cuda(), off.cuda(), W.cuda(), Y, R, R, N, K, E,
                              variant=variant)
    torch.cuda.synchronize()
    for e in range(E):
        a, b = int(ends[e]), int(ends[e + 1])
        if b > a:
            want, slack = O.gated(A[a:b], W[e])
            O.assert_close(Y[a:b], want, slack, f"expert {e}")


def test_weights_past_4_gib(handle):
    """The last expert of a stack whose byte offsets pass 32 bits."""
    E, N, K = 40, 4096, 8192
    W = torch.empty(E, K, 2 * N, dtype=BF, device="cuda")
    assert W.numel() * 2 > 2 ** 32
    w = randn(5, K, 2 * N, std=K ** -0.5)
    W[E - 1] = w.cuda()
    for R, variant in ((3, 0), (3, 2), (3, 3), (3, 4)):
        off = torch.zeros(E + 1, dtype=torch.int32)
        off[E] = R
        A = randn(6, R, K)
        Y = torch.zeros(R, N, dtype=BF, device="cuda")
        sw.swiglu_grouped_forward(handle, A.cuda(), torch.arange(R, dtype=torch.int32).cuda(),
                                  off.cuda(), W, Y, R, R, N, K, E, variant=variant)
        torch.cuda.synchronize()
        want, slack = O.gated(A, w)
        O.assert_close(Y, want, slack, f"variant {variant}")


def test_grouped_empty_sizes(handle):
    sw.swiglu_grouped_forward(handle, None, None, None, None, None, 0, 0, 8, 8, 4)
    Y = torch.full((2, 8), 3.0, dtype=BF, device="cuda")
    off, rows = torch.tensor([0, 2], dtype=torch.int32).cuda(), torch.tensor([1, 0], dtype=torch.int32).cuda()
    for variant in range(5):
        Y.fill_(3.0)
        sw.swiglu_grouped_matmul(handle, None, rows, off, None, Y, 2, 8, 0, 1, variant=variant)
        torch.cuda.synchronize()
        assert bool((Y == 0).all())  # empty sums


# ---------------------------------------------------------------------- combining norm
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,D,k", [(1, 8, 1), (3, 64, 2), (5, 520, 3), (1, 3584, 6), (9, 1536, 8),
                                   (1030, 512, 1), (1029, 1000, 5), (1025, 1536, 8), (1024, 2048, 2),
                                   (2, 4096, 4), (3, 4104, 7), (2, 8192, 9), (2, 16384, 3),
                                   (6, 72, 0)])
def test_combine_norm(handle, T, D, k, dtype):
    for opt in range(4):
        print(f"norm {T}x{D} k={k} {dtype} options {opt}", flush=True)
        shared, post, gate = bool(opt & 1) or k == 0, bool(opt & 2), opt
        B = randn(1, T, k, D, std=0.5)
        w = torch.softmax(randn(2, T, max(k, 1), dtype=torch.float32), -1)[:, :k].contiguous()
        e = torch.randint(0, 9, (T, k), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
        lost = torch.rand(T, k, generator=torch.Generator().manual_seed(4)) < 0.2
        if k and T > 1:
            lost[0] = True  # a token with no expert left
        e = torch.where(lost, -1, e)
        w = torch.where(lost, float("nan"), w)
        B[lost] = float("nan")
        S = randn(5, T, D, std=0.5) if shared else None
        p = randn(6, D, std=0.2) + 1 if post else None
        ld = D + 8
        gt = {0: None, 1: None, 2: randn(7, D, std=0.3) + 1, 3: randn(8, T, ld, std=0.5)}[gate]
        pre, X = randn(9, D, std=0.2) + 1, randn(10, T, D, std=2.0, dtype=dtype)
        Xg = X.cuda()
        out = Xg if opt == 1 else torch.empty_like(Xg)  # once in place
        H = torch.empty(T, D, dtype=BF, device="cuda")
        c = lambda t: None if t is None else t.cuda()
        sw.swiglu_combine_norm(handle, c(B), c(w), c(e), c(S), Xg, c(p), c(gt), c(pre), out, H, T,
                               D, k=k, scale=0.7, eps=1e-5, gate_ld=ld if gate == 3 else 0,
                               dtype=sw.DTYPE_F32 if dtype == torch.float32 else sw.DTYPE_BF16)
        torch.cuda.synchronize()
        g = gt[:, :D] if gate == 3 else gt
        scale, eps = float(np.float32(0.7)), float(np.float32(1e-5))
        x, ex, h, eh = O.combine_norm(B, w, e, S, X, p, g, pre, scale, eps)
        O.assert_close(out, x, ex, f"x options {opt}", half=O.U32 if dtype == torch.float32 else O.HALF_BF16)
        O.assert_close(H, h, eh, f"h options {opt}")


# ------------------------------------------------------------------- refusals, streams
def test_refusals_write_nothing(handle):
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")
    i32 = torch.int32
    A, W, Y = z(8, 16), z(2, 16, 32), torch.full((8, 16), 3.0, dtype=BF, device="cuda")
    rows, off = z(8, dtype=i32), z(3, dtype=i32)
    gf = lambda **o: sw.swiglu_grouped_forward(
        handle, o.get("A", A), o.get("rows", rows), o.get("off", off), o.get("W", W), o.get("Y", Y),
        o.get("T", 8), o.get("R", 8), o.get("N", 16), o.get("K", 16), o.get("E", 2),
        k=o.get("k", 1), variant=o.get("variant", -1))
    bad = [(dict(A=None), 1), (dict(rows=None), 1), (dict(off=None), 1), (dict(W=None), 1),
           (dict(Y=None), 1), (dict(Y=A), 1), (dict(k=0), 1), (dict(E=0), 1), (dict(R=-1), 1),
           (dict(variant=5), 1), (dict(N=12), 2), (dict(K=12), 2), (dict(E=2000), 2),
           (dict(A=A.view(-1)[4:]), 2), (dict(T=2 ** 27), 2)]
    for o, status in bad:
        with pytest.raises(sw.SwiGLUError) as err:
            gf(**o)
        assert err.value.status == status, o
    x, w, e = z(4, 8, dtype=torch.float32), z(4, 2, dtype=torch.float32), z(4, 2, dtype=i32)
    of, r = z(9, dtype=i32), z(8, dtype=i32)
    rt = lambda **o: sw.swiglu_route(handle, o.get("x", x), o.get("w", w), e, o.get("of", of), r,
                                     None, o.get("T", 4), o.get("E", 8), o.get("k", 2),
                                     dtype=o.get("dtype", 1))
    for o, status in [(dict(x=None), 1), (dict(w=None), 1), (dict(of=None), 1), (dict(k=9), 1),
                      (dict(k=0), 1), (dict(E=0), 1), (dict(T=-1), 1), (dict(dtype=2), 1),
                      (dict(T=10 ** 6), 1), (dict(E=2000, k=2), 2), (dict(w=x), 1)]:
        with pytest.raises(sw.SwiGLUError) as err:
            rt(**o)
        assert err.value.status == status, o
    v = z(16)
    nm = lambda **o: sw.swiglu_combine_norm(
        handle, o.get("B", A), o.get("w", z(8, dtype=torch.float32)), o.get("e", rows), None, A,
        None, o.get("gate"), o.get("pre", v), o.get("out", Y), o.get("H", z(8, 16)), o.get("T", 8),
        o.get("D", 16), k=1, gate_ld=o.get("ld", 0))
    for o, status in [(dict(B=None), 1), (dict(w=None), 1), (dict(e=None), 1), (dict(pre=None), 1),
                      (dict(out=None), 1), (dict(H=Y), 1), (dict(H=A), 1), (dict(D=12), 2),
                      (dict(D=20000), 2), (dict(gate=v, ld=8), 1), (dict(T=-1), 1),
                      (dict(gate=z(8, 20), ld=20), 2)]:
        with pytest.raises(sw.SwiGLUError) as err:
            nm(**o)
        assert err.value.status == status, o
    torch.cuda.synchronize()
    assert bool((Y == 3.0).all())


def test_block_on_a_side_stream_and_in_a_graph(handle):
    """Router, products and norm in order on one stream; captured, replayed with eager work
    between, every replay equal to the eager result."""
    T, E, k, D, N = 37, 6, 2, 72, 40
    x, Xr = randn(1, T, E, dtype=torch.float32).cuda(), randn(2, T, D).cuda()
    Wu, Wd = randn(3, E, D, 2 * N, std=0.1).cuda(), randn(4, E, N, D, std=0.1).cuda()
    pre = torch.ones(D, dtype=BF, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    w, e = torch.empty(T, k, device="cuda"), torch.empty(T, k, **i32)
    off, rows = torch.empty(E + 1, **i32), torch.empty(T * k, **i32)
    up, down = torch.empty(T * k, N, dtype=BF, device="cuda"), torch.empty(T * k, D, dtype=BF, device="cuda")
    out, H = torch.empty_like(Xr), torch.empty_like(Xr)

    def step():
        sw.swiglu_route(handle, x, w, e, off, rows, None, T, E, k)
        sw.swiglu_grouped_forward(handle, Xr, rows, off, Wu, up, T, T * k, N, D, E, k=k)
        sw.swiglu_grouped_matmul(handle, up, rows, off, Wd, down, T * k, D, N, E)
        sw.swiglu_combine_norm(handle, down, w, e, None, Xr, None, None, pre, out, H, T, D, k=k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    eager = [t.clone() for t in (w, e, off, rows, up, down, out, H)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(4):
        for t in (up, down, out, H):
            t.fill_(-1)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, (w, e, off, rows, up, down, out, H)))
