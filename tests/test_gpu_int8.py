"""The 8-bit integer operators on the GPU against their 64-bit definitions: quantisation (ties,
rows of zeros, infinities, the smallest and largest values), packing, dense and grouped products in
every kernel variant, refusals, streams and graphs, and a block of them together."""
import numpy as np
import pytest
import torch

import gemm_epilogues_mlp_amd as sw
import more_oracle as M
import ops_oracle as O

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
VARIANTS = [-1, *range(8)]


@pytest.fixture(scope="module")
def handle():
    h = sw.swiglu_create(0)
    yield h
    sw.swiglu_destroy(h)


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------------- quantisation
def run_quantize(handle, x):
    rows, K = x.shape
    q = torch.full((rows, K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows,), -7.0, device="cuda")
    sw.swiglu_quantize_int8(handle, x.cuda(), q, s, rows, K)
    torch.cuda.synchronize()
    return q.cpu(), s.cpu()


def check_quantize(handle, x, what):
    q, s = run_quantize(handle, x)
    Q, S = M.quantize(x)
    assert np.array_equal(q.numpy(), Q), what
    bad = np.isnan(S)
    assert np.array_equal(np.isnan(s.numpy()), bad), what
    want = torch.from_numpy(S[~bad])
    O.assert_close(s[~bad], want, torch.zeros_like(want), what, half=O.U32)


@pytest.mark.parametrize("rows,K", [(1, 16), (5, 512), (3, 528), (2, 1024), (7, 1040), (2, 2048),
                                    (3, 2064), (2, 4112), (2, 8192), (1, 8208), (1, 16400),
                                    (1, 32768), (1, 32784), (1, 131056)])
def test_quantize(handle, rows, K):
    print(f"quantize {rows}x{K}", flush=True)
    x = torch.randn(rows, K, generator=gen(K)) * torch.exp(2 * torch.randn(rows, 1, generator=gen(rows)))
    check_quantize(handle, x.to(BF), f"{rows}x{K}")


def test_quantize_ties(handle):
    """Every half of a step is met exactly with a = 254 2^e: the even code is taken."""
    x = torch.arange(-254, 255, dtype=torch.float32).repeat(2)[:1008]
    x = torch.cat([torch.tensor([254.0] * 16), x]).view(1, 1024)
    for e in (0, 20, -40, 110, -125, -130):
        check_quantize(handle, torch.ldexp(x, torch.tensor(e)).to(BF), f"2^{e}")


def test_quantize_every_significand(handle):
    """All 8-bit significands over four binades against each of 128 largest values."""
    m = torch.arange(128, 256, dtype=torch.float32)
    v = torch.cat([m / 2.0 ** b for b in range(8)])
    x = torch.stack([torch.cat([a.view(1), torch.minimum(v, a), torch.zeros(15)]) for a in m])
    check_quantize(handle, x.to(BF), "significands")


def test_quantize_special_rows(handle):
    inf, nan, big, small = float("inf"), float("nan"), torch.finfo(BF).max, 2.0 ** -133
    rows = [[0.0] * 16, [-0.0] * 16, [inf] + [1.0] * 15, [1.0, -inf] + [0.0] * 14, [nan] * 16,
            [0.0] * 15 + [nan], [big, -big, big / 2, 1.0] + [0.0] * 12, [small] * 8 + [-small] * 8,
            [small * 127, small, small * 3, -small * 64] + [0.0] * 12, [1.0, small] * 8,
            [2.0 ** -60, 2.0 ** -61] * 8, [2.0 ** 60, 2.0 ** 53] * 8, [2.0 ** 61, 2.0 ** 60] * 8]
    check_quantize(handle, torch.tensor(rows, dtype=torch.float64).to(BF), "special")


# ----------------------------------------------------------------------------- packing
@pytest.mark.parametrize("E,rows,K", [(1, 1, 16), (1, 32, 128), (3, 40, 144), (2, 257, 400)])
def test_pack(handle, E, rows, K):
    w = torch.randint(-128, 128, (E, rows, K), generator=gen(K), dtype=torch.int8)
    n = sw.swiglu_int8_packed_bytes(rows, K)
    p = torch.full((E * n + 64,), 55, dtype=torch.int8, device="cuda")
    sw.swiglu_pack_int8_fragments(handle, w.cuda(), p, E, rows, K)
    torch.cuda.synchronize()
    assert np.array_equal(p[:E * n].cpu().numpy(), M.fragments(w.numpy()))
    assert bool((p[E * n:] == 55).all())


# ---------------------------------------------------------------------------- products
def codes(seed, *shape):
    return torch.randint(-127, 128, shape, generator=gen(seed), dtype=torch.int8)


def scales(seed, *shape, mid):
    return torch.exp(0.5 * torch.randn(*shape, generator=gen(seed))) * mid


def pack(handle, w):
    E, rows, K = w.shape
    p = torch.empty(E * sw.swiglu_int8_packed_bytes(rows, K), dtype=torch.int8, device="cuda")
    sw.swiglu_pack_int8_fragments(handle, w.cuda(), p, E, rows, K)
    return p


def dense_inputs(m, n, k, gated):
    C = 2 * n if gated else n
    # products of order 1
    return codes(m + k, m, k), scales(m, m, mid=0.01), codes(n + k, 1, C, k), \
        scales(n, C, mid=0.02 / max(k, 1) ** 0.5)


def run_dense(handle, q, sq, p, s, m, n, k, gated, variant, y=None, stream=None):
    if y is None:
        y = torch.full((m, n), float("nan"), dtype=BF, device="cuda")
    f = sw.swiglu_forward_int8 if gated else sw.swiglu_matmul_int8
    f(handle, q, sq, p, s, y, m, n, k, variant=variant, stream=stream)
    return y


SIZES = [(1, 8, 16), (1, 200, 128), (3, 64, 144), (16, 328, 400), (32, 96, 1040), (33, 40, 656),
         (65, 136, 272), (128, 256, 512), (130, 264, 1536), (257, 520, 784), (300, 72, 64),
         (520, 312, 128), (48, 2056, 896)]


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_dense(handle, m, n, k, gated):
    q, sq, w, s = dense_inputs(m, n, k, gated)
    want, slack = (M.gated if gated else M.products)(q, sq, w[0], s)
    dev = [t.cuda() for t in (q, sq)] + [pack(handle, w), s.cuda()]
    for v in VARIANTS:
        print(f"int8 {'gated' if gated else 'plain'} {m}x{n}x{k} variant {v}", flush=True)
        y = run_dense(handle, *dev, m, n, k, gated, v)
        torch.cuda.synchronize()
        O.assert_close(y, want, slack, f"{m}x{n}x{k} variant {v}")


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_dense_extreme_codes(handle, gated):
    """Sums at the ends of 32 bits: K = 131056 products of -128 by -128 and by 127."""
    m, n, k = 34, 40, 131056
    C = 2 * n if gated else n
    q, w = torch.full((m, k), -128, dtype=torch.int8), torch.full((1, C, k), -128, dtype=torch.int8)
    w[0, ::3] = 127
    sq, s = torch.full((m,), 2.0 ** -14), torch.full((C,), 2.0 ** -16)
    want, slack = (M.gated if gated else M.products)(q, sq, w[0], s)
    dev = [t.cuda() for t in (q, sq)] + [pack(handle, w), s.cuda()]
    for v in VARIANTS:
        print(f"extreme variant {v}", flush=True)
        y = run_dense(handle, *dev, m, n, k, gated, v)
        torch.cuda.synchronize()
        O.assert_close(y, want, slack, f"variant {v}")


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_dense_no_k(handle, gated):
    """K = 0 writes zeros and reads nothing, no scales either."""
    for v in VARIANTS:
        y = torch.full((70, 72), float("nan"), dtype=BF, device="cuda")
        run_dense(handle, None, None, None, None, 70, 72, 0, gated, v, y=y)
        torch.cuda.synchronize()
        assert bool((y == 0).all()), v


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_scales_of_nan_stay_in_their_row(handle, gated):
    m, n, k = 70, 72, 144
    q, sq, w, s = dense_inputs(m, n, k, gated)
    sq[[0, 33, 69]] = float("nan")
    sq[5] = 0.0
    dev = [t.cuda() for t in (q, sq)] + [pack(handle, w), s.cuda()]
    for v in VARIANTS:
        y = run_dense(handle, *dev, m, n, k, gated, v).cpu()
        bad = torch.isnan(y).all(1)
        assert bad.nonzero().flatten().tolist() == [0, 33, 69], v
        assert not torch.isnan(y[~bad]).any() and bool((y[5] == 0).all()), v


# -------------------------------------------------------------------------- by expert
def spans(counts, seed, drop=0):
    R = sum(counts) + drop
    perm = torch.randperm(R, generator=gen(seed))
    rows, at = torch.full((R,), -1, dtype=torch.int32), 0
    for n in counts:
        rows[at:at + n] = perm[at:at + n].sort().values.int()
        at += n
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    return R, off, rows


COUNTS = {"ones": [1, 1, 1], "empty": [0, 3, 0, 0, 17, 0], "tile": [16, 64, 0, 33],
          "ragged": [300, 1, 0, 129, 70, 257], "many": [2] * 70 + [0] * 30 + [5] * 30, "one": [513]}


def grouped_inputs(counts, n, k, gated, top=1, drop=0, seed=3):
    E = len(counts)
    R, off, rows = spans(counts, seed, drop)
    C, T = (2 * n, -(-R // top)) if gated else (n, R)
    return (R, T, off, rows, codes(R + k, T, k), scales(R, T, mid=0.01), codes(E + n, E, C, k),
            scales(E, E, C, mid=0.02 / k ** 0.5))


def grouped_want(off, rows, q, sq, w, s, R, n, gated, top):
    want = torch.full((R, n), float("nan"), dtype=O.F64)
    slack = torch.zeros(R, n, dtype=O.F64)
    for e in range(len(off) - 1):
        a, b = int(off[e]), int(off[e + 1])
        if a == b:
            continue
        if gated:
            t = rows[a:b].long() // top
            want[a:b], slack[a:b] = M.gated(q[t], sq[t], w[e], s[e])
        else:
            at = rows[a:b].long()
            want[at], slack[at] = M.products(q[a:b], sq[a:b], w[e], s[e])
    return want, slack


def run_grouped(handle, dev, R, T, n, k, E, gated, top, variant):
    q, sq, rows, off, p, s = dev
    y = torch.full((R, n), float("nan"), dtype=BF, device="cuda")
    if gated:
        sw.swiglu_grouped_forward_int8(handle, q, sq, rows, off, p, s, y, T, R, n, k, E, k=top,
                                       variant=variant)
    else:
        sw.swiglu_grouped_matmul_int8(handle, q, sq, rows, off, p, s, y, R, n, k, E, variant=variant)
    torch.cuda.synchronize()
    return y.cpu()


def check_grouped(got, want, slack, what):
    written = ~torch.isnan(want)
    assert bool((torch.isnan(got) == ~written).all()), f"{what}: rows of no span stay as they were"
    O.assert_close(got[written], want[written], slack[written], what)


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("n,k", [(8, 16), (72, 144), (264, 656)])
@pytest.mark.parametrize("counts", list(COUNTS))
def test_grouped(handle, counts, n, k, gated):
    c = COUNTS[counts]
    R, T, off, rows, q, sq, w, s = grouped_inputs(c, n, k, gated, top=2, drop=3)
    want, slack = grouped_want(off, rows, q, sq, w, s, R, n, gated, 2)
    dev = [t.cuda() for t in (q, sq, rows, off)] + [pack(handle, w), s.cuda()]
    for v in VARIANTS:
        print(f"grouped {counts} {n}x{k} gated={gated} variant {v}", flush=True)
        y = run_grouped(handle, dev, R, T, n, k, len(c), gated, 2, v)
        check_grouped(y, want, slack, f"{counts} {n}x{k} variant {v}")


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_grouped_bad_offsets_and_slots(handle, gated):
    """Offsets out of order or out of range are held to the sorted rows; a slot that names no row
    gives zeros (gated) or is not written (plain)."""
    c, n, k = [40, 30, 50], 72, 272
    R, T, off, rows, q, sq, w, s = grouped_inputs(c, n, k, gated)
    bad = rows.clone()
    bad[[3, 60]] = torch.tensor([-5, R + 9], dtype=torch.int32)
    p = pack(handle, w)
    for v in VARIANTS:
        print(f"bad slots gated={gated} variant {v}", flush=True)
        y = run_grouped(handle, [q.cuda(), sq.cuda(), bad.cuda(), off.cuda(), p, s.cuda()], R, T, n, k, 3,
                        gated, 1, v)
        want, slack = grouped_want(off, rows, q, sq, w, s, R, n, gated, 1)
        if gated:
            want[[3, 60]] = 0
        else:
            want[rows[[3, 60]].long()] = float("nan")
        check_grouped(y, want, slack, f"variant {v}")
        for o in ([5, 200, -3, 10 ** 9], [-7, 60, 20, 100]):
            print(f"bad offsets {o} variant {v}", flush=True)
            o = torch.tensor(o, dtype=torch.int32)
            held, reach = [], 0
            for e in range(3):
                a = max(min(max(int(o[e]), 0), R), reach)
                reach = max(a, min(max(int(o[e + 1]), 0), R))
                held.append((a, reach))
            y = run_grouped(handle, [q.cuda(), sq.cuda(), rows.cuda(), o.cuda(), p, s.cuda()], R, T, n, k,
                            3, gated, 1, v)
            want = torch.full((R, n), float("nan"), dtype=O.F64)
            slack = torch.zeros(R, n, dtype=O.F64)
            for e, (a, b) in enumerate(held):
                at = rows[a:b].long()
                if gated:
                    want[a:b], slack[a:b] = M.gated(q[at], sq[at], w[e], s[e])
                else:
                    want[at], slack[at] = M.products(q[a:b], sq[a:b], w[e], s[e])
            check_grouped(y, want, slack, f"{o} variant {v}")


def test_variants_agree_bit_for_bit(handle):
    """The sums are whole numbers, so neither the tile nor the split of K shows in a result."""
    q, sq, w, s = dense_inputs(200, 264, 1104, False)
    dev = [t.cuda() for t in (q, sq)] + [pack(handle, w), s.cuda()]
    ys = [run_dense(handle, *dev, 200, 264, 1104, False, v) for v in VARIANTS]
    assert all(torch.equal(ys[0], y) for y in ys[1:])


def test_another_stream(handle):
    q, sq, w, s = dense_inputs(64, 128, 512, True)
    dev = [t.cuda() for t in (q, sq)] + [pack(handle, w), s.cuda()]
    first = run_dense(handle, *dev, 64, 128, 512, True, -1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = torch.full_like(first, float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    run_dense(handle, *dev, 64, 128, 512, True, -1, y=y, stream=side)
    with torch.cuda.stream(side):
        z = run_dense(handle, *dev, 64, 128, 512, True, -1)
    side.synchronize()
    assert torch.equal(first, y) and torch.equal(first, z)


# ---------------------------------------------------------------- a block of them together
@pytest.mark.parametrize("T", [1, 37, 700])
def test_block(handle, T):
    """Quantise, route by score, gated and down products by expert, the combining norm: eager,
    then captured and replayed with poisoned buffers, against the chain of definitions."""
    E, k, D, N = 16, 3, 256, 96
    x = (torch.randn(T, D, generator=gen(T))).to(BF)
    router = torch.randn(D, E, generator=gen(1)) * D ** -0.5
    bias = 0.1 * torch.randn(E, generator=gen(2))
    wu, wd = codes(5, E, 2 * N, D), codes(6, E, D, N)
    su, sd = scales(7, E, 2 * N, mid=D ** -0.5 / 70), scales(8, E, D, mid=N ** -0.5 / 70)
    pre = torch.ones(D, dtype=BF)
    logits = x.float() @ router
    dev = {n: t.cuda() for n, t in dict(x=x, logits=logits, bias=bias, su=su, sd=sd, pre=pre).items()}
    pu, pd = pack(handle, wu), pack(handle, wd)
    i32 = dict(dtype=torch.int32, device="cuda")
    b = dict(q=torch.empty(T, D, dtype=torch.int8, device="cuda"), sq=torch.empty(T, device="cuda"),
             w=torch.empty(T, k, device="cuda"), e=torch.empty(T, k, **i32),
             off=torch.empty(E + 1, **i32), rows=torch.empty(T * k, **i32),
             up=torch.empty(T * k, N, dtype=BF, device="cuda"),
             q2=torch.empty(T * k, N, dtype=torch.int8, device="cuda"),
             s2=torch.empty(T * k, device="cuda"), down=torch.empty(T * k, D, dtype=BF, device="cuda"),
             X=torch.empty(T, D, dtype=BF, device="cuda"), H=torch.empty(T, D, dtype=BF, device="cuda"))
    ws = torch.empty(sw.swiglu_route_workspace_bytes(T, E, k), dtype=torch.uint8, device="cuda")

    def step():
        h = handle
        sw.swiglu_quantize_int8(h, dev["x"], b["q"], b["sq"], T, D)
        sw.swiglu_route_scored(h, dev["logits"], dev["bias"], b["w"], b["e"], b["off"], b["rows"], ws, T,
                               E, k, score=sw.SCORE_SIGMOID, scale=1.5, groups=4, top_groups=2,
                               group_best=2)
        sw.swiglu_grouped_forward_int8(h, b["q"], b["sq"], b["rows"], b["off"], pu, dev["su"], b["up"], T,
                                       T * k, N, D, E, k=k)
        sw.swiglu_quantize_int8(h, b["up"], b["q2"], b["s2"], T * k, N)
        sw.swiglu_grouped_matmul_int8(h, b["q2"], b["s2"], b["rows"], b["off"], pd, dev["sd"], b["down"],
                                      T * k, D, N, E)
        sw.swiglu_combine_norm(h, b["down"], b["w"], b["e"], None, dev["x"], None, None, dev["pre"],
                               b["X"], b["H"], T, D, k=k)
    step()
    torch.cuda.synchronize()
    eager = {n: t.clone() for n, t in b.items()}
    c = {n: t.cpu() for n, t in b.items()}
    # each stage against its definition on the stage before it
    W, X, OFF, ROWS = M.route_scored(logits, bias, k, "sigmoid", True, 1.5, 4, 2, 2)
    assert np.array_equal(c["e"], X) and np.array_equal(c["off"], OFF) and np.array_equal(c["rows"], ROWS)
    Q, S = M.quantize(x)
    assert np.array_equal(c["q"], Q)
    want, slack = grouped_want(c["off"], c["rows"], c["q"], c["sq"], wu, su, T * k, N, True, k)
    O.assert_close(c["up"], want, slack, "up")
    assert np.array_equal(c["q2"], M.quantize(c["up"])[0])
    want, slack = grouped_want(c["off"], c["rows"], c["q2"], c["s2"], wd, sd, T * k, D, False, 1)
    O.assert_close(c["down"], want, slack, "down")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        for t in b.values():
            t.view(torch.uint8).fill_(0xff)
        ws.fill_(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in b.items():
            assert torch.equal(t, eager[n]), (i, n)
