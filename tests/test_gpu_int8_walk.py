"""The 8-bit integer operators where one workgroup does several pieces of work, at the ends of their
sizes, and as programs use them: rings that run on from tile to tile, tensors past 4 GiB and close to
2 GiB, refusals that write nothing, several threads and streams at once, graphs.

The sums are whole numbers, so every variant gives the same bits: a tiled variant is held to the
streaming one, which test_gpu_int8.py holds to the definition, and here too on single rows."""
import threading

import numpy as np
import pytest
import torch

import gemm_epilogues_mlp_amd as sw
import more_oracle as M
import ops_oracle as O

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TILES = {4: (64, 128, 2), 5: (128, 128, 2), 6: (128, 256, 1), 7: (256, 256, 1)}  # rows, columns, a CU


@pytest.fixture(scope="module")
def handle():
    h = sw.swiglu_create(0)
    yield h
    sw.swiglu_destroy(h)


def dev(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(seed, *shape):
    return torch.randint(-127, 128, shape, generator=dev(seed), device="cuda", dtype=torch.int8)


def scales(seed, *shape, mid):
    return torch.exp(0.3 * torch.randn(*shape, generator=dev(seed), device="cuda")) * mid


def pack(handle, w):
    E, rows, K = w.shape
    p = torch.empty(E * sw.swiglu_int8_packed_bytes(rows, K), dtype=torch.int8, device="cuda")
    sw.swiglu_pack_int8_fragments(handle, w, p, E, rows, K)
    return p


def dense(handle, gated, q, sq, p, s, m, n, k, variant, y=None):
    y = torch.full((m, n), float("nan"), dtype=BF, device="cuda") if y is None else y
    (sw.swiglu_forward_int8 if gated else sw.swiglu_matmul_int8)(handle, q, sq, p, s, y, m, n, k,
                                                                  variant=variant)
    return y


def check_rows(y, at, gated, q, sq, w, s, what):
    """Rows `at` of y against the definition."""
    want, slack = (M.gated if gated else M.products)(q[at].cpu(), sq[at].cpu(), w.cpu(), s.cpu())
    O.assert_close(y[at], want, slack, what)


def test_the_walks_are_walks():
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    for v, (bm, bn, per) in TILES.items():
        m, n = walk(bm, bn, per, cus)
        assert -(-m // bm) * -(-n // bn) > 2 * cus * per


def walk(bm, bn, per, cus):
    """Sizes of some 2.3 tiles a workgroup, the last row and column of tiles partial."""
    rows = 12
    cols = int(2.3 * cus * per / rows) + 1
    return rows * bm - bm // 3, cols * bn - 40


# 1 to 9 groups of K (run as 3 at least), odd and even numbers of them
@pytest.mark.parametrize("k", [16, 144, 272, 400, 640, 1040])
@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("variant", list(TILES))
def test_ring_runs_on_from_tile_to_tile(handle, variant, gated, k):
    bm, bn, per = TILES[variant]
    m, c = walk(bm, bn, per, torch.cuda.get_device_properties(0).multi_processor_count)
    n = c // 2 // 8 * 8 if gated else c // 8 * 8
    print(f"walk variant {variant} gated={gated} {m}x{n}x{k}", flush=True)
    C = 2 * n if gated else n
    q, sq, w, s = codes(k, m, k), scales(1, m, mid=0.01), codes(k + 1, 1, C, k), \
        scales(2, C, mid=0.02 / k ** 0.5)
    p = pack(handle, w)
    y = dense(handle, gated, q, sq, p, s, m, n, k, variant)
    want = dense(handle, gated, q, sq, p, s, m, n, k, 2)
    assert torch.equal(y, want)
    check_rows(y, torch.tensor([0, bm - 1, bm, m // 2, m - 1]), gated, q, sq, w[0], s, f"variant {variant}")


def spans(counts, seed, drop=0):
    R = sum(counts) + drop
    perm = torch.randperm(R, generator=torch.Generator().manual_seed(seed))
    rows, at = torch.full((R,), -1, dtype=torch.int32), 0
    for n in counts:
        rows[at:at + n] = perm[at:at + n].sort().values.int()
        at += n
    return R, torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32), rows


def grouped(handle, gated, q, sq, rows, off, p, s, T, R, n, k, E, top, variant):
    y = torch.full((R, n), float("nan"), dtype=BF, device="cuda")
    if gated:
        sw.swiglu_grouped_forward_int8(handle, q, sq, rows, off, p, s, y, T, R, n, k, E, k=top,
                                       variant=variant)
    else:
        sw.swiglu_grouped_matmul_int8(handle, q, sq, rows, off, p, s, y, R, n, k, E, variant=variant)
    return y


@pytest.mark.parametrize("k", [144, 528, 656])
@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
@pytest.mark.parametrize("variant", list(TILES))
def test_ring_runs_on_from_expert_to_expert(handle, variant, gated, k):
    """Spans of every height of a last tile, empty ones among them, and more experts than a wave has
    lanes."""
    counts = [bm for i in range(12) for bm in (0, 1 + 23 * i, 33, 64 + i, 0, 257 + 11 * i, 96)]
    E, n = len(counts), 712
    R, off, rows = spans(counts, 5, drop=7)
    C, T = (2 * n, -(-R // 3)) if gated else (n, R)
    print(f"walk over {E} experts, {R} rows, variant {variant} gated={gated} k={k}", flush=True)
    q, sq, w, s = codes(k, T, k), scales(1, T, mid=0.01), codes(k + 1, E, C, k), \
        scales(2, E, C, mid=0.02 / k ** 0.5)
    p, rows, off = pack(handle, w), rows.cuda(), off.cuda()
    args = (q, sq, rows, off, p, s, T, R, n, k, E, 3)
    y, want = grouped(handle, gated, *args, variant), grouped(handle, gated, *args, 2)
    written = ~torch.isnan(want)
    assert int(written.sum()) == sum(counts) * n
    assert torch.equal(torch.isnan(y), ~written) and torch.equal(y[written], want[written])
    for e in (1, 5, E - 2):
        a, b = int(off[e]), int(off[e + 1])
        at = rows[a:b].long()
        t = at // 3 if gated else torch.arange(a, b, device="cuda")
        out, slack = (M.gated if gated else M.products)(q[t].cpu(), sq[t].cpu(), w[e].cpu(), s[e].cpu())
        O.assert_close(y[a:b] if gated else y[at], out, slack, f"expert {e}")


@pytest.mark.parametrize("variant", [0, 1, 2, 3, 4, 5, 6, 7])
def test_grouped_empty_sizes(handle, variant):
    """No K: zeros in the spans, nothing else and no scales read; no activation rows: zeros."""
    R, off, rows = spans([5, 0, 70], 1, drop=2)
    rows, off = rows.cuda(), off.cuda()
    y = grouped(handle, True, None, None, rows, off, None, None, R, R, 40, 0, 3, 1, variant)
    assert bool((y[:75] == 0).all()) and bool(torch.isnan(y[75:]).all())
    y = grouped(handle, False, None, None, rows, off, None, None, R, R, 40, 0, 3, 1, variant)
    at = rows[:75].long()
    assert bool((y[at] == 0).all()) and int(torch.isnan(y).sum()) == 2 * 40
    p, s = pack(handle, codes(1, 3, 80, 32)), scales(2, 3, 80, mid=1.0)
    y = grouped(handle, True, None, None, rows, off, p, s, 0, R, 40, 32, 3, 1, variant)
    assert bool((y[:75] == 0).all())


def test_experts_past_4_gib(handle):
    """The last expert's weights lie behind 4 GiB of the others'."""
    E, n, k = 18, 16384, 16384
    p = torch.zeros(E * sw.swiglu_int8_packed_bytes(n, k), dtype=torch.int8, device="cuda")
    assert p.numel() > 1 << 32
    w = codes(3, 1, n, k)
    last = pack(handle, w)
    p[-last.numel():] = last
    s = torch.full((E, n), float("nan"), device="cuda")
    s[-1] = scales(4, n, mid=1e-4)
    R = 40
    off = torch.tensor([0] * E + [R], dtype=torch.int32, device="cuda")
    rows = torch.randperm(R, generator=torch.Generator().manual_seed(1)).sort().values.int().cuda()
    q, sq = codes(5, R, k), scales(6, R, mid=0.01)
    want, slack = M.products(q.cpu(), sq.cpu(), w[0].cpu(), s[-1].cpu())
    for v in (0, 1, 2, 3, 4, 5, 6, 7, -1):
        print(f"past 4 GiB variant {v}", flush=True)
        y = grouped(handle, False, q, sq, rows, off, p, s, R, R, n, k, E, 1, v)
        O.assert_close(y, want, slack, f"variant {v}")


@pytest.mark.parametrize("variant", [0, 3, 4, 7])
def test_output_past_4_gib(handle, variant):
    m, n, k = 66000, 32768, 16
    assert 2 * m * n > 1 << 32
    q, sq, w, s = codes(1, m, k), scales(2, m, mid=0.01), codes(3, 1, n, k), scales(4, n, mid=0.01)
    y = dense(handle, False, q, sq, pack(handle, w), s, m, n, k, variant)
    check_rows(y, torch.tensor([0, 1, 65534, 65535, 65536, m - 1]), False, q, sq, w[0], s, f"variant {variant}")
    assert not bool(torch.isnan(y[-300:]).any())


@pytest.mark.parametrize("variant", [0, 1, 2, 3, 4, 5, 6, 7])
def test_activations_close_to_2_gib(handle, variant):
    m, n, k = 16386, 24, 131056
    assert (1 << 31) - k < m * k < 1 << 31
    q, sq, w, s = codes(1, m, k), scales(2, m, mid=0.01), codes(3, 1, n, k), scales(4, n, mid=1e-4)
    y = dense(handle, False, q, sq, pack(handle, w), s, m, n, k, variant)
    check_rows(y, torch.tensor([0, 8191, m - 2, m - 1]), False, q, sq, w[0], s, f"variant {variant}")
    assert not bool(torch.isnan(y).any())


def test_refusals_write_nothing(handle):
    q, sq, s = codes(1, 40, 64), scales(2, 40, mid=1.0), scales(3, 128, mid=1.0)
    w = codes(4, 1, 128, 64)
    p = pack(handle, w)
    y = torch.full((40, 64), 7.0, dtype=BF, device="cuda")
    x = torch.ones(40, 64, dtype=BF, device="cuda")
    rows = torch.arange(40, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    w32, e = torch.full((40, 2), 7.0, device="cuda"), torch.full((40, 2), 7, dtype=torch.int32, device="cuda")
    f = sw
    calls = [
        lambda: f.swiglu_forward_int8(handle, q, sq, p, s, y, 40, 60, 64),
        lambda: f.swiglu_forward_int8(handle, q, sq, p, s, y, 40, 64, 63),
        lambda: f.swiglu_forward_int8(handle, q, sq, p, s, y, 40, 64, 64, variant=8),
        lambda: f.swiglu_forward_int8(handle, y, sq, p, s, y, 40, 64, 64),
        lambda: f.swiglu_matmul_int8(handle, q, sq, p, None, y, 40, 64, 64),
        lambda: f.swiglu_matmul_int8(handle, q, None, p, s, y, 40, 64, 64),
        lambda: f.swiglu_grouped_forward_int8(handle, q, sq, rows, None, p, s, y, 40, 40, 64, 64, 1),
        lambda: f.swiglu_grouped_forward_int8(handle, q, sq, rows, off, p, s, y, 40, 40, 64, 64, 0),
        lambda: f.swiglu_grouped_matmul_int8(handle, q, sq, rows, off, p, s, y, 40, 64, 64, 1025),
        lambda: f.swiglu_quantize_int8(handle, x, y, sq, 40, 40),
        lambda: f.swiglu_quantize_int8(handle, y, y, sq, 40, 64),
        lambda: f.swiglu_pack_int8_fragments(handle, y, y, 1, 40, 64),
        lambda: f.swiglu_route_scored(handle, x, None, w32, e, off, rows, None, 40, 64, 2,
                                      dtype=sw.DTYPE_BF16, groups=3, top_groups=1),
        lambda: f.swiglu_route_scored(handle, x, None, w32, e, off, rows, None, 40, 64, 40,
                                      dtype=sw.DTYPE_BF16, groups=2, top_groups=1),
        lambda: f.swiglu_route_scored(handle, x, w32, w32, e, off, rows, None, 40, 64, 2,
                                      dtype=sw.DTYPE_BF16),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(sw.SwiGLUError) as err:
            call()
        assert err.value.status in (sw.ERR_INVALID_ARG, sw.ERR_UNSUPPORTED), i
    torch.cuda.synchronize()
    assert bool((y == 7).all()) and bool((w32 == 7).all()) and bool((e == 7).all())
    assert off.tolist() == [0, 40] and torch.equal(rows, torch.arange(40, dtype=torch.int32, device="cuda"))


def test_threads_share_a_handle(handle):
    """Four host threads, each with a stream of its own: quantisation, a product, a grouped one and the
    scored router at once; every result is that of the lone call."""
    def work(i, stream, out):
        m, n, k = 70 + 64 * i, 264, 400 + 128 * i
        with torch.cuda.stream(stream):
            g = torch.Generator(device="cuda").manual_seed(i)
            x = torch.randn(m, k, generator=g, device="cuda").to(BF)
            q = torch.empty(m, k, dtype=torch.int8, device="cuda")
            sq = torch.empty(m, device="cuda")
            w = torch.randint(-127, 128, (4, 2 * n, k), generator=g, device="cuda", dtype=torch.int8)
            p = torch.empty(4 * sw.swiglu_int8_packed_bytes(2 * n, k), dtype=torch.int8, device="cuda")
            s = torch.rand(4, 2 * n, generator=g, device="cuda") * 1e-2
            lg = torch.randn(m, 32, generator=g, device="cuda")
            i32 = dict(dtype=torch.int32, device="cuda")
            wt, e = torch.empty(m, 2, device="cuda"), torch.empty(m, 2, **i32)
            off, rows = torch.empty(33, **i32), torch.empty(2 * m, **i32)
            ws = torch.empty(sw.swiglu_route_workspace_bytes(m, 32, 2), dtype=torch.uint8, device="cuda")
            goff = torch.tensor([0, m // 3, m // 3, m - 5, m], **i32)
            grows = torch.arange(m, **i32)
            y, gy = (torch.empty(m, n, dtype=BF, device="cuda") for _ in range(2))
            sw.swiglu_pack_int8_fragments(handle, w, p, 4, 2 * n, k)
            for _ in range(6):
                sw.swiglu_quantize_int8(handle, x, q, sq, m, k)
                sw.swiglu_forward_int8(handle, q, sq, p, s, y, m, n, k)
                sw.swiglu_grouped_forward_int8(handle, q, sq, grows, goff, p, s, gy, m, m, n, k, 4)
                sw.swiglu_route_scored(handle, lg, None, wt, e, off, rows, ws, m, 32, 2,
                                       score=sw.SCORE_SIGMOID, groups=4, top_groups=2, group_best=2)
            out[i] = [t.cpu() for t in (q, sq, y, gy, wt, e, off, rows)]
    lone, together = {}, {}
    streams = [torch.cuda.Stream() for _ in range(4)]
    for i, st in enumerate(streams):
        work(i, st, lone)
        st.synchronize()
    threads = [threading.Thread(target=work, args=(i, st, together)) for i, st in enumerate(streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(together) == 4
    for i in lone:
        assert all(torch.equal(a, b) for a, b in zip(lone[i], together[i])), i


@pytest.mark.parametrize("m,n,k", [(1, 264, 400), (40, 264, 400), (300, 520, 784)])
def test_graph_replays_equal_eager(handle, m, n, k):
    """Two graphs of the same calls on one set of buffers, replayed in turn, with new inputs and poisoned
    outputs between the replays."""
    w, s = codes(1, 1, 2 * n, k), scales(2, 2 * n, mid=1e-2)
    p = pack(handle, w)
    x = torch.empty(m, k, dtype=BF, device="cuda")
    q, sq = torch.empty(m, k, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    y = torch.empty(m, n, dtype=BF, device="cuda")

    def step():
        sw.swiglu_quantize_int8(handle, x, q, sq, m, k)
        sw.swiglu_forward_int8(handle, q, sq, p, s, y, m, n, k)
    x.normal_(generator=dev(0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graphs = []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step()
    for i in range(5):
        x.normal_(generator=dev(i))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (q, sq, y)]
        for t in (q, sq, y):
            t.view(torch.uint8).fill_(0x7f)
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (q, sq, y))), i
