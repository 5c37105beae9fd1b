"""The scored router on the GPU against its 64-bit definition: both scores, bias, groups, masks that
leave nothing, ties, scores that only 64 bits tell apart, both dtypes, one and two launches."""
import itertools

import numpy as np
import pytest
import torch

import gemm_epilogues_mlp_amd as sw
import more_oracle as M
import ops_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def handle():
    h = sw.swiglu_create(0)
    yield h
    sw.swiglu_destroy(h)


def run(handle, x, bias, k, score, renorm, scale, groups, top, best):
    T, E = x.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    e, off, rows = torch.full((T, k), -9, **i32), torch.full((E + 1,), -9, **i32), \
        torch.full((T * k,), -9, **i32)
    ws = torch.randint(0, 255, (sw.swiglu_route_workspace_bytes(T, E, k),), dtype=torch.uint8,
                       device="cuda")
    sw.swiglu_route_scored(handle, x.cuda(), None if bias is None else bias.cuda(), w, e, off, rows, ws,
                           T, E, k, score=sw.SCORE_SIGMOID if score == "sigmoid" else sw.SCORE_SOFTMAX,
                           renormalize=renorm, scale=scale, groups=groups, top_groups=top,
                           group_best=best, dtype=sw.DTYPE_F32 if x.dtype == F32 else sw.DTYPE_BF16)
    torch.cuda.synchronize()
    return w.cpu(), e.cpu(), off.cpu(), rows.cpu()


def check(handle, x, bias, k, score="sigmoid", renorm=True, scale=1.0, groups=1, top=1, best=1):
    what = f"{tuple(x.shape)} {x.dtype} k={k} {score} renorm={renorm} groups={groups}/{top}/{best}"
    print(what, flush=True)
    w, e, off, rows = run(handle, x, bias, k, score, renorm, scale, groups, top, best)
    W, X, OFF, ROWS = M.route_scored(x, bias, k, score, renorm, scale, groups, top, best)
    assert np.array_equal(e.numpy(), X), what
    assert np.array_equal(off.numpy(), OFF), what
    assert np.array_equal(rows.numpy(), ROWS), what
    # computed in 64 bits, rounded once
    want = torch.from_numpy(W)
    O.assert_close(w, want, 1e-12 * want.abs(), what, half=O.U32)


def logits(T, E, dtype, masked=0.1):
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(T + E)) * 1.5
    off = torch.rand(T, E, generator=torch.Generator().manual_seed(T)) < masked
    off |= torch.rand(T, 1, generator=torch.Generator().manual_seed(E)) < masked
    return torch.where(off, float("-inf"), x).to(dtype)


def biases(E):
    return 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,groups,top,best", [
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (3, 5, 5, 5, 5, 2), (17, 8, 1, 2, 1, 1),
    (64, 60, 8, 4, 2, 2), (65, 64, 8, 8, 3, 2), (200, 72, 4, 3, 1, 1), (513, 128, 8, 4, 2, 2),
    (1000, 200, 3, 8, 8, 2), (333, 256, 8, 8, 4, 2), (130, 500, 17, 10, 4, 2),
    (90, 1000, 64, 50, 20, 1), (700, 160, 2, 1, 1, 1), (128, 100, 32, 2, 2, 2), (9, 128, 2, 64, 3, 2),
    (40, 1024, 8, 64, 7, 2)])
def test_scored(handle, T, E, k, groups, top, best, dtype):
    for score, renorm, bias in itertools.product(("sigmoid", "softmax"), (True, False),
                                                 (None, biases(E))):
        check(handle, logits(T, E, dtype), bias, k, score, renorm, 2.5, groups, top, best)


@pytest.mark.parametrize("E,k,groups,top,best", [(60, 1, 4, 2, 2), (128, 8, 8, 4, 2), (200, 3, 8, 3, 1),
                                                 (256, 8, 8, 4, 2), (500, 7, 10, 4, 2), (1000, 2, 50, 20, 1)])
def test_few_slots(handle, E, k, groups, top, best):
    """Up to 512 slots, where one workgroup sorts: tokens that it scores by itself and, beyond one
    pass of its lanes, those that others score."""
    for T in sorted({8, 9, 16, 17, 32, 33, 64, 512 // k}):
        if T * k <= 512:
            check(handle, logits(T, E, BF if T % 2 else F32), biases(E), k, "sigmoid", True, 2.5, groups,
                  top, best)
            check(handle, logits(T, E, F32, masked=0.95), None, k, "softmax", False, 1.0, groups, top,
                  best)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_special_logits(handle, score):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(BF).min
    rows = [[-inf] * 6, [nan] * 6, [nan, 1, -inf, 2, nan, 0], [inf, 1, inf, 2, 0, -inf], [low] * 6,
            [low, -inf, low, nan, -inf, -inf], [0.0, -0.0, 0.0, -0.0, 0.0, 0.0],
            [3, 3, 3, 1, 3, 3], [30, -100, 0, 30, -100, 0], [-inf, -inf, -inf, 1, 2, nan],
            [50, 60, 40, 70, 80, 60], [-800, -750, -720, -900, -708, -1000]]
    for dtype, renorm, k in itertools.product((F32, BF), (True, False), (1, 3, 6)):
        x = torch.tensor(rows, dtype=dtype)
        check(handle, x, None, k, score, renorm)
        check(handle, x, torch.zeros(6), k, score, renorm)
        if k <= 4:
            for best in (1, 2):
                check(handle, x, None, k, score, renorm, groups=3, top=2, best=best)
                check(handle, x, torch.tensor([0, .5, 0, -.5, 0, .25]), k, score, renorm, groups=3,
                      top=2, best=best)


def test_special_biases(handle):
    """An expert whose score plus bias is -inf or NaN is closed, one at +inf comes first."""
    inf, nan = float("inf"), float("nan")
    x = logits(50, 12, F32)
    for b in ([0.0] * 11 + [nan], [-inf, 0, nan] * 4, [inf, 0, -inf, 0] * 3, [-inf] * 12,
              [1e30, -1e30, 0.0] * 4):
        check(handle, x, torch.tensor(b), 4)
        check(handle, x, torch.tensor(b), 4, groups=3, top=2, best=1)


@pytest.mark.parametrize("groups,top,best", [(1, 1, 1), (8, 3, 2), (8, 3, 1)])
def test_scores_that_32_bits_do_not_tell_apart(handle, groups, top, best):
    """Logits of some 1e-10: every score is 0.5 in fp32, and the definition still orders them."""
    for T, E, k in ((5, 64, 6), (200, 64, 6)):
        perm = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t)) for t in range(T)])
        x = (perm.float() - 31) * 1e-10
        check(handle, x, None, k, "sigmoid", groups=groups, top=top, best=best)
        check(handle, x, torch.full((E,), 0.25), k, "sigmoid", groups=groups, top=top, best=best)


def test_ties_take_the_lower_index(handle):
    """Few distinct logits and biases: equal experts, and equal groups, in every token."""
    for T in (20, 400):
        g = torch.Generator().manual_seed(T)
        x = torch.randint(0, 3, (T, 64), generator=g).float()
        b = torch.randint(0, 2, (64,), generator=g).float()
        for dtype, bias in itertools.product((F32, BF), (None, b)):
            check(handle, x.to(dtype), bias, 6, "sigmoid")
            check(handle, x.to(dtype), bias, 6, "sigmoid", groups=8, top=3, best=2)
            check(handle, x.to(dtype), bias, 6, "softmax", groups=16, top=5, best=1)


def test_unaligned_rows_and_bias(handle):
    x = torch.randn(40 * 64 + 1, generator=torch.Generator().manual_seed(2))
    b = torch.randn(65, generator=torch.Generator().manual_seed(3))
    i32 = dict(dtype=torch.int32, device="cuda")
    w, e = torch.empty(40, 4, device="cuda"), torch.empty(40, 4, **i32)
    off, rows = torch.empty(65, **i32), torch.empty(160, **i32)
    sw.swiglu_route_scored(handle, x.cuda()[1:], b.cuda()[1:], w, e, off, rows, None, 40, 64, 4)
    torch.cuda.synchronize()
    want = M.route_scored(x[1:].view(40, 64), b[1:], 4, "softmax", True, 1.0, 1, 1, 1)
    assert np.array_equal(e.cpu().numpy(), want[1])


def test_no_tokens(handle):
    _, _, off, _ = run(handle, torch.zeros(0, 12), None, 2, "sigmoid", True, 1.0, 3, 1, 2)
    assert bool((off == 0).all())


def test_repeats(handle):
    x = logits(4000, 64, BF)
    args = (handle, x, biases(64), 6, "sigmoid", True, 2.5, 8, 4, 2)
    first = run(*args)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, run(*args)))


def test_choice_without_bias_is_the_routers(handle):
    """Softmax scores without bias and groups: the experts and the order of swiglu_route."""
    x = logits(900, 72, F32)
    w, e, off, rows = run(handle, x, None, 5, "softmax", True, 1.0, 1, 1, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    w2, e2 = torch.empty(900, 5, device="cuda"), torch.empty(900, 5, **i32)
    off2, rows2 = torch.empty(73, **i32), torch.empty(4500, **i32)
    ws = torch.empty(sw.swiglu_route_workspace_bytes(900, 72, 5), dtype=torch.uint8, device="cuda")
    sw.swiglu_route(handle, x.cuda(), w2, e2, off2, rows2, ws, 900, 72, 5)
    torch.cuda.synchronize()
    assert torch.equal(e, e2.cpu()) and torch.equal(off, off2.cpu()) and torch.equal(rows, rows2.cpu())


@pytest.mark.parametrize("T,E,k,groups,top,best", [(9000, 32, 4, 8, 3, 2), (20000, 16, 2, 1, 1, 1),
                                                   (4100, 256, 8, 8, 4, 2)])
def test_many_tokens(handle, T, E, k, groups, top, best):
    """More tokens than the workgroups take in one pass."""
    check(handle, logits(T, E, BF), biases(E), k, "sigmoid", True, 2.5, groups, top, best)


def test_graph_replays_equal_eager(handle):
    T, E, k = 700, 64, 6
    x, b = torch.empty(T, E, device="cuda"), biases(E).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    out = [torch.empty(T, k, device="cuda"), torch.empty(T, k, **i32), torch.empty(E + 1, **i32),
           torch.empty(T * k, **i32)]
    ws = torch.empty(sw.swiglu_route_workspace_bytes(T, E, k), dtype=torch.uint8, device="cuda")

    def step():
        sw.swiglu_route_scored(handle, x, b, *out, ws, T, E, k, score=sw.SCORE_SIGMOID, groups=8,
                               top_groups=4, group_best=2)
    side = torch.cuda.Stream()
    x.normal_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.normal_()
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in out]
        for t in (*out, ws):
            t.view(torch.uint8).fill_(0x7f)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, out)), i
