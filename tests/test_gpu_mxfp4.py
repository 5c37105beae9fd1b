"""MXFP4 on the GPU: quantisation and its inverse bit for bit against the
definition, the gated product against 64-bit sums of the same values (every
kernel variant), refusals, streams and graphs."""
import numpy as np
import pytest
import torch

import gemm_epilogues_mlp_amd as sw
import ops_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    h = sw.swiglu_create(0)
    yield h
    sw.swiglu_destroy(h)


def bf16(x):
    return torch.as_tensor(np.ascontiguousarray(x)).to(torch.bfloat16)


def f64(t):
    return t.to(torch.float64).numpy()


def quantized(handle, x):
    rows, K = x.shape
    q = torch.full((sw.swiglu_mxfp4_bytes(rows, K),), 0xEE, dtype=torch.uint8, device="cuda")
    s = torch.full((sw.swiglu_mxfp4_scale_bytes(rows, K),), 0xEE, dtype=torch.uint8, device="cuda")
    sw.swiglu_quantize_mxfp4(handle, x.cuda(), q, s, rows, K)
    torch.cuda.synchronize()
    return q, s


def check_quantize(handle, x, what):
    q, s = quantized(handle, x)
    codes, scales = O.quantize(f64(x))
    want_s = O.fragment_scales(scales)
    assert np.array_equal(s.cpu().numpy(), want_s), what
    # a block with a NaN has unspecified codes
    nan = np.repeat(scales == 255, 32, axis=1)
    got, want = q.cpu().numpy(), O.fragment_codes(np.where(nan, 0, codes))
    mask = O.fragment_codes(np.where(nan, 0, 0xF).astype(np.uint8))
    assert np.array_equal(got & mask, want & mask), what
    out = torch.full(x.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    sw.swiglu_dequantize_mxfp4(handle, q, s, out, *x.shape)
    torch.cuda.synchronize()
    v = bf16(O.values(codes, scales))
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(v)), what
    ok = ~torch.isnan(v)
    assert torch.equal(out.cpu()[ok].view(torch.int16), v[ok].view(torch.int16)), what


@pytest.mark.parametrize("rows,K", [(1, 32), (1, 64), (7, 96), (32, 256), (33, 288), (100, 896),
                                    (257, 1568)])
def test_quantize_random(handle, rows, K):
    rng = np.random.default_rng(rows * 1000 + K)
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-60, 60, (rows, 1)))
    x[rng.random((rows, K)) < 0.1] = 0.0
    check_quantize(handle, bf16(x), f"{rows}x{K}")


def test_quantize_every_bf16_value(handle):
    """Each of the 65536 patterns beside larger leaders, so that it falls on every part of
    the grid, and by itself in a block of zeros (its own scale)."""
    bits = np.arange(65536, dtype=np.uint16).view(np.int16)
    x = torch.from_numpy(bits.copy()).view(torch.bfloat16)
    alone = torch.zeros(65536 // 8, 8, 32, dtype=torch.bfloat16)
    alone[:, :, 5] = x.view(-1, 8)
    check_quantize(handle, alone.reshape(65536 // 8, 256), "alone")
    # magnitudes around a leader of 4 x 2^n: 31 neighbours of one leader a block
    for n in (-126, -120, 0, 3, 100, 125):
        lead = 2.0 ** n
        grid = np.linspace(-7.99, 7.99, 31 * 64).reshape(64, 31) * (lead / 4)
        b = np.concatenate([np.full((64, 1), lead), grid], 1)
        check_quantize(handle, bf16(b.reshape(8, 256)), f"leader 2^{n}")


def test_quantize_ties(handle):
    ties = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 7, 6.5, 4.9375, 5.0625, 0.2490234375])
    b = np.zeros((2, 32))
    b[0, 0], b[1, 0] = 4.0, -4.0
    b[0, 1:13], b[1, 1:13] = ties, -ties
    for n in (-100, 0, 90):
        check_quantize(handle, bf16(b * 2.0 ** n), f"ties 2^{n}")


def test_quantize_special_values(handle):
    b = np.zeros((6, 64))
    b[0, 3], b[0, 40] = np.inf, 1.0
    b[1, 3] = -np.inf
    b[2, 7], b[2, 50] = np.nan, 2.0
    b[3, :] = 3.3895313892515355e38          # the largest bf16
    b[4, :] = 2.0 ** -133                     # the smallest subnormal
    b[5, :] = -0.0
    check_quantize(handle, bf16(b), "special")


# ------------------------------------------------------------------------ the product
def product(handle, M, N, K, variant, seed, x=None):
    rng = np.random.default_rng(seed)
    x = bf16(rng.standard_normal((M, K))) if x is None else x
    w = bf16(rng.standard_normal((2 * N, K)) * K ** -0.5)
    q, s = quantized(handle, x)
    wq, ws = quantized(handle, w)
    y = torch.full((M + 1, N), -7.0, dtype=torch.bfloat16, device="cuda")
    sw.swiglu_forward_mxfp4(handle, q, s, wq, ws, y, M, N, K, variant=variant)
    torch.cuda.synchronize()
    assert bool((y[M] == -7.0).all()), "wrote past its rows"
    a = torch.from_numpy(O.values(*O.quantize(f64(x))))
    b = torch.from_numpy(O.values(*O.quantize(f64(w))))
    return y[:M], O.gated(a, b.t().contiguous())


SHAPES = [(1, 8, 32), (5, 24, 64), (33, 72, 96), (64, 136, 256), (130, 264, 288), (257, 520, 544),
          (300, 128, 1056)]


@pytest.mark.parametrize("variant", [-1, 0, 1, 2, 3])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_product(handle, variant, shape):
    print(f"mxfp4 product {shape} variant {variant}", flush=True)
    y, (want, slack) = product(handle, *shape, variant, 11)
    O.assert_close(y, want, slack, f"{shape} variant {variant}")


@pytest.mark.parametrize("shape", [(1024, 4864, 896), (16, 2368, 3584), (700, 1000, 3552)], ids=str)
def test_product_larger(handle, shape):
    y, (want, slack) = product(handle, *shape, -1, 12)
    O.assert_close(y, want, slack, str(shape))


def test_product_scales_far_apart(handle):
    """Rows and blocks whose scales differ by many binades (the matrix instruction applies
    them block by block)."""
    rng = np.random.default_rng(5)
    M, K = 96, 512
    x = rng.standard_normal((M, K // 32, 32)) * np.exp2(rng.integers(-20, 20, (M, K // 32, 1)))
    for variant in range(4):
        y, (want, slack) = product(handle, M, 64, K, variant, 6, bf16(x.reshape(M, K)))
        O.assert_close(y, want, slack, f"variant {variant}")


def test_nan_reaches_its_row_only(handle):
    rng = np.random.default_rng(3)
    M, N, K = 70, 40, 128
    x = bf16(rng.standard_normal((M, K)))
    x[37, 70] = float("nan")
    for variant in range(4):
        y, (want, slack) = product(handle, M, N, K, variant, 4, x)
        y = y.cpu()
        assert bool(torch.isnan(y[37]).all())
        keep = torch.arange(M) != 37
        O.assert_close(y[keep], want[keep], slack[keep], f"variant {variant}")


def test_empty_sizes(handle):
    y = torch.full((4, 8), 3.0, dtype=torch.bfloat16, device="cuda")
    sw.swiglu_forward_mxfp4(handle, None, None, None, None, y, 4, 8, 0)
    torch.cuda.synchronize()
    assert bool((y == 0).all())  # empty sums
    sw.swiglu_forward_mxfp4(handle, None, None, None, None, None, 0, 8, 32)
    sw.swiglu_quantize_mxfp4(handle, None, None, None, 0, 32)
    sw.swiglu_dequantize_mxfp4(handle, None, None, None, 3, 0)


def test_refusals_write_nothing(handle):
    x = torch.ones(64, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(8192, dtype=torch.uint8, device="cuda")
    s = torch.zeros(512, dtype=torch.uint8, device="cuda")
    y = torch.full((64, 8), 3.0, dtype=torch.bfloat16, device="cuda")
    cases = [
        (lambda: sw.swiglu_quantize_mxfp4(handle, x, q, s, 64, 40), sw.ERR_UNSUPPORTED),
        (lambda: sw.swiglu_quantize_mxfp4(handle, x, q, None, 64, 64), sw.ERR_INVALID_ARG),
        (lambda: sw.swiglu_quantize_mxfp4(handle, x, x, s, 64, 64), sw.ERR_INVALID_ARG),
        (lambda: sw.swiglu_quantize_mxfp4(handle, x, q[4:], s, 32, 64), sw.ERR_UNSUPPORTED),
        (lambda: sw.swiglu_forward_mxfp4(handle, q, s, q, s, y, 64, 12, 64), sw.ERR_UNSUPPORTED),
        (lambda: sw.swiglu_forward_mxfp4(handle, q, s, q, s, y, 64, 8, 48), sw.ERR_UNSUPPORTED),
        (lambda: sw.swiglu_forward_mxfp4(handle, q, s, q, s, q, 64, 8, 64), sw.ERR_INVALID_ARG),
        (lambda: sw.swiglu_forward_mxfp4(handle, q, s, q, s, y, 64, 8, 64, variant=4),
         sw.ERR_INVALID_ARG),
    ]
    for call, status in cases:
        with pytest.raises(sw.SwiGLUError) as e:
            call()
        assert e.value.status == status
    torch.cuda.synchronize()
    assert bool((y == 3.0).all()) and bool((q == 0).all())


def test_graph_replays_equal_eager(handle):
    rng = np.random.default_rng(8)
    M, N, K = 48, 264, 320
    x, w = bf16(rng.standard_normal((M, K))).cuda(), bf16(rng.standard_normal((2 * N, K)) * 0.05)
    wq, ws = quantized(handle, w)
    q = torch.empty(sw.swiglu_mxfp4_bytes(M, K), dtype=torch.uint8, device="cuda")
    s = torch.empty(sw.swiglu_mxfp4_scale_bytes(M, K), dtype=torch.uint8, device="cuda")
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")

    def step():
        sw.swiglu_quantize_mxfp4(handle, x, q, s, M, K)
        sw.swiglu_forward_mxfp4(handle, q, s, wq, ws, y, M, N, K)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    eager = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(4):
        q.fill_(0x77), s.fill_(0), y.fill_(-1)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
