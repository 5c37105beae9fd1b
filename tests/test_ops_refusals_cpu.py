"""What the mixture-of-experts and MXFP4 entry points refuse, without a GPU.

A stand-in handle names a device that is never current, so a call whose
arguments pass every check ends at the device check (ERR_DEVICE) and no call
reaches a launch, on any machine.  Pointers are plain numbers: the checks do
not read through them."""
import ctypes

import pytest

import gemm_epilogues_mlp_amd as sw

OK, INVALID, UNSUPPORTED, DEVICE = sw.OK, sw.ERR_INVALID_ARG, sw.ERR_UNSUPPORTED, sw.ERR_DEVICE
GIB = 1 << 30
P = [(i + 1) * (1 << 44) for i in range(12)]  # far apart: no accidental overlap


@pytest.fixture(scope="module")
def handle():
    ctx = ctypes.create_string_buffer(b"\x7f" * 4096, 4096)
    yield ctypes.addressof(ctx)


def status(fn, defaults, changes):
    args = dict(defaults)
    args.update(changes)
    return getattr(sw.load(), fn)(*args.values())


def check(fn, defaults, cases):
    assert status(fn, defaults, {}) == DEVICE, "the default call is a good one"
    for changes, want in cases:
        assert status(fn, defaults, changes) == want, changes


def test_route(handle):
    T, E, k = 100, 64, 6
    d = dict(h=handle, x=P[0], w=P[1], e=P[2], off=P[3], rows=P[4], ws=P[5],
             wsb=sw.swiglu_route_workspace_bytes(T, E, k), T=T, E=E, k=k, renorm=1,
             dtype=sw.DTYPE_F32, stream=None)
    check("swiglu_route", d, [
        (dict(h=None), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
        (dict(e=None), INVALID), (dict(off=None), INVALID), (dict(rows=None), INVALID),
        (dict(ws=None), INVALID), (dict(wsb=d["wsb"] - 1), INVALID), (dict(T=-1), INVALID),
        (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(dtype=2), INVALID),
        (dict(dtype=-1), INVALID), (dict(E=1025), UNSUPPORTED), (dict(E=128, k=65), UNSUPPORTED),
        (dict(T=GIB // 6 + 1), UNSUPPORTED), (dict(T=1 << 62), UNSUPPORTED),
        (dict(x=P[0] + 2), UNSUPPORTED), (dict(w=P[1] + 2), UNSUPPORTED),
        (dict(ws=P[5] + 8), UNSUPPORTED), (dict(w=P[0] + 4 * T * E - 4), INVALID),
        (dict(e=P[1]), INVALID), (dict(ws=P[4]), INVALID),
        (dict(x=P[0] + 2, dtype=sw.DTYPE_BF16), DEVICE),
        (dict(w=P[0] + 4 * T * E), DEVICE), (dict(T=1, ws=None, wsb=0), DEVICE),
        (dict(T=0, x=None, w=None, e=None, rows=None, ws=None, wsb=0), DEVICE)])


def test_route_workspace_bytes():
    f = sw.swiglu_route_workspace_bytes
    assert f(1, 64, 6) == 0 and f(64, 64, 8) == 0  # one workgroup needs none
    assert f(8191, 128, 8) == 256 * 128 * 4        # a count for each of 256 workgroups and expert
    for bad in ((-1, 8, 1), (8, 0, 1), (8, 8, 9), (8, 8, 0), (8, 1025, 2), (GIB + 1, 8, 1),
                (8, 128, 65)):
        assert f(*bad) == 0


def grouped_cases(up):
    return [
        (dict(h=None), INVALID), (dict(A=None), INVALID), (dict(rows=None), INVALID),
        (dict(off=None), INVALID), (dict(W=None), INVALID), (dict(Y=None), INVALID),
        (dict(R=-1), INVALID), (dict(N=-8), INVALID), (dict(K=-8), INVALID), (dict(E=0), INVALID),
        (dict(variant=5), INVALID), (dict(N=60), UNSUPPORTED), (dict(K=36), UNSUPPORTED),
        (dict(E=1025), UNSUPPORTED), (dict(A=P[0] + 8), UNSUPPORTED), (dict(W=P[3] + 8), UNSUPPORTED),
        (dict(Y=P[4] + 2), UNSUPPORTED), (dict(rows=P[1] + 2), UNSUPPORTED),
        (dict(off=P[2] + 1), UNSUPPORTED), (dict(N=(1 << 23) + 8, K=8), UNSUPPORTED),
        (dict(K=1 << 24), UNSUPPORTED),                 # an expert's weights of 2 GiB and more
        (dict(R=1 << 40), UNSUPPORTED), (dict(N=1 << 62), UNSUPPORTED),
        (dict(Y=P[0]), INVALID), (dict(Y=P[3] + 64), INVALID), (dict(Y=P[1]), INVALID),
        (dict(R=0, A=None, rows=None, off=None, W=None, Y=None), OK), (dict(N=0, Y=None), OK),
        (dict(K=0, A=None, W=None), DEVICE), (dict(variant=4), DEVICE),
        (dict(E=1000, K=4096, N=4096), DEVICE),          # 32 GiB and more of experts
    ]


def test_grouped_forward(handle):
    d = dict(h=handle, A=P[0], rows=P[1], off=P[2], W=P[3], Y=P[4], T=10, R=20, N=64, K=40, E=8, k=2,
             variant=-1, stream=None)
    check("swiglu_grouped_forward", d, grouped_cases(True) + [
        (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(T=GIB // 40 + 1), UNSUPPORTED),
        (dict(T=0, A=None), DEVICE)])


def test_grouped_matmul(handle):
    d = dict(h=handle, A=P[0], rows=P[1], off=P[2], W=P[3], Y=P[4], R=20, N=64, K=40, E=8, variant=-1,
             stream=None)
    check("swiglu_grouped_matmul", d, grouped_cases(False) + [(dict(R=GIB // 40 + 1), UNSUPPORTED)])


def test_combine_norm(handle):
    d = dict(h=handle, B=P[0], w=P[1], e=P[2], S=P[3], X=P[4], post=P[5], gate=P[6], pre=P[7],
             out=P[8], H=P[9], T=10, D=64, k=2, scale=1.0, eps=1e-6, ld=64, dtype=sw.DTYPE_BF16,
             stream=None)
    check("swiglu_combine_norm", d, [
        (dict(h=None), INVALID), (dict(B=None), INVALID), (dict(w=None), INVALID),
        (dict(e=None), INVALID), (dict(X=None), INVALID), (dict(pre=None), INVALID),
        (dict(out=None), INVALID), (dict(H=None), INVALID), (dict(T=-1), INVALID),
        (dict(D=-8), INVALID), (dict(k=-1), INVALID), (dict(ld=-8), INVALID), (dict(ld=56), INVALID),
        (dict(dtype=3), INVALID), (dict(D=60), UNSUPPORTED), (dict(D=16392, ld=16392), UNSUPPORTED),
        (dict(ld=68), UNSUPPORTED), (dict(X=P[4] + 8), UNSUPPORTED), (dict(w=P[1] + 2), UNSUPPORTED),
        (dict(gate=P[6] + 8), UNSUPPORTED), (dict(T=1 << 40), UNSUPPORTED),
        (dict(k=1 << 45), UNSUPPORTED), (dict(H=P[4]), INVALID), (dict(H=P[8]), INVALID),
        (dict(out=P[0] + 16), INVALID), (dict(out=P[4] + 16), INVALID), (dict(H=P[6]), INVALID),
        (dict(out=P[4]), DEVICE),                        # the stream updated in place
        (dict(S=None, post=None, gate=None), DEVICE), (dict(k=0, B=None, w=None, e=None), DEVICE),
        (dict(ld=0), DEVICE), (dict(T=0, X=None, out=None), OK), (dict(D=0, X=None), OK)])


@pytest.mark.parametrize("back", [False, True])
def test_quantize_mxfp4(handle, back):
    a = dict(X=P[0], Q=P[1], S=P[2])
    d = dict(h=handle, **({n: a[n] for n in ("Q", "S", "X")} if back else a), rows=10, K=64,
             stream=None)
    cases = [(dict(h=None), INVALID), (dict(X=None), INVALID), (dict(Q=None), INVALID),
             (dict(S=None), INVALID), (dict(rows=-1), INVALID), (dict(K=-32), INVALID),
             (dict(K=48), UNSUPPORTED), (dict(X=P[0] + 8), UNSUPPORTED),
             (dict(Q=P[1] + 8), UNSUPPORTED), (dict(S=P[2] + 4), UNSUPPORTED),
             (dict(rows=1 << 40), UNSUPPORTED), (dict(rows=1 << 30, K=1 << 30), UNSUPPORTED),
             (dict(X=P[1]), INVALID), (dict(X=P[2]), INVALID), (dict(rows=0, X=None), OK),
             (dict(K=0, Q=None), OK)]
    if not back:
        cases.append((dict(S=P[1]), INVALID))            # both are outputs
    check("swiglu_dequantize_mxfp4" if back else "swiglu_quantize_mxfp4", d, cases)


def test_forward_mxfp4(handle):
    d = dict(h=handle, Q=P[0], SQ=P[1], W=P[2], SW=P[3], Y=P[4], M=10, N=64, K=64, variant=-1,
             stream=None)
    check("swiglu_forward_mxfp4", d, [
        (dict(h=None), INVALID), (dict(Q=None), INVALID), (dict(SQ=None), INVALID),
        (dict(W=None), INVALID), (dict(SW=None), INVALID), (dict(Y=None), INVALID),
        (dict(M=-1), INVALID), (dict(N=-8), INVALID), (dict(K=-32), INVALID), (dict(variant=4), INVALID),
        (dict(N=60), UNSUPPORTED), (dict(K=48), UNSUPPORTED), (dict(Y=P[4] + 8), UNSUPPORTED),
        (dict(Q=P[0] + 8), UNSUPPORTED), (dict(SW=P[3] + 8), UNSUPPORTED),
        (dict(K=(1 << 22) + 32), UNSUPPORTED), (dict(M=1 << 30), UNSUPPORTED),
        (dict(M=1 << 24, variant=0), UNSUPPORTED),       # more row groups than a grid has
        (dict(Y=P[0]), INVALID), (dict(Y=P[1]), INVALID), (dict(Y=P[2]), INVALID),
        (dict(Y=P[3]), INVALID), (dict(K=0, Q=None, SQ=None, W=None, SW=None), DEVICE),
        (dict(M=0, Y=None), OK), (dict(N=0, Y=None), OK)])


def test_mxfp4_bytes():
    assert sw.swiglu_mxfp4_bytes(1, 32) == 4096 and sw.swiglu_mxfp4_scale_bytes(1, 32) == 256
    assert sw.swiglu_mxfp4_bytes(33, 288) == 4 * 4096 and sw.swiglu_mxfp4_scale_bytes(33, 288) == 4 * 256
    for bad in ((0, 32), (4, 0), (-1, 32), (4, -1), (1 << 31, 32), (4, 1 << 31)):
        assert sw.swiglu_mxfp4_bytes(*bad) == 0 and sw.swiglu_mxfp4_scale_bytes(*bad) == 0
