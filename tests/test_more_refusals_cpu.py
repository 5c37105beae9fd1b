"""What the scored router and the 8-bit integer entry points refuse, and the sizes at the ends of
what they take, without a GPU.

As in test_ops_refusals_cpu.py: a stand-in handle names a device that is never current, so a call
that passes every check ends at the device check (ERR_DEVICE) and none reaches a launch."""
import ctypes
import os
import shutil
import subprocess

import pytest

import gemm_epilogues_mlp_amd as sw

OK, INVALID, UNSUPPORTED, DEVICE = sw.OK, sw.ERR_INVALID_ARG, sw.ERR_UNSUPPORTED, sw.ERR_DEVICE
GIB = 1 << 30
P = [(i + 1) * (1 << 47) for i in range(12)]  # far apart: no accidental overlap
HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gemm_epilogues_mlp_amd", "csrc")


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


def test_route_scored(handle):
    T, E, k = 100, 64, 6
    d = dict(h=handle, x=P[0], b=P[6], w=P[1], e=P[2], off=P[3], rows=P[4], ws=P[5],
             wsb=sw.swiglu_route_workspace_bytes(T, E, k), T=T, E=E, k=k, score=sw.SCORE_SIGMOID, renorm=1,
             scale=2.5, groups=8, top=4, best=2, dtype=sw.DTYPE_F32, stream=None)
    check("swiglu_route_scored", d, [
        (dict(h=None), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
        (dict(e=None), INVALID), (dict(off=None), INVALID), (dict(rows=None), INVALID),
        (dict(ws=None), INVALID), (dict(wsb=d["wsb"] - 1), INVALID), (dict(T=-1), INVALID),
        (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(dtype=2), INVALID),
        (dict(score=2), INVALID), (dict(score=-1), INVALID), (dict(groups=0), INVALID),
        (dict(groups=-8), INVALID), (dict(groups=7), INVALID), (dict(groups=128), INVALID),
        (dict(top=0), INVALID), (dict(top=9), INVALID), (dict(best=0), INVALID), (dict(best=3), INVALID),
        (dict(top=1, k=9, wsb=GIB), INVALID),            # one group of 8 has no 9 experts
        (dict(top=1, k=8, wsb=GIB), DEVICE), (dict(groups=1, top=1, best=1), DEVICE),
        (dict(groups=64, top=6), DEVICE), (dict(E=128, groups=128, top=64, wsb=GIB), UNSUPPORTED),
        (dict(E=1025, groups=1, top=1, wsb=GIB), UNSUPPORTED),
        (dict(E=128, groups=1, top=1, k=65, wsb=GIB), UNSUPPORTED), (dict(T=GIB // 6 + 1), UNSUPPORTED),
        (dict(T=1 << 62), UNSUPPORTED), (dict(x=P[0] + 2), UNSUPPORTED), (dict(b=P[6] + 2), UNSUPPORTED),
        (dict(ws=P[5] + 8), UNSUPPORTED), (dict(w=P[0] + 4 * T * E - 4), INVALID), (dict(e=P[1]), INVALID),
        (dict(w=P[6]), INVALID), (dict(off=P[6] + 4 * E - 4), INVALID), (dict(ws=P[6] + 16), INVALID),
        (dict(b=None), DEVICE), (dict(off=P[6] + 4 * E), DEVICE),
        (dict(T=0, x=None, w=None, e=None, rows=None, ws=None, wsb=0), DEVICE)])


def test_quantize_int8(handle):
    d = dict(h=handle, X=P[0], Q=P[1], S=P[2], rows=10, K=64, stream=None)
    check("swiglu_quantize_int8", d, [
        (dict(h=None), INVALID), (dict(X=None), INVALID), (dict(Q=None), INVALID), (dict(S=None), INVALID),
        (dict(rows=-1), INVALID), (dict(K=-16), INVALID), (dict(K=24), UNSUPPORTED),
        (dict(K=1 << 17), UNSUPPORTED), (dict(K=(1 << 17) - 16), DEVICE), (dict(X=P[0] + 8), UNSUPPORTED),
        (dict(Q=P[1] + 8), UNSUPPORTED), (dict(S=P[2] + 2), UNSUPPORTED), (dict(S=P[2] + 4), DEVICE),
        (dict(rows=1 << 40), UNSUPPORTED), (dict(rows=(1 << 62) + 1), UNSUPPORTED), (dict(Q=P[0]), INVALID),
        (dict(Q=P[0] + 2 * 640 - 16), INVALID), (dict(Q=P[0] + 2 * 640), DEVICE), (dict(S=P[1]), INVALID),
        (dict(S=P[0] + 1276), INVALID), (dict(rows=0, X=None), OK), (dict(K=0, Q=None), OK)])


def test_quantize_int8_launch_size(handle):
    f = sw.load().swiglu_quantize_int8
    # a wave a row for the narrowest, 16 for the widest
    for K, threads in ((16, 64), (1024, 64), (1040, 256), (8192, 256), (8208, 512), (16384, 512),
                       (16400, 1024), (131056, 1024)):
        most = (2 ** 32 - 1) // threads // 4 * 4
        assert f(handle, P[0], P[1], P[2], min(most, 2 ** 26 - 4), K, None) == DEVICE, K
        assert f(handle, P[0], P[1], P[2], most + 4, K, None) == UNSUPPORTED, K
        assert f(handle, P[0], P[1], P[2], 2 ** 22 - 1, K, None) == DEVICE, K


def test_pack_int8(handle):
    d = dict(h=handle, W=P[0], P=P[1], E=2, rows=40, K=144, stream=None)
    n = sw.swiglu_int8_packed_bytes(40, 144)
    check("swiglu_pack_int8_fragments", d, [
        (dict(h=None), INVALID), (dict(W=None), INVALID), (dict(P=None), INVALID), (dict(E=-1), INVALID),
        (dict(rows=-1), INVALID), (dict(K=-16), INVALID), (dict(K=24), UNSUPPORTED),
        (dict(W=P[0] + 8), UNSUPPORTED), (dict(P=P[1] + 8), UNSUPPORTED),
        (dict(rows=1 << 20, K=2048), UNSUPPORTED), (dict(rows=(1 << 20) - 32, K=2048), DEVICE),
        (dict(E=1 << 40), UNSUPPORTED), (dict(rows=1 << 40), UNSUPPORTED), (dict(K=1 << 40), UNSUPPORTED),
        (dict(P=P[0]), INVALID), (dict(W=P[1] + 2 * n - 16), INVALID), (dict(W=P[1] + 2 * n), DEVICE),
        (dict(E=0, W=None), OK), (dict(rows=0, W=None), OK), (dict(K=0, P=None), OK)])


def test_int8_packed_bytes():
    f = sw.swiglu_int8_packed_bytes
    assert f(1, 16) == 4096 and f(33, 144) == 4 * 4096 and f(37888, 3584) == 37888 * 3584
    for bad in ((0, 32), (4, 0), (-1, 32), (4, -1), (1 << 31, 32), (4, 1 << 31)):
        assert f(*bad) == 0


def product_cases(M, K):
    """For calls of `M` activation rows under the name `M`, width `K`."""
    return [
        (dict(h=None), INVALID), (dict(Q=None), INVALID), (dict(SQ=None), INVALID),
        (dict(P=None), INVALID), (dict(SW=None), INVALID), (dict(Y=None), INVALID),
        (dict(N=-8), INVALID), (dict(K=-16), INVALID), (dict(variant=8), INVALID), (dict(N=60), UNSUPPORTED),
        (dict(K=24), UNSUPPORTED), (dict(K=1 << 17), UNSUPPORTED), (dict(K=(1 << 17) - 16), DEVICE),
        (dict(Q=P[0] + 8), UNSUPPORTED), (dict(SQ=P[1] + 2), UNSUPPORTED), (dict(SQ=P[1] + 4), DEVICE),
        (dict(P=P[2] + 8), UNSUPPORTED), (dict(SW=P[3] + 4), UNSUPPORTED), (dict(Y=P[4] + 8), UNSUPPORTED),
        (dict(N=(1 << 23) + 8, K=16), UNSUPPORTED), (dict(N=1 << 20, K=2048), UNSUPPORTED),
        (dict(Y=P[0]), INVALID), (dict(Y=P[1]), INVALID), (dict(Y=P[2]), INVALID), (dict(Y=P[3]), INVALID),
        (dict(N=0, Y=None), OK), (dict(K=0, Q=None, SQ=None, P=None, SW=None), DEVICE),
        *((dict(variant=v), DEVICE) for v in range(8))]


@pytest.mark.parametrize("name", ["swiglu_forward_int8", "swiglu_matmul_int8"])
def test_dense_int8(handle, name):
    d = dict(h=handle, Q=P[0], SQ=P[1], P=P[2], SW=P[3], Y=P[4], M=10, N=64, K=64, variant=-1, stream=None)
    check(name, d, product_cases(10, 64) + [
        (dict(M=-1), INVALID), (dict(M=0, Y=None), OK), (dict(M=GIB // 32), UNSUPPORTED),
        (dict(M=GIB // 32 - 1), DEVICE), (dict(M=1 << 40), UNSUPPORTED), (dict(M=(1 << 63) - 1), UNSUPPORTED)])


@pytest.mark.parametrize("gated", [True, False], ids=["gated", "plain"])
def test_grouped_int8(handle, gated):
    d = dict(h=handle, Q=P[0], SQ=P[1], rows=P[5], off=P[6], P=P[2], SW=P[3], Y=P[4], T=10, R=20, N=64,
             K=64, E=8, k=2, variant=-1, stream=None)
    if not gated:
        del d["T"], d["k"]
    cases = product_cases(10, 64) + [
        (dict(rows=None), INVALID), (dict(off=None), INVALID), (dict(R=-1), INVALID), (dict(E=0), INVALID),
        (dict(E=1025), UNSUPPORTED), (dict(E=1000, N=4096, K=4096), DEVICE), (dict(rows=P[5] + 2), UNSUPPORTED),
        (dict(off=P[6] + 1), UNSUPPORTED), (dict(Y=P[5]), INVALID), (dict(Y=P[6] + 16), INVALID),
        (dict(R=1 << 40), UNSUPPORTED), (dict(N=1 << 62), UNSUPPORTED),
        (dict(R=0, Q=None, SQ=None, rows=None, off=None, P=None, SW=None, Y=None), OK)]
    cases += [(dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(T=GIB // 32), UNSUPPORTED),
              (dict(T=GIB // 32 - 1), DEVICE), (dict(T=0, Q=None, SQ=None), DEVICE)] if gated else \
        [(dict(R=GIB // 32), UNSUPPORTED)]
    check("swiglu_grouped_forward_int8" if gated else "swiglu_grouped_matmul_int8", d, cases)


def test_int8_launch_size(handle):
    """What a variant's grid does not hold is refused; the rule takes one that does."""
    dense, grouped = sw.load().swiglu_forward_int8, sw.load().swiglu_grouped_matmul_int8
    for v, rows in enumerate((16, 16, 32, 64)):
        most = 65535 * rows
        assert dense(handle, P[0], P[1], P[2], P[3], P[4], most, 8, 16, v, None) == DEVICE, v
        assert dense(handle, P[0], P[1], P[2], P[3], P[4], most + 1, 8, 16, v, None) == UNSUPPORTED, v
        assert dense(handle, P[0], P[1], P[2], P[3], P[4], most + 1, 8, 16, -1, None) == DEVICE, v
    for v, (rows, cols) in enumerate(((16, 16), (16, 32), (32, 32), (64, 64))):
        # one expert: pieces of 512 threads at most, in eights
        n = 2 ** 11
        args = (P[0], P[1], P[5], P[6], P[2], P[3], P[4])
        most = (2 ** 23 // n - 1) * rows
        assert grouped(handle, *args, most, n * cols, 16, 1, v, None) == DEVICE, v
        assert grouped(handle, *args, most + 1, n * cols, 16, 1, v, None) == UNSUPPORTED, v
        assert grouped(handle, *args, most + 1, n * cols, 16, 1, -1, None) == DEVICE, v
    for v, (rows, cols) in enumerate(((64, 128), (128, 128), (128, 256)), 4):
        # no K: nothing bounds the rows but the tiles' numbers (and Y's 2^46 bytes)
        n = 2 ** 23 // cols
        most = (2 ** 31 - 4097) // n * rows
        assert most * 2 ** 23 <= 2 ** 46
        for m, want in ((most, DEVICE), (most + 1, UNSUPPORTED)):
            assert dense(handle, None, None, None, None, P[4], m, 2 ** 22, 0, v, None) == want, v
    assert dense(handle, None, None, None, None, P[4], 2 ** 31 - 1025, 8, 0, -1, None) == DEVICE
    assert dense(handle, None, None, None, None, P[4], 2 ** 31 - 1023, 8, 0, -1, None) == UNSUPPORTED


def test_no_size_overflows_a_check(tmp_path):
    """The checks themselves under the undefined-behaviour sanitizer (a host build), each
    size swept to both ends of 64 bits."""
    cxx = next((c for c in ("/opt/rocm/llvm/bin/clang++", shutil.which("g++"), shutil.which("clang++"))
                if c and os.path.exists(c)), None)
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "int8_checks_driver")
    subprocess.run([cxx, "-std=c++20", "-O0", "-g", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-I", os.path.join(HERE, "emu"), "-I", CSRC,
                    os.path.join(HERE, "checks", "int8_checks_driver.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), r.stdout + r.stderr
