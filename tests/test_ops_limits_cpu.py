"""Sizes at the ends of what the mixture-of-experts and MXFP4 entry points
take, without a GPU: the largest ones, and those whose byte counts pass 64 bits.

As in test_ops_refusals_cpu.py the stand-in handle's device is never current:
a call that passes every check ends with ERR_DEVICE, and none launches."""
import ctypes
import os
import shutil
import subprocess

import pytest

import gemm_epilogues_mlp_amd as sw

DEVICE, UNSUPPORTED = sw.ERR_DEVICE, sw.ERR_UNSUPPORTED
HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gemm_epilogues_mlp_amd", "csrc")
P = [(i + 1) * (1 << 48) for i in range(12)]  # far apart: no accidental overlap


@pytest.fixture(scope="module")
def handle():
    ctx = ctypes.create_string_buffer(b"\x7f" * 4096, 4096)
    yield ctypes.addressof(ctx)


def norm(handle, T, D, k=2, ld=0, dtype=sw.DTYPE_BF16):
    return sw.load().swiglu_combine_norm(handle, P[0], P[1], P[2], P[3], P[4], P[5], P[6], P[7],
                                         P[8], P[9], T, D, k, 1.0, 1e-6, ld, dtype, None)


def test_norm_gate_stride(handle):
    """A gate's row stride whose bytes pass 64 bits is refused, not wrapped."""
    assert norm(handle, 10, 64, ld=1 << 40) == DEVICE
    for bits in range(43, 63):
        assert norm(handle, 10, 64, ld=1 << bits) == UNSUPPORTED, bits
        assert norm(handle, 10, 64, ld=(1 << bits) + 64) == UNSUPPORTED, bits
    assert norm(handle, 10, 64, ld=(1 << 63) - 8) == UNSUPPORTED


def test_no_size_overflows_a_check(tmp_path):
    """The checks themselves under the undefined-behaviour sanitizer (a host build), each
    size swept to both ends of 64 bits."""
    cxx = next((c for c in ("/opt/rocm/llvm/bin/clang++", shutil.which("g++"), shutil.which("clang++"))
                if c and os.path.exists(c)), None)
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "checks_driver")
    subprocess.run([cxx, "-std=c++20", "-O0", "-g", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-I", os.path.join(HERE, "emu"), "-I", CSRC,
                    os.path.join(HERE, "checks", "checks_driver.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), r.stdout + r.stderr


# A launch has fewer than 2^32 threads along x: what would need more is refused with the
# other sizes, before anything else happens, not by the launch.
def test_norm_launch_size(handle):
    for D, most in ((8, 2 ** 26 - 4), (2048, 2 ** 26 - 4), (2056, 2 ** 23 - 1), (8192, 2 ** 23 - 1),
                    (8200, 2 ** 22 - 1), (16384, 2 ** 22 - 1)):
        for dtype in (sw.DTYPE_BF16, sw.DTYPE_F32):
            assert norm(handle, most, D, k=1, dtype=dtype) == DEVICE, D
            assert norm(handle, most + 1, D, k=1, dtype=dtype) == UNSUPPORTED, D


def up(handle, R, N, K, E, variant):
    return sw.load().swiglu_grouped_forward(handle, P[0], P[1], P[2], P[3], P[4], 8, R, N, K, E, 1,
                                            variant, None)


def test_grouped_launch_size(handle):
    # one expert, K = 8: workgroups of R rows in tiles, 2 N weight columns in tiles (the tiles of
    # 128 x 128 and 256 x 256 run at most twice as many workgroups, and only below 1024 of them)
    for variant, bm, bnw, threads in ((0, 16, 128, 512), (1, 64, 128, 256), (2, 128, 128, 256),
                                      (3, 256, 256, 512), (4, 64, 64, 256)):
        cols = 2 ** 12                       # column tiles
        rows = 2 ** 32 // threads // cols    # row tiles that make 2^32 threads
        N = cols * bnw // 2
        assert up(handle, (rows - 1) * bm, N, 8, 1, variant) == DEVICE, variant
        assert up(handle, (rows - 1) * bm + 1, N, 8, 1, variant) == UNSUPPORTED, variant
    # the same rows in the kernel that the rule takes for them
    assert up(handle, 2 ** 15, 2 ** 18, 8, 1, 0) == UNSUPPORTED
    assert up(handle, 2 ** 15, 2 ** 18, 8, 1, -1) == DEVICE


@pytest.mark.parametrize("name", ["swiglu_quantize_mxfp4", "swiglu_dequantize_mxfp4"])
def test_mxfp4_conversion_launch_size(handle, name):
    rows = 32 * (2 ** 24 - 1)                # 64 GiB of codes less a block
    assert getattr(sw.load(), name)(handle, P[0], P[1], P[2], rows, 256, None) == DEVICE
    assert getattr(sw.load(), name)(handle, P[0], P[1], P[2], rows + 1, 256, None) == UNSUPPORTED


def test_mxfp4_product_launch_size(handle):
    f = sw.load().swiglu_forward_mxfp4
    for variant in (-1, 0, 1, 2, 3):         # K = 0: no weights, whose 2 GiB end sooner
        assert f(handle, None, None, None, None, P[4], 8, 2 ** 27 - 16, 0, variant, None) == DEVICE
        assert f(handle, None, None, None, None, P[4], 8, 2 ** 27, 0, variant, None) == UNSUPPORTED
