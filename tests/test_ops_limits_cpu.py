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
