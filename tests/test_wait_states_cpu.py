"""A scalar register that a vector instruction wrote (v_readfirstlane, v_readlane) may be read by a
vector memory instruction five wait states later at the earliest.  The compiler keeps that for the
instructions it emits, not for those inside asm, as the direct loads to LDS are: read too early, the
stale base or bound of a buffer resource lets a load past its tensor through.  The 8-bit integer
kernels make resources as they go, so the machine code of the built library is looked over here (no
GPU)."""
import re
import subprocess

import pytest

import gemm_epilogues_mlp_amd as sw
from test_code_objects_cpu import MAGIC
from test_kernel_resources_cpu import _tool

STATES = 5


def scalars(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.match(r"s(\d+)$", operand)
    return {int(m[1])} if m else set()


def too_early(lines):
    """(kernel, instruction that wrote, load) of every LDS load that reads a scalar too early, and how
    many loads there are, in a disassembly."""
    found, loads, kernel, last = [], 0, "", []
    for line in lines:
        m = re.match(r"^[0-9a-f]+ <(\w+)>:", line)
        if m:
            kernel, last = m[1], []
            continue
        text = line.split("//")[0].strip()
        if not text or text.endswith(":") or not re.match(r"^[a-z]+_", text):
            continue
        op, _, rest = text.partition(" ")
        args = [a.strip().split(" ")[0] for a in rest.split(",")]
        if op.startswith("buffer_load") and text.endswith(" lds"):
            loads += 1
            reads = set().union(*map(scalars, args))
            states = 0
            for o, writes, t in reversed(last):
                if states >= STATES:
                    break
                if o.startswith("v_") and writes & reads:
                    found.append((kernel, t, text))
                    break
                states += int(t.split()[1], 0) + 1 if o == "s_nop" else 1
        last = (last + [(op, scalars(args[0]) if args else set(), text)])[-2 * STATES:]
    return found, loads


@pytest.fixture(scope="module")
def disassembly(tmp_path_factory):
    objcopy, bundler, objdump = _tool("llvm-objcopy"), _tool("clang-offload-bundler"), _tool("llvm-objdump")
    if not (objcopy and bundler and objdump):
        pytest.skip("ROCm LLVM tools not found")
    d = tmp_path_factory.mktemp("waits")
    fat = d / "fat.bin"
    subprocess.run([objcopy, "--dump-section", f".hip_fatbin={fat}", sw.lib_path(), str(d / "copy.so")],
                   check=True)
    data = fat.read_bytes()
    at = [m.start() for m in re.finditer(re.escape(MAGIC), data)]
    for a, b in zip(at, at[1:] + [len(data)]):
        if b"int8_tile_kernel" in data[a:b]:
            part, obj = d / "part", d / "gfx950.o"
            part.write_bytes(data[a:b])
            subprocess.run([bundler, "--unbundle", "--type=o", f"--input={part}",
                            "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", f"--output={obj}"], check=True)
            return subprocess.run([objdump, "-d", "--no-show-raw-insn", str(obj)], check=True,
                                  capture_output=True, text=True).stdout.splitlines()
    raise AssertionError("no code object with the 8-bit integer tiles")


def test_int8_loads_wait_for_their_resources(disassembly):
    found, loads = too_early(disassembly)
    assert loads > 500
    assert not found, found[:5]


def test_a_load_too_early_is_seen():
    load = "buffer_load_dwordx4 v1, s[8:11], 0 offen lds"
    write = "v_readfirstlane_b32 s10, v2"
    head = "0000000000001000 <kernel>:"
    assert too_early([head, write, "s_nop 3", load])[0] == [("kernel", write, load)]
    assert too_early([head, write, "s_mov_b32 m0, s3", "s_nop 2", load])[0] == [("kernel", write, load)]
    for between in (["s_nop 4"], ["s_nop 1", "v_mov_b32_e32 v1, v2"] * 2, ["s_mov_b32 s10, s4"] * 5):
        assert too_early([head, write, *between, load]) == ([], 1)
    assert too_early([head, "v_readfirstlane_b32 s12, v2", load]) == ([], 1)
