"""The direct loads to LDS of every kernel, in the machine code of the built library (no GPU).

They stand in inline assembly, for which the compiler counts no wait states.  A vector memory
instruction may read a scalar register five states after a vector instruction (v_readfirstlane,
v_readlane, a comparison) wrote it at the earliest, and a load to LDS may read M0 one state after a
scalar write.  A load that comes earlier may take an old base or bound and reach past its tensor.

Every word of a load's resource is followed back over all paths that lead to it, branches and the
ends of loops included."""
import re
import subprocess

import pytest

import gemm_epilogues_mlp_amd as sw
from test_code_objects_cpu import MAGIC
from test_kernel_resources_cpu import _tool

VALU_STATES, M0_STATES = 5, 1


def scalars(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$", operand)
    if m:
        return {f"s{i}" for i in range(int(m[1]), int(m[2]) + 1)}
    return {operand} if re.match(r"(s\d+|m0|vcc)$", operand) else set()


def kernels(listing):
    """(name, start, [(address, opcode, operands, comment)]) of every function of a disassembly."""
    name, start, body = None, 0, []
    for line in listing:
        m = re.match(r"^([0-9a-f]+) <(\w+)>:", line)
        if m:
            if name:
                yield name, start, body
            name, start, body = m[2], int(m[1], 16), []
            continue
        m = re.match(r"^\s+([a-z]\w+)(.*?)\s*// ([0-9A-F]+):(.*)$", line)
        if m:
            body.append((int(m[3], 16), m[1], m[2].strip(), m[4]))
    if name:
        yield name, start, body


def operands(text):
    return [a.strip().split(" ")[0] for a in text.split(",")]


def is_load(op, text):
    return op.startswith("buffer_load") and text.endswith(" lds")


class Step:
    """What an instruction does to the ages of scalar registers, and where it goes."""

    def __init__(self, name, start, body, i, at):
        _, op, text, comment = body[i]
        args = operands(text)
        self.load = is_load(op, text)
        self.reads = set().union(*map(scalars, args)) if self.load else set()
        self.states = int(text, 0) + 1 if op == "s_nop" else 1
        self.valu, self.salu = set(), set()
        if op.startswith("v_"):
            self.valu = scalars(args[0])
            if len(args) > 1 and ("_co_" in op or op.startswith("v_div_scale")):
                self.valu |= scalars(args[1])
        elif op.startswith("s_") and not re.match(r"s_(cmp|bitcmp|cbranch|branch|waitcnt|barrier|nop)", op):
            self.salu = scalars(args[0])
        self.next = []
        if op not in ("s_endpgm", "s_branch", "s_setpc_b64") and i + 1 < len(body):
            self.next.append(i + 1)
        if op.startswith(("s_cbranch", "s_branch")):
            m = re.search(r"<" + re.escape(name) + r"(?:\+0x([0-9a-f]+))?>", comment)
            assert m, (name, op, text, comment)
            self.next.append(at[start + int(m[1] or "0", 16)])


def too_early(name, start, body):
    """({address of a load: {register: states since its write}}, number of loads) of one function."""
    at = {a: i for i, (a, *_) in enumerate(body)}
    steps = [Step(name, start, body, i, at) for i in range(len(body))]
    loads = sum(s.load for s in steps)
    if not loads:
        return {}, 0
    # registers written by vector instructions, and M0 by a scalar one ("M0"), with the fewest states
    # that have passed since on any path
    before, found, work = {0: {}}, {}, [0]
    while work:
        i = work.pop()
        ages = dict(before[i])
        while True:
            s = steps[i]
            if s.load:
                for r in (s.reads | {"m0", "M0"}) & set(ages):
                    if ages[r] < (M0_STATES if r == "M0" else VALU_STATES):
                        seen = found.setdefault(body[i][0], {})
                        seen[r] = min(ages[r], seen.get(r, ages[r]))
            ages = {r: n + s.states for r, n in ages.items() if n + s.states < VALU_STATES}
            for r in s.salu:
                ages.pop(r, None)
            if "m0" in s.salu:
                ages["M0"] = 0
            ages.update(dict.fromkeys(s.valu, 0))
            if s.next == [i + 1] and i + 1 not in before:
                i += 1
                continue
            break
        for n in s.next:
            known = before.get(n)
            if known is None:
                before[n] = dict(ages)
                work.append(n)
            elif any(a < known.get(r, VALU_STATES) for r, a in ages.items()):
                for r, a in ages.items():
                    known[r] = min(a, known.get(r, a))
                work.append(n)
    return found, loads


@pytest.fixture(scope="module")
def objects(tmp_path_factory):
    """The disassembly of each code object of the library that has kernels."""
    objcopy, bundler, objdump = _tool("llvm-objcopy"), _tool("clang-offload-bundler"), _tool("llvm-objdump")
    if not (objcopy and bundler and objdump):
        pytest.skip("ROCm LLVM tools not found")
    d = tmp_path_factory.mktemp("waits")
    fat = d / "fat.bin"
    subprocess.run([objcopy, "--dump-section", f".hip_fatbin={fat}", sw.lib_path(), str(d / "copy.so")],
                   check=True)
    data = fat.read_bytes()
    at = [m.start() for m in re.finditer(re.escape(MAGIC), data)]
    out = []
    for i, (a, b) in enumerate(zip(at, at[1:] + [len(data)])):
        part, obj = d / f"part{i}", d / f"gfx950_{i}.o"
        part.write_bytes(data[a:b])
        subprocess.run([bundler, "--unbundle", "--type=o", f"--input={part}",
                        "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", f"--output={obj}"], check=True)
        out.append(subprocess.run([objdump, "-d", "--no-show-raw-insn", str(obj)], check=True,
                                  capture_output=True, text=True).stdout.splitlines())
    return out


def test_no_load_reads_a_scalar_too_early(objects):
    total, bad = {}, {}
    for listing in objects:
        for name, start, body in kernels(listing):
            found, loads = too_early(name, start, body)
            if loads:
                total[name] = loads
            if found:
                bad[name] = (len(found), next(iter(found.items())))
    for part in ("tiled_kernel", "tiled_persist_kernel", "tiled_split_kernel", "f8_kernel", "f8_split_kernel",
                 "grouped_tile_kernel", "fp4_tile_kernel", "int8_tile_kernel"):
        assert any(part in n for n in total), part
    assert sum(total.values()) > 4000
    assert not bad, (sum(n for n, _ in bad.values()), list(bad.items())[:3])


# ---- the search itself, on listings written by hand
LOAD = "buffer_load_dwordx4 v1, s[8:11], 0 offen lds"


def seen(*lines):
    """Registers found at the loads of a function of these lines, "label:" and "op -> label" among them."""
    labels, body, at = {}, [], 0x1000
    for line in lines:
        if line.endswith(":"):
            labels[line[:-1]] = at
        else:
            body.append((at, line))
            at += 4
    text = ["0000000000001000 <kernel>:"]
    for at, line in body:
        op, _, label = line.partition(" -> ")
        to = f" <kernel+0x{labels[label] - 0x1000:x}>" if label else ""
        text.append(f"\t{op}{' 7' if label else ''}  // {at:012X}: BF8800F5{to}")
    name, start, parsed = next(kernels(text))
    found, _ = too_early(name, start, parsed)
    return set().union(*map(set, found.values())) if found else set()


def test_words_written_too_early_are_each_seen():
    one, two = "v_readfirstlane_b32 s10, v2", "v_readlane_b32 s8, v2, 3"
    assert seen(one, two, LOAD) == {"s8", "s10"}
    assert seen(one, "s_nop 3", LOAD) == {"s10"}
    assert seen(one, "s_nop 4", LOAD) == set()
    assert seen(one, *["v_mov_b32_e32 v1, v2"] * 4, LOAD) == {"s10"}
    assert seen(one, *["v_mov_b32_e32 v1, v2"] * 5, LOAD) == set()
    assert seen("v_readfirstlane_b32 s12, v2", LOAD) == set()
    assert seen("v_cmp_gt_i32_e64 s[10:11], v1, v2", LOAD) == {"s10", "s11"}
    # a scalar instruction has written it since, which the hardware waits for
    assert seen(one, "s_mov_b32 s10, s4", LOAD) == set()


def test_m0_written_too_early_is_seen():
    assert seen("s_mov_b32 m0, s3", LOAD) == {"M0"}
    assert seen("s_mov_b32 m0, s3", "s_nop 0", LOAD) == set()
    assert seen("v_readfirstlane_b32 m0, v3", "s_nop 0", LOAD) == {"m0"}


def test_writes_on_other_paths_are_seen():
    one = "v_readfirstlane_b32 s10, v2"
    # at the end of a loop, before the load at its head
    assert seen("head:", LOAD, "s_nop 4", one, "s_cbranch_scc1 -> head", "s_endpgm") == {"s10"}
    assert seen("head:", LOAD, one, "s_nop 4", "s_cbranch_scc1 -> head", "s_endpgm") == set()
    # on one of two ways to it
    assert seen("s_nop 4", "s_cbranch_scc1 -> far", "s_nop 4", "s_branch -> load", "far:", one, "load:", LOAD,
                "s_endpgm") == {"s10"}
    # past an unconditional branch there is no way
    assert seen(one, "s_branch -> far", LOAD, "far:", "s_nop 7", LOAD, "s_endpgm") == set()
