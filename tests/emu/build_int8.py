"""Build the CPU bounds and LDS-ordering emulation of the 8-bit integer kernels
(host clang++ with AddressSanitizer) from their current source.  Returns the binary
path.  The rewrites are those of build_ops.py, and one more: the threads of a workgroup run
one after another, so a slot that another wave's DMA brings is not there yet; its LDS read is
logged and its value taken from memory.  The planted mistakes are off unless the driver is
run with --plant N."""
import os
import re
import shutil
import subprocess

import build as emu_build

HERE, CSRC = emu_build.HERE, emu_build.CSRC
NAME = "swiglu_int8.hip"
SLOTS = [
    (r"const int slot = (reinterpret_cast<const int\*>\(smem \+ C::ROW_OFF \+ par \* 4 \* BM\)\[r\]);",
     r"const int there = \1; ::emu_use(&there, 4); const int slot = r < o.rows ? a.rows[o.pos0 + r] : -1;", 2),
    (r"row = slots\[r\];",
     r"{ const int there = slots[r]; ::emu_use(&there, 4); row = r < cur.rows ? a.rows[cur.pos0 + r] : -1; }", 1),
]
# 1: the tile's ring waits for one stage fewer
# 2: the kernel ends without draining the loads issued past its last tile
# 3: the first tile's slots are read without the wait for them
# 4: a tile's slots are asked for when its scales are
PLANTS = [
    (r"^      wait_vmcnt<2 \* C::LOADS>\(\);$",
     "      if (::g_emu_plant == 1) wait_vmcnt<3 * C::LOADS>(); else wait_vmcnt<2 * C::LOADS>();"),
    (r"^(  // the zero loads issued past the last tile still write LDS\n)  wait_vmcnt<0>\(\);$",
     "\\1  if (::g_emu_plant != 2) wait_vmcnt<0>();"),
    (r"^(    load_slots\(cur, 0\);\n)    wait_vmcnt<0>\(\);$", "\\1    if (::g_emu_plant != 3) wait_vmcnt<0>();"),
    (r"KIND == kFirst && nxt.rows > 0\) load_slots",
     "(::g_emu_plant == 4 ? KIND == kBeforeLast : KIND == kFirst) && nxt.rows > 0) load_slots"),
]


def rewrite(src: str) -> str:
    src = re.sub(r"__shared__\s+__attribute__\(\(aligned\(\d+\)\)\)\s+uint8_t\s+(\w+)\[([^\]]+)\];",
                 r"uint8_t* \1 = ::emu_lds(\2);", src)
    src = re.sub(r"__shared__\s+__attribute__\(\(aligned\(\d+\)\)\)\s+(\w+)\s+(\w+)\[([^\]]+)\];",
                 r"\1* \2 = reinterpret_cast<\1*>(::emu_lds(sizeof(\1) * (\3)));", src)
    src = src.replace('#include "swiglu_ops_device.hpp"', '#include "int8_device.hpp"')
    if "__shared__" in src or "asm volatile" in src or "hipLaunchKernel" in src:
        raise RuntimeError(f"{NAME}: a construct the emulation does not rewrite")
    for pattern, repl, count in SLOTS:
        src, n = re.subn(pattern, repl, src)
        if n != count:
            raise RuntimeError(f"{NAME}: slots read {n} times: {pattern}")
    for pattern, repl in PLANTS:
        src, n = re.subn(pattern, repl, src, flags=re.M)
        if n != 1:
            raise RuntimeError(f"{NAME}: plant point found {n} times: {pattern}")
    return src


def build(out_dir: str) -> str:
    cc = emu_build.clangxx()
    if cc is None:
        raise RuntimeError("clang++ not found")
    os.makedirs(out_dir, exist_ok=True)
    with open(os.path.join(CSRC, NAME)) as f:
        src = rewrite(f.read())
    with open(os.path.join(out_dir, "swiglu_int8_emu.cpp"), "w") as f:
        f.write(src)
    shutil.copy(os.path.join(CSRC, "swiglu_internal.h"), out_dir)
    for name in ("swiglu_device.hpp", "swiglu_ops_device.hpp", "int8_device.hpp", "emu_int8_driver.cpp",
                 "emu_race.cpp"):
        shutil.copy(os.path.join(HERE, name), out_dir)
    exe = os.path.join(out_dir, "emu_int8_driver")
    common = [cc, "-std=c++20", "-O1", "-g", "-fsanitize=address", "-fno-omit-frame-pointer",
              "-Wno-unknown-attributes", "-Wno-ignored-attributes", "-Wno-psabi", "-I", out_dir,
              "-I", HERE]
    race_o = os.path.join(out_dir, "emu_race.o")
    subprocess.run(common + ["-c", os.path.join(out_dir, "emu_race.cpp"), "-o", race_o], check=True)
    subprocess.run(common + ["-fsanitize-coverage=func,trace-loads,trace-stores",
                             os.path.join(out_dir, "emu_int8_driver.cpp"), race_o, "-o", exe],
                   check=True)
    return exe


if __name__ == "__main__":
    import sys
    print(build(sys.argv[1] if len(sys.argv) > 1 else "/tmp/swiglu_emu_int8"))
