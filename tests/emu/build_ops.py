"""Build the CPU bounds and LDS-ordering emulation of the grouped products and
the MXFP4 kernels (host clang++ with AddressSanitizer) from their current
source.  Returns the binary path.

As build.py does for swiglu_kernels.hip: each `__shared__` array becomes a
pointer from emu_lds(), the empty asm statement that hides a value from the
compiler and the occupancy attribute are dropped; the launches go through the
stand-in's launch_op, which runs the workgroups on the host.  The planted
mistakes are off unless the driver is run with --plant N."""
import os
import re
import shutil
import subprocess

import build as emu_build

HERE, CSRC = emu_build.HERE, emu_build.CSRC
FILES = ("swiglu_grouped.hip", "swiglu_fp4.hip")

# 1: the grouped tile's K loop waits for one K step fewer of its DMA
# 2: a grouped tile reuses the stage ring for Y without the barrier that ends the K loop
# 3: the next unit's loads start without the barrier behind this one's rows of Y
# 4: the MXFP4 tile's ring waits for one stage fewer
# 5: the MXFP4 tile waits as if a group's scales were never in flight
# 6: the MXFP4 kernel ends without draining the loads issued past its last tile
# 7: the sums of the wave groups on other k are read without the barrier behind them
PLANTS = {
    "swiglu_grouped.hip": [
        (r"^        wait_vmcnt<\(STAGES - 2\) \* C::LOADS>\(\);$",
         "        if (::g_emu_plant == 1) wait_vmcnt<(STAGES - 1) * C::LOADS>();"
         " else wait_vmcnt<(STAGES - 2) * C::LOADS>();"),
        (r"^  wait_vmcnt<0>\(\);\n  __syncthreads\(\);\n(?=  uint16_t\* ys)",
         "  wait_vmcnt<0>();\n  if (::g_emu_plant != 2) __syncthreads();\n"),
        (r"^    __syncthreads\(\);  // the next unit's loads",
         "    if (::g_emu_plant != 3) __syncthreads();  // the next unit's loads"),
        (r"^    __syncthreads\(\);\n(?=    if \(kg == 0\))",
         "    if (::g_emu_plant != 7) __syncthreads();\n"),
    ],
    "swiglu_fp4.hip": [
        (r"^      wait_vmcnt<C::IN_FLIGHT>\(\);$",
         "      if (::g_emu_plant == 4) wait_vmcnt<C::IN_FLIGHT + C::LOADS>();"
         " else if (::g_emu_plant == 5) wait_vmcnt<C::IN_FLIGHT + C::SC_LOADS>();"
         " else wait_vmcnt<C::IN_FLIGHT>();"),
        (r"^(  // the zero loads issued past the last tile still write LDS\n)  wait_vmcnt<0>\(\);$",
         "\\1  if (::g_emu_plant != 6) wait_vmcnt<0>();"),
    ],
}


def rewrite(name: str, src: str) -> str:
    src = re.sub(r"__shared__\s+__attribute__\(\(aligned\(\d+\)\)\)\s+uint8_t\s+(\w+)\[([^\]]+)\];",
                 r"uint8_t* \1 = ::emu_lds(\2);", src)
    src = re.sub(r"__shared__\s+__attribute__\(\(aligned\(\d+\)\)\)\s+(\w+)\s+(\w+)\[([^\]]+)\];",
                 r"\1* \2 = reinterpret_cast<\1*>(::emu_lds(sizeof(\1) * (\3)));", src)
    src = re.sub(r'asm volatile\(""\s*:\s*"\+v"\((\w+)\)\);', r"(void)\1;", src)
    src = re.sub(r"__attribute__\(\(amdgpu_waves_per_eu\([^)]*\)\)\)", "", src)
    if "__shared__" in src or "asm volatile" in src or "hipLaunchKernel" in src:
        raise RuntimeError(f"{name}: a construct the emulation does not rewrite")
    for pattern, repl in PLANTS[name]:
        src, n = re.subn(pattern, repl, src, flags=re.M)
        if n != 1:
            raise RuntimeError(f"{name}: plant point found {n} times: {pattern}")
    return src


def build(out_dir: str) -> str:
    cc = emu_build.clangxx()
    if cc is None:
        raise RuntimeError("clang++ not found")
    os.makedirs(out_dir, exist_ok=True)
    for name in FILES:
        with open(os.path.join(CSRC, name)) as f:
            src = rewrite(name, f.read())
        with open(os.path.join(out_dir, name.replace(".hip", "_emu.cpp")), "w") as f:
            f.write(src)
    shutil.copy(os.path.join(CSRC, "swiglu_internal.h"), out_dir)
    for name in ("swiglu_device.hpp", "swiglu_ops_device.hpp", "emu_ops_driver.cpp", "emu_race.cpp"):
        shutil.copy(os.path.join(HERE, name), out_dir)
    exe = os.path.join(out_dir, "emu_ops_driver")
    common = [cc, "-std=c++20", "-O1", "-g", "-fsanitize=address", "-fno-omit-frame-pointer",
              "-Wno-unknown-attributes", "-Wno-ignored-attributes", "-Wno-psabi", "-I", out_dir,
              "-I", HERE]
    race_o = os.path.join(out_dir, "emu_race.o")
    subprocess.run(common + ["-c", os.path.join(out_dir, "emu_race.cpp"), "-o", race_o], check=True)
    subprocess.run(common + ["-fsanitize-coverage=func,trace-loads,trace-stores",
                             os.path.join(out_dir, "emu_ops_driver.cpp"), race_o, "-o", exe],
                   check=True)
    return exe


if __name__ == "__main__":
    import sys
    print(build(sys.argv[1] if len(sys.argv) > 1 else "/tmp/swiglu_emu_ops"))
