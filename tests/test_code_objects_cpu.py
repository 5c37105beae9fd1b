"""Resources of the kernels of every source file, read from the built library
(no GPU).  Each HIP source becomes a code object of its own, and the library's
.hip_fatbin section holds their bundles one after another; unbundling the
section as a whole gives the first one only, so it is cut at each bundle's
magic here.  No kernel uses scratch memory (a spill's loads are not in the
counts that the DMA rings wait for), and none asks for more LDS than a CU has."""
import re
import subprocess

import pytest

import gemm_epilogues_mlp_amd as sw
from gemm_epilogues_mlp_amd import _build
from test_kernel_resources_cpu import LDS_PER_CU, _tool

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def metadata(notes):
    """One mapping per kernel of a code object's notes: its top-level keys."""
    out, cur = [], None
    for line in notes.splitlines():
        if re.match(r"^  - \.", line):
            cur = {}
            out.append(cur)
        m = re.match(r"^  [ -] \.(\w+):\s+(.*)$", line)
        if m and cur is not None:
            cur[m.group(1)] = m.group(2).strip()
    return [k for k in out if "name" in k]


@pytest.fixture(scope="module")
def objects(tmp_path_factory):
    """The kernels of each bundle of the library, in its order."""
    objcopy, bundler, readelf = _tool("llvm-objcopy"), _tool("clang-offload-bundler"), \
        _tool("llvm-readelf")
    if not (objcopy and bundler and readelf):
        pytest.skip("ROCm LLVM tools not found")
    d = tmp_path_factory.mktemp("bundles")
    fat = d / "fat.bin"
    subprocess.run([objcopy, "--dump-section", f".hip_fatbin={fat}", sw.lib_path(),
                    str(d / "copy.so")], check=True)
    data = fat.read_bytes()
    at = [m.start() for m in re.finditer(re.escape(MAGIC), data)]
    out = []
    for i, (a, b) in enumerate(zip(at, at[1:] + [len(data)])):
        part, dev = d / f"bundle{i}", d / f"gfx950_{i}.o"
        part.write_bytes(data[a:b])
        subprocess.run([bundler, "--unbundle", "--type=o", f"--input={part}",
                        "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", f"--output={dev}"], check=True)
        notes = subprocess.run([readelf, "--notes", str(dev)], check=True, capture_output=True,
                               text=True).stdout
        out.append(metadata(notes))
    return out


def test_every_source_has_a_bundle(objects):
    """One with kernels for each .hip source: nothing of the library goes unread."""
    hip = [s for s in _build.SOURCES if s.endswith(".hip")]
    assert len([o for o in objects if o]) == len(hip), [len(o) for o in objects]


def test_every_operator_is_listed(objects):
    names = [k["name"] for o in objects for k in o]
    assert len(names) == len(set(names))
    for part in ("tiled_kernel", "packed_kernel", "route_small_kernel", "route_select_kernel",
                 "route_place_kernel", "grouped_stream_kernel", "grouped_tile_kernel",
                 "combine_norm_kernel", "fp4_tile_kernel", "fp4_stream_kernel",
                 "quantize_fp4_kernel", "dequantize_fp4_kernel"):
        assert any(part in n for n in names), part


def test_no_kernel_uses_scratch(objects):
    bad = [(k["name"], k.get("private_segment_fixed_size"), k.get("vgpr_spill_count"))
           for o in objects for k in o
           if k.get("private_segment_fixed_size") != "0" or k.get("vgpr_spill_count") != "0"
           or k.get("uses_dynamic_stack") != "false"]
    assert not bad, bad


def test_lds_fits_a_cu(objects):
    for o in objects:
        for k in o:
            assert int(k["group_segment_fixed_size"]) <= LDS_PER_CU, k["name"]


def test_a_spill_is_seen():
    """The notes' form as the reader takes it, with a kernel that spills behind one that does not."""
    notes = "\n".join(["amdhsa.kernels:", "  - .args:", "      - .offset: 0", "    .name: clean",
                       "    .private_segment_fixed_size: 0", "    .vgpr_spill_count: 0",
                       "  - .args:", "    .name: spills", "    .private_segment_fixed_size: 16",
                       "    .vgpr_spill_count: 3", "amdhsa.target: gfx950"])
    got = metadata(notes)
    assert [k["name"] for k in got] == ["clean", "spills"]
    assert got[1]["vgpr_spill_count"] == "3" and got[0]["private_segment_fixed_size"] == "0"
