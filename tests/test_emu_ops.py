"""CPU bounds and LDS-ordering emulation of the grouped products and the MXFP4
kernels (no GPU), as test_emu_bounds.py does for the dense kernels: every LDS
offset, DMA source and global access of every variant is checked against the
buffers, and every LDS access against the barriers and DMA waits.

A launch with few workgroups has each of them walk over many units or tiles:
the ring that is refilled behind a unit's rows of Y, and the MXFP4 ring that
runs on from one tile to the next, with 1 group of K (run as 2), 2, and an odd
number of them (the ring's halves change places between tiles)."""
import concurrent.futures as cf
import os
import subprocess
import sys

import pytest

COUNTS = ["40,1,0,300,17", "0,0", "1,1,1", "16,64,0,33", "384,129"]
GROUPED = [("grouped", up, v, n, k, 3, 5, c) for up in (1, 0) for v in range(5)
           for n, k in ((72, 72), (264, 200), (8, 0)) for c in COUNTS]
# 8 workgroups for all units; spans whose last tiles have every height
WALKS = [("--grid", 8, "grouped", up, v, 264, k, 3, 5, "300,1,0,600,140,70") for up in (1, 0)
         for v in range(1, 5) for k in (8, 136, 320)]
FP4 = [("fp4", v, m, n, k) for v in range(4) for m, n, k in ((1, 8, 32), (70, 72, 96), (300, 136, 544))]
TILES = [("--cus", 8, "fp4", v, 900, 648, k) for v in (2, 3) for k in (32, 288, 768, 1056)]
# a device of fewer CUs than the eight ranges that the tiles are dealt out in
FEW = [("--cus", c, "fp4", v, 900, 648, 288) for v in (2, 3) for c in (1, 3, 7)]
CONVERT = [("convert", rows, k) for rows, k in ((1, 32), (33, 288), (100, 896))]
WALK = ("--grid", 8, "grouped", 1)
SPANS = (264, 136, 3, 5, "300,1,0,600,140,70")
LANDS, WAVES = "while a DMA into it may land", "LDS accesses of two waves between the same barriers"
PLANTED = [(("--plant", p, *WALK, v, *SPANS), LANDS) for p in (1, 2, 3) for v in range(1, 5)] + \
    [(("--plant", 7, *WALK, 4, *SPANS), WAVES)] + \
    [(("--plant", p, "--cus", 8, "fp4", v, 900, 648, 768), LANDS) for p in (4, 5) for v in (2, 3)] + \
    [(("--plant", 6, "--cus", 8, "fp4", v, 900, 648, 768), "still in flight when its thread ends")
     for v in (2, 3)]


@pytest.fixture(scope="module")
def runs(tmp_path_factory):
    sys.path.insert(0, os.path.join(os.path.dirname(__file__), "emu"))
    import build as emu_build
    import build_ops
    if emu_build.clangxx() is None:
        pytest.skip("no host clang++")
    exe = build_ops.build(str(tmp_path_factory.mktemp("emu_ops")))
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0")

    def run(args):
        r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=300, env=env)
        return r.returncode, r.stdout + r.stderr
    with cf.ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as ex:
        jobs = GROUPED + WALKS + FP4 + TILES + FEW + CONVERT + [p for p, _ in PLANTED]
        yield dict(zip(jobs, ex.map(run, jobs)))


def clean(runs, jobs):
    for job in jobs:
        rc, out = runs[job]
        assert rc == 0 and "errors: 0" in out, f"{job}: {out[-3000:]}"


def test_grouped_launches(runs):
    clean(runs, GROUPED)


def test_grouped_workgroups_walk_over_units(runs):
    clean(runs, WALKS)


def test_mxfp4_products(runs):
    clean(runs, FP4)


def test_mxfp4_workgroups_walk_over_tiles(runs):
    clean(runs, TILES)


def test_mxfp4_on_few_compute_units(runs):
    clean(runs, FEW)


def test_mxfp4_conversions(runs):
    clean(runs, CONVERT)


@pytest.mark.parametrize("job,message", PLANTED, ids=lambda x: " ".join(map(str, x)) if isinstance(x, tuple) else "")
def test_planted_mistakes_are_found(runs, job, message):
    """build_ops.py plants them in the emulation's copy of the source."""
    rc, out = runs[job]
    assert rc != 0 and message in out, out[-3000:]
