"""CPU bounds and LDS-ordering emulation of the 8-bit integer kernels (no GPU), as
test_emu_ops.py does for the other operators: every LDS offset, DMA source and global access of
every variant is checked against the buffers, every LDS access against the barriers and DMA waits,
and every output element that has to be written is, and no other."""
import concurrent.futures as cf
import os
import subprocess
import sys

import pytest

COUNTS = ["40,1,0,300,17", "0,0", "1,1,1", "16,64,0,33", "384,129"]
DENSE = [("dense", gated, v, m, n, k) for gated in (1, 0) for v in range(8)
         for m, n, k in ((1, 8, 16), (70, 72, 80), (300, 136, 544), (33, 264, 0))]
GROUPED = [("grouped", gated, v, n, k, 3, 5, c) for gated in (1, 0) for v in range(8)
           for n, k in ((72, 80), (264, 208), (8, 0)) for c in COUNTS]
# 8 workgroups for all tiles: the ring runs on from one to the next, with 1 to 9 groups of K (run
# as 2 or 4 at least), an odd number of them too (the ring's halves change places), and
# spans whose last tiles have every height
WALKS = [("--cus", 8, "dense", gated, v, 900, 648, k) for gated in (1, 0) for v in (4, 5, 6, 7)
         for k in (16, 272, 1040)] + \
    [("--cus", 8, "grouped", gated, v, 264, k, 3, 5, "300,1,0,600,140,70") for gated in (1, 0)
     for v in (4, 5, 6, 7) for k in (16, 528, 656, 1040)]
# a device of fewer CUs than the eight ranges that the tiles are dealt out in
FEW = [("--cus", c, *job) for c in (1, 3) for job in (("dense", 1, 7, 900, 648, 272),
                                                      ("grouped", 0, 5, 264, 144, 3, 5, "300,1,0,600"))]
# more than 64 experts: the spans' table is searched in parts
MANY = [("--cus", 8, "grouped", gated, v, 40, 144, 2, 3, ",".join(["2"] * 70 + ["0"] * 70 + ["70"] * 9))
        for gated in (1, 0) for v in range(8)]
OTHER = [("quantize", rows, k) for rows, k in ((5, 16), (6, 1024), (3, 1040), (2, 9008), (2, 20000), (2, 40000))] + \
    [("pack", *a) for a in ((1, 1, 16), (3, 40, 144), (2, 64, 256))]
LANDS, FLIGHT = "while a DMA into it may land", "still in flight when its thread ends"
WALK = ("--cus", 8, "grouped")
SPANS = (264, 656, 3, 5, "300,1,0,600,140,70")
PLANTED = [(("--plant", p, *WALK, 1, v, *SPANS), LANDS) for p in (1, 3, 4) for v in (4, 5, 6, 7)] + \
    [(("--plant", 1, "--cus", 8, "dense", 0, v, 900, 648, 528), LANDS) for v in (4, 5, 6, 7)] + \
    [(("--plant", 2, *WALK, 0, v, *SPANS), FLIGHT) for v in (4, 5, 6, 7)]


@pytest.fixture(scope="module")
def runs(tmp_path_factory):
    sys.path.insert(0, os.path.join(os.path.dirname(__file__), "emu"))
    import build as emu_build
    import build_int8
    if emu_build.clangxx() is None:
        pytest.skip("no host clang++")
    exe = build_int8.build(str(tmp_path_factory.mktemp("emu_int8")))
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0")

    def run(args):
        r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=300, env=env)
        return r.returncode, r.stdout + r.stderr
    with cf.ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as ex:
        jobs = DENSE + GROUPED + WALKS + FEW + MANY + OTHER + [p for p, _ in PLANTED]
        yield dict(zip(jobs, ex.map(run, jobs)))


def clean(runs, jobs):
    for job in jobs:
        rc, out = runs[job]
        assert rc == 0 and "errors: 0" in out, f"{job}: {out[-3000:]}"


def test_dense_launches(runs):
    clean(runs, DENSE)


def test_grouped_launches(runs):
    clean(runs, GROUPED)


def test_workgroups_walk_over_tiles(runs):
    clean(runs, WALKS)


def test_few_compute_units(runs):
    clean(runs, FEW)


def test_many_experts(runs):
    clean(runs, MANY)


def test_quantisation_and_packing(runs):
    clean(runs, OTHER)


@pytest.mark.parametrize("job,message", PLANTED, ids=lambda x: " ".join(map(str, x)) if isinstance(x, tuple) else "")
def test_planted_mistakes_are_found(runs, job, message):
    """build_int8.py plants them in the emulation's copy of the source."""
    rc, out = runs[job]
    assert rc != 0 and message in out, out[-3000:]
