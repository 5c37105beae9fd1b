"""The example's block with its experts on 8-bit integers behind the scored router, run as a
user runs it: against the same block in plain operations, and replayed from a graph."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.mark.parametrize("tokens,experts,top,width,expert_width,shared_width",
                         [(1, 16, 4, 256, 144, 264), (37, 12, 3, 320, 80, 128),
                          (700, 8, 2, 512, 256, 520)])
def test_block(tokens, experts, top, width, expert_width, shared_width):
    import moe_block
    got = moe_block.main(["--tokens", str(tokens), "--experts", str(experts), "--top", str(top),
                          "--width", str(width), "--expert-width", str(expert_width),
                          "--shared-width", str(shared_width), "--int8", "--check", "--steps", "3"])
    # the two sides round the same intermediates to bf16, each off by at most half a step
    # (2^-8 of the value), a few times over.  Where the gated values differ by that, so may their
    # codes: were the two sides' code roundings independent, each of variance s^2 / 12, they would
    # differ by s / sqrt(6) with s = max / 127, and a row's maximum is at most 10 times its rms
    # (sqrt(K) at most, 9 to 16 here)
    assert got["error"] < 4 * 2.0 ** -8 + 10 / (127 * 6 ** 0.5)
    assert got["same"]
