"""The example's block (router, experts, MXFP4 shared expert, norms) run as a user runs it:
against the same block in plain operations, and replayed from a graph."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.mark.parametrize("tokens,experts,top,width,expert_width,shared_width",
                         [(1, 16, 4, 256, 136, 264), (37, 12, 3, 320, 72, 128),
                          (700, 8, 2, 512, 256, 520)])
def test_block(tokens, experts, top, width, expert_width, shared_width):
    import moe_block
    got = moe_block.main(["--tokens", str(tokens), "--experts", str(experts), "--top", str(top),
                          "--width", str(width), "--expert-width", str(expert_width),
                          "--shared-width", str(shared_width), "--check", "--steps", "3"])
    # the two sides round the same intermediates to bf16, each off by at most half a
    # step (2^-8 of the value); gate, products and norms carry a few such roundings on
    assert got["error"] < 4 * 2.0 ** -8
    assert got["same"]
