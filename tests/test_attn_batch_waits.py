"""Which waits the roles of the batch attention kernel use.

A role that a whole warp runs, with collective instructions (votes, shuffles, tensor
memory) between its waits, may only use the wait that gives all lanes one answer: lanes
that gave up one by one would stand in the CTA's last barrier while the others wait
for them in the next collective instruction.
"""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4_gemm_keyed_gb300", "csrc")
LANE = re.compile(r"\b(lane_wait|wait_or_abort|mbar_wait_or_abort|mbar_wait|mbar_try_wait)\s*\(")


def body_of(source, name):
    """The definition of function `name`, by its braces."""
    at = re.search(r"__device__ void %s\([^;{]*\{" % name, source)
    depth, i = 1, at.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(source[i], 0)
        i += 1
    return source[at.start():i]


def test_roles_of_whole_warps_wait_as_warps():
    source = open(os.path.join(CSRC, "attn_batch.cu")).read()
    for role in ("softmax", "expand_tiles"):
        body = body_of(source, role)
        assert len(re.findall(r"\bwarp_wait\s*\(", body)) >= 3
        assert not LANE.search(body), role


def test_a_warp_that_gives_up_on_a_tile_gives_up_the_role():
    """multiply: the wait for a tile to mend is the warp's, and its failure ends the item loop."""
    body = body_of(open(os.path.join(CSRC, "attn_batch.cu")).read(), "multiply")
    after = body[body.index("for (int i = whole; i < tiles; ++i) {"):]
    assert re.match(r".*?if \(!warp_wait\(.*?\)\) \{\s*ok = false;\s*break;", after, re.S)
    assert "if (__any_sync(0xFFFFFFFFu, !ok)) break;" in after
