"""The tensor memory that one softmax group of the tree attention reads and the other has waited for: a thread's
synchronisation with another orders tensor memory only between the two fences around it."""
import os
import re

from paged_kv_cache_minmax_gb300 import build

SOURCE = open(os.path.join(build.CSRC, "tree_attn.cu")).read()


def body(name):
    at = SOURCE.index(name + "(")
    at = SOURCE.index("{", SOURCE.index(")", at))
    depth = 0
    for i in range(at, len(SOURCE)):
        depth += {"{": 1, "}": -1}.get(SOURCE[i], 0)
        if depth == 0:
            return re.sub(r"//[^\n]*", "", SOURCE[at:i])


def test_the_groups_meet_between_fences():
    text = body("groups_meet")
    order = [text.index(x) for x in ("tc_fence_before()", "__syncwarp()", "mbar_arrive(", "wait_for(", "tc_fence_after()")]
    assert order == sorted(order)
