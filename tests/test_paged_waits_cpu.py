"""Roles of the paged decode kernel that can give up: a producer or the MMA warp leaves its loop
when a bounded wait runs out, so nobody may wait for one of them at a barrier without a limit
(barriers among warps that never leave their loops are fine)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "compressed_sliding_window_b200", "csrc")


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_no_barrier_between_roles_that_give_up():
    code = _code("paged_decode.cuh")
    roles = code[code.index("if (warp < kProducers) {"):code.index("const int sw = warp - kProducers - 1;")]
    for wait in ("named_bar_sync", "barrier.cta", "bar.sync", "__syncthreads"):
        assert wait not in roles, wait
    # the only raw barriers left are the ones behind named_bar_sync
    assert "barrier.cta" not in code and "bar.sync" not in code
