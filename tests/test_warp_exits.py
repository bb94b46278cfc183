"""The few-row kernel's tile loop holds full-mask warp operations, so its warps have
to leave it whole: a lane that left alone (its wait for a free stage ran out) would
meet its neighbours at different barriers, and the kernel would not wind down."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_io_aware_96_b200", "csrc")


def test_tile_loop_is_left_by_vote_only():
    with open(os.path.join(CSRC, "fa_diff_rows.cuh")) as f:
        src = f.read()
    start = src.index("for (int i = 0; i < mine; ++i) {")
    depth, end = 0, start
    for end in range(src.index("{", start), len(src)):
        depth += (src[end] == "{") - (src[end] == "}")
        if depth == 0:
            break
    loop = src[start:end]
    assert "__shfl_xor_sync(0xffffffffu" in loop and "mbar_arrive(&empty[st])" in loop  # the loop that is meant
    exits = [line.strip() for line in loop.splitlines() if re.search(r"\b(break|return|continue|goto)\b", line.split("//")[0])]
    assert exits and all("__all_sync(0xffffffffu" in line for line in exits), exits
