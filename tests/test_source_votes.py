"""Loops in which the lanes of a warp vote: all of them have to leave in the same turn,
so whatever ends such a loop must be the same in every lane.  (Shown on the source: a
wait that runs out with lanes apart could hang a GPU.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_gqa_row_gb300", "csrc")


def test_the_4_bit_decode_producer_compares_one_lanes_clock():
    with open(os.path.join(CSRC, "decode4.cu")) as f:
        src = f.read()
    loop = src[src.index("if (warp == kProducerWarp) {\n    // ==="):src.index("// Drain: do not leave the CTA")]
    assert "__all_sync(0xffffffffu, done)" in loop  # the votes
    reads = [m.start() for m in re.finditer(r"global_timer_ns\(\)", loop)]
    assert len(reads) == 2  # where the clock starts, and where it is compared
    for at in reads:
        assert loop[:at].endswith("__shfl_sync(0xffffffffu, "), loop[at - 60:at + 20]
        assert loop[at:].startswith("global_timer_ns(), 0)")
