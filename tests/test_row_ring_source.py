"""What no run can show of the row ring's fetch: the hardware's order hides a
missing barrier, and a lane that leaves alone needs another warp's wait to expire
at that moment.  The source is read instead."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "blockwise_fp8_linear_fp8bq_b200",
                      "csrc", "row_ring.cuh")


def fetch_body():
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    return text[text.index("void fetch()"):text.index("void wait()")]


def test_values_copied_by_lanes_are_ordered_before_the_arrival():
    body = fetch_body()
    copied = body.rindex("dst[k] = src[k]")
    arrive = body.index("mbar_arrive_expect_tx", copied)
    assert "__syncwarp()" in body[copied:arrive]


def test_a_warp_leaves_together():
    body = fetch_body()
    reads = [m.start() for m in re.finditer("abort_flag", body)]
    assert len(reads) == 1
    assert re.search(r"__shfl_sync\([^;]*abort_flag[^;]*, 0\) != 0\) return;", body)
