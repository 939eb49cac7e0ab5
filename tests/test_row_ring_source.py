"""What no run can show of the row operators' kernels: the hardware's order hides
a missing barrier, a lane that leaves alone needs another warp's wait to expire at
that moment, and a promise to the compiler that does not hold need not be used.
The sources are read instead."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "blockwise_fp8_linear_fp8bq_b200", "csrc")
SOURCE = os.path.join(CSRC, "row_ring.cuh")


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


def test_early_kernels_promise_no_constant_memory():
    """A kernel that may start before the one that writes its inputs has ended."""
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for kernel in re.finditer(r"__global__[^;{]*\{", text):
            body = text[kernel.end():text.find("\n}\n", kernel.end())]
            if "cudaGridDependencySynchronize" in body:
                assert "__restrict__" not in kernel.group(0) and "__ldg" not in body, kernel.group(0)
