"""Read from the kernels' source (no GPU): cp.async.wait_group makes a copy visible only to the
thread that asked for it.  Where the lanes of a warp or the warps of a block read one another's
copies, a barrier has to stand between the wait and the reads; a vote or an mbarrier of other copies
orders nothing for them."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_moe_layer_bias_gb300", "csrc")
BARRIER = r"__syncwarp\(\)|__syncthreads\(\)"
# what reads copies of other lanes or warps (the functions' own definitions are `void run_...`)
READS = r"(?<!void )\brun_task<|(?<!void )\brun_item<"


def code_of(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"/\*.*?\*/|//[^\n]*", "", text, flags=re.S)


@pytest.mark.parametrize("name", ["w4.cu"])
def test_a_barrier_between_the_wait_for_copies_and_their_reads(name):
    text = code_of(name)
    waits = [m.end() for m in re.finditer(r"(?<!void )\bcp_wait<[^>]*>\(\);", text)]
    reads = list(re.finditer(READS, text))
    assert len(waits) >= 4 and len(reads) >= 2   # the patterns still find what they are for
    for at in waits:
        nxt = re.search(f"{BARRIER}|{READS}", text[at:])
        assert nxt is None or re.fullmatch(BARRIER, nxt.group()), text[at - 200:at + 400]
