"""What the sources of e0_sample have to keep, whatever a GPU happens to do."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_gathered_expert_gb300", "csrc")


def test_other_blocks_have_begun_before_their_memory_is_written():
    """Writing to the shared memory of a cluster's block that has not begun is undefined: k_sample says that it has begun
    first of all, and waits for the others before its first write to one."""
    src = open(os.path.join(CSRC, "e0_sample.cu")).read()
    arrive, wait = (re.search(r"void (\w+)\(\) \{ asm volatile\(\"barrier\.cluster\.%s\.\w+\.aligned;\"" % what, src)
                    for what in ("arrive", "wait"))
    assert arrive and wait
    kernel = src[src.index("k_sample(SampleArgs A)"):]
    first = min(kernel.index(x) for x in ("put(", "meet()", "return", "__syncthreads()"))
    assert kernel.index(arrive.group(1) + "();") < first
    remote = min(kernel.index(x) for x in ("of_block(", "meet()"))
    assert kernel.index(wait.group(1) + "();") < remote
    # no thread leaves between the two, and both are passed once
    between = kernel[kernel.index(arrive.group(1) + "();"):kernel.index(wait.group(1) + "();")]
    assert "return;" not in between
    assert kernel.count(arrive.group(1) + "();") == kernel.count(wait.group(1) + "();") == 1
