"""Source check of the kernel of many tokens with 4-bit weights: every wait on a
barrier has a limit, and a block that gives up still lets its copies and its
products end and frees its tensor memory."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_mixed_precision_gb300", "csrc")


def test_waits_are_bounded():
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "w4_wide.cu")).read())
    body = src[src.index("w4_wide_kernel(const __grid_constant__"):src.index("cudaError_t launch_wide(")]
    # one place asks the bounded wait; every role goes through it and looks at its answer
    assert body.count("pipe::wait_bar(") == 1 and "mbar_wait" not in body and "mbar_try_wait" not in body
    uses = [m.start() for m in re.finditer(r"\bwait\(&ctl", body)]
    assert len(uses) == 6
    assert all(body[i - 1] == "!" for i in uses)
    # copies in flight, then the products in flight, are waited for; the memory is freed by all paths
    assert body.count("pipe::drain_wait(&ctl->b_full[s]") == 1 and body.count("pipe::drain_wait(&ctl->mma_done") == 1
    end = body[body.rindex("__syncthreads();"):]
    assert "ptx::tmem_dealloc(tmem, kTmemCols)" in end
    assert "return;" not in body
