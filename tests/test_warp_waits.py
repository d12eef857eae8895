"""Source check of the kernels whose warps load from and store to TMEM, which are
instructions of all 32 lanes: the answer of a wait that all lanes make never parts
them.  A lane that gave up goes on with its warp, which leaves as one."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_mixed_precision_gb300", "csrc")

# file, kernel, where the roles that wait with all lanes begin
ROLES = [("gemm.cu", "fp8_gemm_kernel", "const int ew = warp - C::kCtlWarps;"),
         ("gated.cu", "gated_fwd_kernel", "const int ew = warp - 2, q = warp & 3"),
         ("gated.cu", "gated_small_kernel", "const int q = warp & 3, f = q * 32 + lane"),
         ("w4_wide.cu", "w4_wide_kernel", "} else if (warp < 6) {")]


def _roles(name, kernel, begin):
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for m in re.finditer(r"\b%s\(" % kernel, src):
        i, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(src[i], 0)
            i += 1
        if src[i:].lstrip().startswith("{"):
            j, depth = src.index("{", i) + 1, 1
            while depth:
                depth += {"{": 1, "}": -1}.get(src[j], 0)
                j += 1
            body = src[i:j]
            assert body.count(begin) == 1
            return body[body.index(begin):]
    raise AssertionError(f"{kernel} not found")


@pytest.mark.parametrize("name,kernel,begin", ROLES)
def test_a_wait_that_gives_up_does_not_part_a_warp(name, kernel, begin):
    text = _roles(name, kernel, begin)
    waits = list(re.finditer(r"\bwait(?:_bar(?:<PR>)?)?\(&ctl->", text))
    assert waits
    for m in waits:
        start = max(text.rfind(c, 0, m.start()) for c in ";{}") + 1
        statement = text[start:text.index(";", m.end())].strip()
        vote = re.match(r"if \(__any_sync\(0xffffffffu, !wait\w*(<PR>)?\(.*\)\)\)", statement)
        assert vote or re.match(r"(lost \|= !)?wait", statement), statement
    for m in re.finditer(r"if \(([^;{]*(?:\blost\b|\*abort)[^;{]*)\)\s*(?:\{[^}]*break;|break;)", text):
        assert re.fullmatch(r"__any_sync\(0xffffffffu, (lost|\*abort)\)", m[1]), m[0]
