"""Source check of the norm's and the gated feed-forward's kernels: a bounded
wait that gives up ends the kernel's requests, and no CTA leaves while a copy
that it asked for may still land in its shared memory.  (A wait that runs out
needs hardware that fails; the GEMM's probe covers the wait itself.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_mixed_precision_gb300", "csrc")


def _source(name):
    s = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", s)


def _block(src, at, pair):
    """Index behind the bracket that closes the first one from `at`."""
    i = src.index(pair[0], at) + 1
    depth = 1
    while depth:
        depth += {pair[0]: 1, pair[1]: -1}.get(src[i], 0)
        i += 1
    return i


def _body(src, name):
    """The body of the function or kernel `name`, at its definition."""
    for m in re.finditer(r"\b%s\(" % name, src):
        end = _block(src, m.start(), "()")
        if src[end:].lstrip().startswith("{"):
            return src[end:_block(src, end, "{}")]
    raise AssertionError(f"{name} not found")


@pytest.mark.parametrize("name,kernel", [("norm.cu", "rmsnorm_cols_kernel"), ("gated.cu", "gated_bwd_cast_kernel")])
def test_tile_kernels_stop_and_drain(name, kernel):
    body = _body(_source(name), kernel)
    assert "wait_bar(" in body
    assert re.search(r"int \*abort = &S\.abort;", body), "a wait that gave up is known to its thread alone"
    leave = body[body.index("drain_wait("):]
    assert "return;" in leave and "prefetch(id" in leave, "more copies are asked for after a wait gave up"


def test_ring_producer_waits_for_its_last_copies():
    body = _body(_source("norm.cu"), "ring_produce")
    loop_end = body.index("++issued;")
    assert "drain_wait(" in body[loop_end:]
    assert not re.search(r"if\s*\(!ok\)", body[loop_end:]), "only a producer that gave up waits for its copies"
