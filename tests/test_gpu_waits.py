"""Bounded waits of whole warps: one answer for all lanes."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TIMEOUT = 5


def test_lanes_that_wait_together_get_one_answer():
    """Even lanes give up, the barrier then completes within the odd lanes' time."""
    import fp8_mixed_precision_gb300 as fp
    assert fp.fp8_get_device_status() == 0
    answers = fp.fp8_debug_wait_together(5_000_000)  # 5, 20 and 80 ms
    assert fp.fp8_get_device_status() == TIMEOUT
    assert answers.tolist() == [0] * 32
    assert fp.fp8_get_device_status() == 0
    # and the library goes on: a product that waits together
    w = fp.fp8_w4_quantize(torch.randn((4096, 2048), device="cuda").bfloat16())
    x = torch.randn((40, 2048), device="cuda").bfloat16()
    assert torch.equal(fp.fp8_w4_linear(x, w), fp.fp8_w4_linear(x, w)) and fp.fp8_get_device_status() == 0


def test_refusals():
    import fp8_mixed_precision_gb300 as fp
    for limit in (0, 50_000_001):
        with pytest.raises(fp.FP8Error):
            fp.fp8_debug_wait_together(limit)
