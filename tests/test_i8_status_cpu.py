"""Host-side checks of the 8-bit product's device status; no GPU is used."""
import os
import re

import ternary_weight_a8_b200 as tb
from conftest import ROOT


def test_selftest_refusals():
    fn = tb.lib().bitlinear_selftest_i8_wait_timeout
    assert fn(None, 256, 1000, None) == tb.BL_ERR_INVALID_ARG and "workspace is NULL" in tb.last_error()
    assert fn(8, 256, 1000, None) == tb.BL_ERR_MISALIGNED


def test_every_recorded_timeout_reaches_the_devices_word():
    """In the product's source a timeout is recorded at one place, in the call's workspace and in the device's word."""
    with open(os.path.join(ROOT, "ternary_weight_a8_b200", "csrc", "i8_gemm.cu")) as fh:
        code = re.sub(r"//[^\n]*", "", fh.read())
    assert code.count("kStatusTimeout") == 2
    assert re.search(r"atomicOr\(ctl\.status, kStatusTimeout\);\s*atomicOr\(&g_status, kStatusTimeout\);", code)
