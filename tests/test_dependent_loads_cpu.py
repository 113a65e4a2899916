"""What a kernel reads when it is launched as a programmatic dependent; no GPU is used.

Such a kernel is resident while the kernel before it writes, so a call's
arguments must not go through the read-only path: PTX defines ld.global.nc
(and __ldg, which compiles to it) for memory that nothing writes during the
kernel's life only, and the compiler may move such a load over the wait for
the kernel before.  A stale value would be a matter of timing, so the sources
are looked at instead.
"""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "ternary_weight_a8_b200", "csrc")
READ_ONLY = re.compile(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc\b")


def _code(name):
    with open(os.path.join(CSRC, name)) as fh:
        return re.sub(r"//[^\n]*", "", fh.read())


@pytest.mark.parametrize("name", ["common.cuh", "i8_gemv.cu", "i8_gemm.cu"])
def test_arguments_are_not_read_through_the_read_only_path(name):
    found = [m.group(0) for m in READ_ONLY.finditer(_code(name))]
    assert not found, "%s: %s" % (name, found)


def test_the_pattern_sees_both_spellings():
    assert READ_ONLY.search("x = __ldg(p);") and READ_ONLY.search('asm("ld.global.nc.v4.u32 ...");')
    assert not READ_ONLY.search("__ldcg(p)") and not READ_ONLY.search('"ld.global.L1::no_allocate.v4.u32"')
