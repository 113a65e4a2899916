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


# pack.cu's kernels are launched as ordinary ones.
FILES = sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh")) and n != "pack.cu")
# Packed weights are, by the header's rule, not written by the kernel just before a ternary product.
PACKED = {"lut_gemv.cu": "__ldg(row + w)"}


@pytest.mark.parametrize("name", FILES)
def test_arguments_are_not_read_through_the_read_only_path(name):
    code = _code(name).replace(PACKED.get(name, "\0"), "")
    found = [m.group(0) for m in READ_ONLY.finditer(code)]
    assert not found, "%s: %s" % (name, found)


def test_the_pattern_sees_both_spellings():
    assert READ_ONLY.search("x = __ldg(p);") and READ_ONLY.search('asm("ld.global.nc.v4.u32 ...");')
    assert not READ_ONLY.search("__ldcg(p)") and not READ_ONLY.search('"ld.global.L1::no_allocate.v4.u32"')


def _kernels(code):
    """(name, body) of the file's __global__ functions that are not launched with <<<>>>."""
    launch_bounds = r"(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(?:__maxnreg__\((?:[^()]|\([^()]*\))*\)\s*)?"
    for m in re.finditer(r"__global__\s+void\s+" + launch_bounds + r"(\w+)\s*\(", code):
        start = code.index("{", m.end())
        depth, end = 0, start
        while True:
            depth += {"{": 1, "}": -1}.get(code[end], 0)
            if depth == 0:
                break
            end += 1
        if not re.search(m.group(1) + r"\s*<<<", code):
            yield m.group(1), code[start:end]


def test_every_dependent_kernel_waits_for_the_kernel_before_it():
    """One that does not may read what is still being written, and lets the kernel behind it start as early: a wait is for
    the preceding kernel only, which has to have waited itself."""
    seen = set()
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu"):
            for kernel, body in _kernels(_code(name)):
                seen.add(kernel)
                assert "griddep_wait()" in body, "%s: %s" % (name, kernel)
    assert {"layout_kernel", "gemm_bf16_kernel", "i8_gemm_kernel", "gemv_group_kernel",
            "gemm_kernel", "add_rmsnorm_backward_kernel", "act_quant_kernel"} <= seen
