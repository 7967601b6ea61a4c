"""Orders in the operators' kernel sources that no run on a GPU can show to be wrong
without hanging or faulting it (no GPU needed)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_moe_decode_gemv_gb300", "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", lambda m: m.group(0) if "-----" in m.group(0) else "", text)


@pytest.mark.parametrize("role", ["token rows", "MMAs", "decode", "epilogue"])
def test_bounded_waits_begin_after_the_kernel_before(role):
    """A chained kernel may start while the one before it still runs: a wait that gives
    up after some seconds must not begin before that one has ended."""
    text = source("moe_qgemm.cuh")
    part = text[text.index(f"// ---------------- {role} ----------------"):]
    assert "griddepcontrol.wait" in part and part.index("griddepcontrol.wait") < part.index("wait(smem_u32")


@pytest.mark.parametrize("name", ["moe_gated.cu", "moe_gemm16.cuh", "moe_outer.cuh", "moe_qgemm.cuh", "moe_stream.cuh",
                                  "moe_stream16.cuh"])
def test_chained_kernels_promise_no_constant_inputs(name):
    """A chained kernel's inputs may be written while it already runs, until its wait:
    none is declared const __restrict__, which allows reads ahead of the wait."""
    for kernel in re.split(r"__global__", source(name))[1:]:
        head, body = kernel.split("{", 1)
        if "griddepcontrol.wait" in body.split("__global__")[0]:
            assert "__restrict__" not in head, head
