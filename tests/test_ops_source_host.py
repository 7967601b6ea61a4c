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
