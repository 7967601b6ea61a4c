"""The build compiles a unit twice only where the debug build differs (no GPU needed)."""
import os
import re

from quantized_moe_decode_gemv_gb300 import build as B


def _reads_the_macro(path, seen):
    if path in seen or not os.path.exists(path):
        return False
    seen.add(path)
    text = open(path).read()
    if re.search(r"\bMOE_CHECKS\b", text):
        return True
    return any(_reads_the_macro(os.path.join(d, n), seen) for n in re.findall(r'#include "([^"]+)"', text)
               for d in (B.CSRC, B.INCLUDE))


def test_units_without_a_check_are_compiled_once():
    names = {name: src for src, name, _ in B.SOURCES}
    assert B.NO_CHECKS <= set(names)
    for name, src in names.items():
        # a header that only documents the macro counts for no unit by itself
        uses = _reads_the_macro(os.path.join(B.CSRC, src), {os.path.join(B.INCLUDE, "moe_layer.h")})
        assert uses == (name not in B.NO_CHECKS), name
