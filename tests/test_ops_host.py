"""Refusals of the operator handles on the host, and the bit encodings of the
fp4 re-layout (no GPU needed)."""
import ctypes
import os

import pytest

import quantized_moe_decode_gemv_gb300 as pkg
from quantized_moe_decode_gemv_gb300 import _capi

FAKE = 0x1000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_capi.LIB_PATH):
        pytest.fail("libmoe_gb300.so is not built; run __graft_entry__.build()")
    return _capi.load_library()


def _linear(lib, w=None, **kw):
    base = dict(in_features=256, out_features=96, group_size=64)
    base.update(kw)
    raw = base.pop("raw", {})
    c = pkg.QLinearConfig(**base).to_c()
    for n, v in raw.items():
        setattr(c, n, v)
    if w is not None:
        w = ctypes.byref(_capi.moe_qlinear_weights(**w))
    return _capi.STATUS_NAMES[lib.moe_qlinear_validate(ctypes.byref(c), w)]


W = {"q": FAKE, "s": FAKE, "b": FAKE}
G = {"gate_q": FAKE, "gate_s": FAKE, "gate_b": FAKE}


@pytest.mark.parametrize("kw,w,want", [
    ({}, W, "MOE_OK"), ({}, None, "MOE_OK"),
    ({"out_features": 1}, W, "MOE_OK"),
    ({"in_features": 0}, W, "MOE_ERR_INVALID_ARG"), ({"out_features": -4}, W, "MOE_ERR_INVALID_ARG"),
    ({"max_tokens": 0}, W, "MOE_ERR_INVALID_ARG"),
    ({"group_size": 48}, W, "MOE_ERR_SHAPE"), ({"group_size": 16}, W, "MOE_ERR_SHAPE"),
    ({"in_features": 288}, W, "MOE_ERR_SHAPE"), ({"in_features": 288, "group_size": 32}, W, "MOE_OK"),
    ({"fmt": "nvfp4"}, W, "MOE_ERR_SHAPE"), ({"fmt": "nvfp4", "group_size": 16, "in_features": 48}, W, "MOE_OK"),
    ({"fmt": "mxfp4", "group_size": 32}, {"q": FAKE, "s": FAKE}, "MOE_OK"),
    ({"fmt": "nvfp4", "group_size": 16}, {"q": FAKE, "s": FAKE}, "MOE_ERR_INVALID_ARG"),
    ({}, {"q": FAKE, "s": FAKE}, "MOE_ERR_INVALID_ARG"), ({}, {"s": FAKE, "b": FAKE}, "MOE_ERR_INVALID_ARG"),
    ({"act": "swiglu"}, W, "MOE_ERR_INVALID_ARG"), ({"act": "swiglu"}, {**W, **G}, "MOE_OK"),
    ({"act": "relu2"}, {**W, **G}, "MOE_ERR_SHAPE"), ({}, {**W, **G}, "MOE_ERR_SHAPE"),
    ({"bias": True}, {**W, "bias": FAKE}, "MOE_OK"), ({"bias": True}, W, "MOE_ERR_INVALID_ARG"),
    ({}, {**W, "bias": FAKE}, "MOE_ERR_SHAPE"), ({"bias": True, "act": "relu2"}, W, "MOE_ERR_UNSUPPORTED"),
    ({"act_dtype": "fp32"}, W, "MOE_ERR_UNSUPPORTED"), ({"scale_dtype": "fp32"}, W, "MOE_ERR_UNSUPPORTED"),
    ({"scale_dtype": "fp32", "fmt": "nvfp4", "group_size": 16}, W, "MOE_OK"),
    ({"in_features": 65536 + 64}, W, "MOE_ERR_UNSUPPORTED"), ({"out_features": (1 << 24) + 1}, W, "MOE_ERR_UNSUPPORTED"),
    ({"raw": {"act": 3}}, W, "MOE_ERR_INVALID_ARG"), ({"raw": {"weight_format": 9}}, W, "MOE_ERR_INVALID_ARG"),
    ({"raw": {"act_dtype": -1}}, W, "MOE_ERR_INVALID_ARG"),
])
def test_linear_refusals(lib, kw, w, want):
    assert _linear(lib, w, **kw) == want, lib.moe_qlinear_last_error(None)


@pytest.mark.parametrize("kw,want", [
    ({}, "MOE_OK"), ({"in_features": 8, "out_features": 8}, "MOE_OK"), ({"in_features": 100}, "MOE_ERR_SHAPE"),
    ({"out_features": 12}, "MOE_ERR_SHAPE"), ({"out_features": 0}, "MOE_ERR_INVALID_ARG"),
    ({"max_tokens": 0}, "MOE_ERR_INVALID_ARG"), ({"act_dtype": "fp32"}, "MOE_ERR_UNSUPPORTED"),
    ({"in_features": 65544}, "MOE_ERR_UNSUPPORTED"),
])
def test_gated_refusals(lib, kw, want):
    base = dict(in_features=256, out_features=96)
    base.update(kw)
    c = pkg.GatedConfig(**base).to_c()
    assert _capi.STATUS_NAMES[lib.moe_gated_validate(ctypes.byref(c))] == want


def test_null_arguments(lib):
    assert lib.moe_qlinear_validate(None, None) == 1 and lib.moe_gated_validate(None) == 1
    h = ctypes.c_void_p(5)
    c = pkg.QLinearConfig(in_features=256, out_features=96).to_c()
    assert lib.moe_qlinear_create(ctypes.byref(c), None, None, ctypes.byref(h)) == 1 and not h.value
    assert lib.moe_qlinear_create(ctypes.byref(c), None, None, None) == 1
    g = pkg.GatedConfig(in_features=256, out_features=96).to_c()
    assert lib.moe_gated_create(ctypes.byref(g), None) == 1
    assert lib.moe_gated_create(None, ctypes.byref(h)) == 1 and not h.value
    assert lib.moe_qlinear_forward(None, None, 0, 0, None, 0, None) == 1
    assert lib.moe_gated_forward(None, None, 0, 0, None, None, None, 0, None, None, None) == 1
    assert lib.moe_gated_backward(None, None, 0, 0, None, 0, None, None, None, None, None, 0, None, None, None) == 1
    for p in ("moe_qlinear", "moe_gated"):
        assert getattr(lib, p + "_destroy")(None) == 0
        assert getattr(lib, p + "_device_status")(None, None) == 1
        assert getattr(lib, p + "_device_bytes")(None) == 0
        assert getattr(lib, p + "_last_launch_count")(None) == 0


def test_unknown_names_are_refused():
    with pytest.raises(pkg.MoEError):
        pkg.QLinearConfig(in_features=256, out_features=96, act="gelu").to_c()
    with pytest.raises(pkg.MoEError):
        pkg.QLinearConfig(in_features=256, out_features=96, fmt="int4").to_c()
    with pytest.raises(pkg.MoEError):
        pkg.GatedConfig(in_features=256, out_features=96, act="none").to_c()


# ---------------------------------------------------------------------------
# the fp4 decode's arithmetic, restated on integers
# ---------------------------------------------------------------------------

E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def _place(code, i, fp16):
    s, eem = code >> 3, code & 7
    if fp16:
        return s << (15, 12, 14, 13)[i] | eem << (9 - 3 * i)
    return s << (15, 12, 14, 13)[i] | eem << (6, 3, 0, 9)[i]


def _take(w, i, fp16):
    if fp16:
        return (w & 0x8E008E00, (w << 3) & 0x8E008E00, (w << 6) & 0x0E000E00 | (w << 1) & 0x80008000,
                (w << 9) & 0x0E000E00 | (w << 2) & 0x80008000)[i] & 0xFFFFFFFF
    return (w & 0x81C081C0, (w << 3) & 0x81C081C0, (w << 6) & 0x01C001C0 | (w << 1) & 0x80008000,
            (w >> 3) & 0x01C001C0 | (w << 2) & 0x80008000)[i] & 0xFFFFFFFF


def _value(bits, fp16):
    e, m, eb = (bits >> 10 & 31, bits & 1023, 10) if fp16 else (bits >> 7 & 255, bits & 127, 7)
    bias = 15 if fp16 else 127
    v = m * 2.0 ** (1 - bias - eb) if e == 0 else (1 + m / 2 ** eb) * 2.0 ** (e - bias)
    return -v if bits & 0x8000 else v


@pytest.mark.parametrize("fp16", [False, True])
def test_fp4_words_hold_every_code_apart(fp16):
    unit = 2.0 ** (-14 if fp16 else -126)
    used = 0
    for i in range(4):
        mask = _place(15, i, fp16)
        assert bin(mask).count("1") == 4 and not used & mask
        used |= mask
    assert used == 0xFFFF
    for i in range(4):
        for code in range(16):
            for other in (0, 15):
                half = sum(_place(code if j == i else other, j, fp16) for j in range(4))
                for lo, hi in ((half, 0xFFFF), (half, 0), (0xFFFF, half), (0, half)):
                    r = _take(lo | hi << 16, i, fp16)
                    got = _value(r & 0xFFFF if lo == half else r >> 16, fp16)
                    want = E2M1[code & 7] * (-1 if code & 8 else 1) * unit
                    assert got == want, (i, code, other)
