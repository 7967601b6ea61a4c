"""Refusals of the orthogonalised update on the host, and its plain forms (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

import quantized_moe_decode_gemv_gb300 as pkg
from quantized_moe_decode_gemv_gb300 import _capi, _train_ops
from tests import ortho_reference as orf
from tests.test_ops_streams_host import STREAM, Tensor, handle


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_capi.LIB_PATH):
        pytest.fail("libmoe_gb300.so is not built; run __graft_entry__.build()")
    return _capi.load_library()


NAN = float("nan")


@pytest.mark.parametrize("kw,want", [
    ({}, "MOE_OK"), ({"rows": 1, "cols": 1}, "MOE_OK"), ({"rows": 32768, "cols": 32768}, "MOE_OK"),
    ({"rows": 0}, "MOE_ERR_INVALID_ARG"), ({"cols": -1}, "MOE_ERR_INVALID_ARG"), ({"steps": 0}, "MOE_ERR_INVALID_ARG"),
    ({"max_matrices": 0}, "MOE_ERR_INVALID_ARG"), ({"eps": -1e-9}, "MOE_ERR_INVALID_ARG"), ({"eps": NAN}, "MOE_ERR_INVALID_ARG"),
    ({"coefficients": (NAN, 0, 0)}, "MOE_ERR_INVALID_ARG"), ({"coefficients": (1, float("inf"), 0)}, "MOE_ERR_INVALID_ARG"),
    ({"rows": 32769}, "MOE_ERR_UNSUPPORTED"), ({"steps": 65}, "MOE_ERR_UNSUPPORTED"), ({"steps": 64}, "MOE_OK"),
    ({"max_matrices": 1 << 23}, "MOE_OK"), ({"max_matrices": (1 << 24) + 1}, "MOE_ERR_UNSUPPORTED"),
    ({"coefficients": (1.5, -0.5, 0.0), "steps": 30}, "MOE_OK"), ({"coefficients": (15 / 8, -10 / 8, 3 / 8), "steps": 30}, "MOE_OK"),
    ({"coefficients": (3.4445, 4.775, 2.0315)}, "MOE_ERR_UNSUPPORTED"), ({"coefficients": (2.0, 0.0, 0.0)}, "MOE_ERR_UNSUPPORTED"),
    ({"coefficients": (1e30, -1e30, 0.0)}, "MOE_ERR_UNSUPPORTED"), ({"coefficients": (0.0, 0.0, 0.0)}, "MOE_OK"),
    ({"eps": 0.0}, "MOE_OK"), ({"dtype": "fp32"}, "MOE_OK"), ({"dtype": "fp16"}, "MOE_OK"),
])
def test_config_refusals(lib, kw, want):
    c = pkg.OrthoConfig(**{**dict(rows=64, cols=96), **kw}).to_c()
    assert _capi.STATUS_NAMES[lib.moe_ortho_validate(ctypes.byref(c))] == want, lib.moe_ortho_last_error(None)


def test_names_and_sizes():
    for kw in ({"dtype": "fp8"}, {"coefficients": (1.0, 2.0)}, {"rows": 2 ** 31}, {"cols": 2 ** 32 + 8}, {"steps": 2 ** 32 + 5},
               {"max_matrices": 2 ** 32 + 1}):
        with pytest.raises(pkg.MoEError) as err:
            pkg.OrthoConfig(**{**dict(rows=64, cols=96), **kw}).to_c()
        assert err.value.status == 1


def test_null_arguments(lib):
    assert lib.moe_ortho_validate(None) == 1
    h = ctypes.c_void_p(5)
    c = pkg.OrthoConfig(rows=64, cols=96).to_c()
    assert lib.moe_ortho_create(ctypes.byref(c), None) == 1
    assert lib.moe_ortho_create(None, ctypes.byref(h)) == 1 and not h.value
    assert lib.moe_ortho_forward(None, None, 0, 0, 0, None, 0, 0, None) == 1
    assert lib.moe_ortho_destroy(None) == 0 and lib.moe_ortho_device_status(None, None) == 1
    assert lib.moe_ortho_device_bytes(None) == 0 and lib.moe_ortho_last_launch_count(None) == 0


@pytest.mark.parametrize("stream,used", [(STREAM, [STREAM]), (None, [])])
def test_what_a_given_stream_uses_is_marked(stream, used):
    h = handle(_train_ops.Orthogonalizer, _R=64, _C=96, _bf16=torch.bfloat16, _call=lambda *a: 0, config=pkg.OrthoConfig(64, 96))
    g, out = Tensor(64, 96), Tensor(64, 96)
    h.forward(g, stream=stream)
    assert g.used == used
    h.forward(g, out=out, stream=stream)
    assert g.used == 2 * used and out.used == used


def test_exact_on_a_diagonal_matrix():
    """Singular values by hand: each follows the polynomial alone."""
    s = torch.tensor([3.0, 2.0, 0.5, 0.01], dtype=torch.float64)
    g = torch.zeros(4, 6, dtype=torch.float64)
    g[range(4), [2, 0, 5, 1]] = s
    for m in (g, g.T):
        want = s / (s.norm() + 1e-7)
        for _ in range(5):
            want = 3.4445 * want - 4.775 * want ** 3 + 2.0315 * want ** 5
        got = orf.exact(m)
        got = got if m is g else got.T
        assert torch.allclose(got[range(4), [2, 0, 5, 1]], want, rtol=1e-12, atol=1e-12)
        assert abs(got.norm() - want.norm()) < 1e-12


@pytest.mark.parametrize("kind", ["tokens", "few", "normal"])
@pytest.mark.parametrize("rows,cols", [(16, 16), (40, 25), (96, 400), (300, 300)])
def test_the_precision_held_is_enough(kind, rows, cols):
    """fp16 where the kernels hold it: below the rounding of the output."""
    for dtype in ("bf16", "fp32"):
        g = orf.gradient(rows, cols, dtype, 2, kind, device="cpu")
        assert orf.distance(orf.held(g), orf.exact(g)) <= orf.HELD


def test_chained_kernels_promise_no_constant_inputs():
    path = os.path.join(os.path.dirname(_capi.__file__), "csrc", "moe_ortho.cuh")
    text = re.sub(r"//[^\n]*", lambda m: m.group(0) if "-----" in m.group(0) else "", open(path).read())
    kernels = {re.search(r"\bk_\w+", k).group(0): k.split("{", 1) for k in re.split(r"__global__", text)[1:]}
    assert set(kernels) == {"k_ortho", "k_ortho_norm", "k_ortho_start"}
    for name, (head, body) in kernels.items():
        # (k_ortho is launched after its inputs' kernel has ended, and its CTAs write what others read)
        assert ("griddepcontrol.wait" in body) == (name != "k_ortho") and "__restrict__" not in head


def test_waits_for_other_tiles_come_before_what_they_guard():
    """Copies and epilogues of a tile begin after the products that it reads are done."""
    path = os.path.join(os.path.dirname(_capi.__file__), "csrc", "moe_ortho.cuh")
    text = open(path).read()
    text = text[text.index("k_ortho(const"):]
    copies = text[text.index("tensor copies ----"):text.index("MMAs (")]
    assert copies.index("wait_inputs") < copies.index("tma_3d")
    counts, epilogue = text[text.index("counts of finished"):text.index("epilogue ----")], text[text.index("epilogue ----"):]
    assert epilogue.index("wait_inputs(U)") < min(epilogue.index(s) for s in ("fetch(0)", "diag[row]", "or_store("))
    # and a tile counts as done after its stores
    assert epilogue.rindex("out[k * A.ld_out]") < epilogue.index("fence.proxy.async") < epilogue.index("bar_arrive(smem_u32(&stored")
    assert counts.index("wait_long(&stored") < counts.index("red.release.gpu")
    # a split's partial sums are added after those of all splits have arrived
    assert epilogue.index("red.release.gpu") < epilogue.index("or_wait_count(count") < epilogue.index("part -=")
