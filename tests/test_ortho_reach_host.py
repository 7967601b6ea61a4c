"""Coefficients of the orthogonalised update that are accepted keep every finite matrix finite (no
GPU needed)."""
import ctypes
import os
import random

import pytest
import torch

import quantized_moe_decode_gemv_gb300 as pkg
from quantized_moe_decode_gemv_gb300 import _capi
from tests import ortho_precision as op
from tests import ortho_reference as orf


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_capi.LIB_PATH):
        pytest.fail("libmoe_gb300.so is not built; run __graft_entry__.build()")
    return _capi.load_library()


def status(lib, coefficients, steps):
    c = pkg.OrthoConfig(rows=64, cols=64, steps=steps, coefficients=coefficients, eps=0.0).to_c()
    return _capi.STATUS_NAMES[lib.moe_ortho_validate(ctypes.byref(c))]


@pytest.mark.parametrize("coefficients,steps,want", [
    (orf.MUON, 5, "MOE_OK"), (orf.MUON, 64, "MOE_OK"), ((1.5, -0.5, 0.0), 64, "MOE_OK"), ((2.0, -1.5, 0.5), 64, "MOE_OK"),
    ((15 / 8, -10 / 8, 3 / 8), 64, "MOE_OK"), ((1.0, 0.0, 0.0), 64, "MOE_OK"), ((2.5, -3.5, 2.0), 5, "MOE_OK"),
    ((2.5, -3.5, 2.0), 30, "MOE_ERR_UNSUPPORTED"), ((0.5, 0.5, 0.0), 64, "MOE_ERR_UNSUPPORTED"), ((2.0, 0.0, 0.0), 1, "MOE_OK"),
    ((1.0, -1.0, 1.0), 64, "MOE_ERR_UNSUPPORTED"),
])
def test_singular_values_that_rounding_pushes_up(lib, coefficients, steps, want):
    assert status(lib, coefficients, steps) == want


def ones(n, seed):
    """Matrices of rank one: a singular value of 1, where rounding alone decides on which side."""
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(n, 24, 1, generator=gen) @ torch.randn(n, 1, 32, generator=gen)


def test_what_is_accepted_stays_finite(lib):
    """Polynomials with p(1) = 1 of any slope there, and others, as many steps as are accepted."""
    rng = random.Random(1)
    g, accepted, refused = ones(12, 3), 0, 0
    for i in range(300):
        a, b = rng.uniform(0.2, 4.0), rng.uniform(-7.0, 1.0)
        c = 1 - a - b if i % 3 else rng.uniform(-1.0, 3.5)
        steps = rng.choice([3, 5, 8, 16, 30, 64])
        if status(lib, (a, b, c), steps) != "MOE_OK":
            refused += 1
            continue
        accepted += 1
        x = op.model(g, steps, (a, b, c), eps=0.0)
        assert torch.isfinite(x).all(), (a, b, c, steps)
        # the largest singular value: 4, and what the last step's rounding adds
        assert torch.linalg.matrix_norm(x, 2).max() <= 4.0 * (1 + 2.0 ** -9), (a, b, c, steps)
    assert accepted >= 60 and refused >= 60
