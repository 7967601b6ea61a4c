"""The precision of the orthogonalised update on the GPU over steps and coefficients."""
import pytest
import torch

from tests import ortho_precision as op
from tests import ortho_reference as orf
from tests.test_ortho_precision_host import FEW

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


def handle(pkg, rows, cols, n=1, dtype="fp32", **kw):
    return pkg.Orthogonalizer(pkg.OrthoConfig(rows=rows, cols=cols, max_matrices=n, dtype=dtype, **kw))


@pytest.mark.parametrize("rows,cols,steps,coefficients", FEW)
def test_few_tokens(pkg, rows, cols, steps, coefficients):
    g = orf.gradient(rows, cols, "fp32", 2, "few")[None]
    h = handle(pkg, rows, cols, steps=steps, coefficients=coefficients)
    off = op.distances(h(g), op.exact(g, steps, coefficients)).item()
    assert off <= op.bound(min(rows, cols), steps, coefficients), off
    assert h.device_status() == 0
