"""The precision of the orthogonalised update on the GPU over steps and coefficients."""
import pytest
import torch

from tests import ortho_precision as op
from tests import ortho_reference as orf
from tests.test_ortho_precision_host import FEW, KINDS, SIDES, STEPS, spectrum

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
    print(f"{rows} x {cols} {steps} {coefficients[0]}: {off:.2e}")
    assert off <= op.bound(min(rows, cols), steps, coefficients), off
    assert h.device_status() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("steps,coefficients", STEPS)
def test_spectra(pkg, kind, steps, coefficients):
    """Stacks of a few dozen rows and fewer, nearly singular ones among them."""
    for n, rows, cols in SIDES:
        side, long = min(rows, cols), max(rows, cols)
        g = spectrum(n, side, long, kind, 8, "cuda")
        g = g if rows <= cols else g.transpose(1, 2).contiguous()
        h = handle(pkg, rows, cols, n, steps=steps, coefficients=coefficients)
        off = op.distances(h(g), op.exact(g, steps, coefficients))
        print(f"{rows} x {cols} {kind} {steps} {coefficients[0]}: {off.median():.2e} {off.max():.2e}")
        assert off.max() <= op.bound(side, steps, coefficients), (rows, cols, off.max())
        assert h.device_status() == 0


@pytest.mark.parametrize("rows,cols", [(300, 520), (1024, 1024), (2048, 600)])
@pytest.mark.parametrize("steps", [6, 8, 12])
def test_larger_matrices(pkg, rows, cols, steps):
    for kind in ("normal", "tokens"):
        g = orf.gradient(rows, cols, "fp32", 3, kind)[None]
        off = op.distances(handle(pkg, rows, cols, steps=steps)(g), op.exact(g, steps)).item()
        print(f"{rows} x {cols} {kind} {steps}: {off:.2e}")
        assert off <= op.bound(min(rows, cols), steps, orf.MUON)
