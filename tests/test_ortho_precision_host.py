"""The roundings of the orthogonalised update over steps and coefficients, simulated (no GPU needed)."""
import pytest
import torch

from tests import ortho_precision as op
from tests import ortho_reference as orf

# matrices of few tokens, and steps after which a second term that ends at 2^-24 has been
# multiplied into the result
FEW = [(64, 8192, 10, orf.MUON), (8192, 64, 10, orf.MUON), (256, 1024, 9, orf.MUON), (64, 8192, 24, (1.5, -0.5, 0.0)),
       (64, 4096, 16, (2.0, -1.5, 0.5)), (64, 8192, 16, (15 / 8, -10 / 8, 3 / 8))]


@pytest.mark.parametrize("rows,cols,steps,coefficients", FEW)
def test_few_tokens(rows, cols, steps, coefficients):
    g = orf.gradient(rows, cols, "fp32", 2, "few", device="cpu")[None]
    want = op.exact(g, steps, coefficients)
    bound = op.bound(min(rows, cols), steps, coefficients)
    off = [op.distances(op.model(g, steps, coefficients, sums=sums).bfloat16(), want).item() for sums in (torch.float64, torch.float32)]
    assert max(off) <= bound / 2     # room for sums in another order
    # a second term at its own size loses several times as much
    assert op.distances(op.model(g, steps, coefficients, lo_scale=1.0).bfloat16(), want).item() > 3 * max(off)
