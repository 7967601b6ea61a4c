"""Stacks of many small matrices on the GPU: each CTA of the orthogonalised update has long runs
of units with nothing to wait for, and counts every one of them."""
import pytest
import torch

from tests import ortho_reference as orf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


def handle(pkg, rows, cols, n=1, dtype="bf16", **kw):
    return pkg.Orthogonalizer(pkg.OrthoConfig(rows=rows, cols=cols, max_matrices=n, dtype=dtype, **kw))


@pytest.mark.parametrize("n,rows,cols", [(153, 32, 32), (4096, 32, 32), (3000, 40, 24), (2500, 24, 40), (1300, 130, 20), (40000, 4, 6)])
def test_many_small_matrices(pkg, n, rows, cols):
    """The same matrix gives the same result wherever it lies in the stack, and alone; one step keeps
    to the definition for all of them."""
    few = 37
    g = torch.stack([orf.gradient(rows, cols, "bf16", i, "normal") for i in range(few)])
    stack = g[torch.arange(n, device="cuda") % few].contiguous()
    op, one = handle(pkg, rows, cols, n), handle(pkg, rows, cols)
    got = op(stack)
    assert op.device_status() == 0
    assert torch.equal(got, got[:few][torch.arange(n, device="cuda") % few])
    for i in range(0, few, 6):
        assert torch.equal(got[i], one(g[i]))   # (the same tiles, K not split: sums in the same order)
    step = handle(pkg, rows, cols, n, steps=1)
    got = step(stack)
    assert step.device_status() == 0
    for i in range(0, few, 6):
        # a rounding to bf16 is off by at most 2^-8 of each value, so of the norm; before it, HELD
        assert orf.distance(got[i], orf.exact(g[i], steps=1)) <= 2.0 ** -8 + orf.HELD
