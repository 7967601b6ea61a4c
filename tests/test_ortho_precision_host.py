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


def spectrum(n, side, long, kind, seed, device="cpu"):
    """n matrices [side, long]: normal values, or singular values spread evenly, over four decades
    evenly or at random, or all equal but one that is nearly zero."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64)

    if kind == "normal":
        return normal(n, side, long).float().to(device)
    at = {"even": torch.rand(n, side, generator=gen, dtype=torch.float64),
          "decades": 10.0 ** -torch.linspace(0, 4, side, dtype=torch.float64).expand(n, side),
          "log": 10.0 ** (-3.3 * torch.rand(n, side, generator=gen, dtype=torch.float64)),
          "singular": torch.cat([torch.ones(n, side - 1, dtype=torch.float64),
                                 1e-3 * torch.rand(n, 1, generator=gen, dtype=torch.float64)], 1)}[kind]
    u, v = torch.linalg.qr(normal(n, side, side))[0], torch.linalg.qr(normal(n, long, side))[0]
    return ((u * at[:, None]) @ v.transpose(1, 2)).float().to(device)


KINDS = ("normal", "even", "decades", "log", "singular")
SIDES = [(60, 24, 24), (60, 24, 64), (40, 40, 40), (20, 64, 80), (100, 16, 16), (200, 2, 3), (100, 8, 8), (100, 5, 4)]
STEPS = [(3, orf.MUON), (5, orf.MUON), (6, orf.MUON), (8, orf.MUON), (12, orf.MUON), (5, (1.5, -0.5, 0.0)), (12, (2.0, -1.5, 0.5)),
         (8, (15 / 8, -10 / 8, 3 / 8))]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("steps,coefficients", STEPS)
def test_spectra(kind, steps, coefficients):
    for n, rows, cols in SIDES:
        side, long = min(rows, cols), max(rows, cols)
        g = spectrum(n, side, long, kind, 7)
        g = g if rows <= cols else g.transpose(1, 2).contiguous()
        off = op.distances(op.model(g, steps, coefficients).bfloat16(), op.exact(g, steps, coefficients))
        assert off.max() <= op.bound(side, steps, coefficients), (rows, cols, off.max())


def test_many_steps_stay_bounded():
    """Coefficients that never settle: the errors do not grow beyond what the bound has for any number."""
    for steps in (16, 24, 64):
        for n, side in ((40, 24), (20, 64), (100, 3)):
            g = spectrum(n, side, side + 8, "normal", steps)
            off = op.distances(op.model(g, steps).bfloat16(), op.exact(g, steps))
            assert off.max() <= min(op.bound(side, steps, orf.MUON), 0.2 if side >= 16 else 0.5)
