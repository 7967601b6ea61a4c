"""How far an orthogonalised update may be off over all steps and coefficients, and the model of
its roundings that this rests on.

`model` takes the kernels' steps with their roundings: fp16 operands, the diagonals apart, X as
hi + 2^-11 lo, X itself in fp32; products in 64 bits (or fp32, to see what sums add).  `bound` is
what the header states, as a share of the norm of the 64-bit result:

  table   what the operands' roundings do.  Coefficients that never settle multiply a singular
          value's error from step to step; the values are no smaller than the largest that `model`
          gave over thousands of matrices of five kinds of spectra (smaller sides of 16 to 128,
          out rounded to bf16: 3.4e-3 in five steps, 4.2e-3 in six, 7.0e-3 in eight, 2.7e-2 in twelve,
          0.14 in 24 and 64).  Smaller sides below 16 have few errors that could average: 1.4e-2,
          2.0e-2, 4.5e-2, 0.22, 0.45, within eight times the table.  Coefficients that settle: out's
          rounding, below 4e-3 whatever the steps.
  noise   X's rounding has parts in directions that X has not, where each step multiplies by a.
          Two fp16 terms of 11 bits leave at most 2^-22 of an element, 2^-24 in the mean square; fp32
          sums of K terms some 2^-24 sqrt(K / 16) of the result a step.  The norm grows to
          sqrt(rank) meanwhile, so |a|^steps 2^-22 has room for a geometric series of them.
"""
import math

import torch

from tests import ortho_reference as orf

SETTLING = [(1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (15 / 8, -10 / 8, 3 / 8)]
TABLE = ((5, 4e-3), (6, 5e-3), (8, 8e-3), (12, 3e-2), (64, 0.2))


def bound(side, steps, coefficients):
    """`side`: the smaller one."""
    base = 4e-3
    if tuple(coefficients) not in SETTLING:
        base = next(b for s, b in TABLE if steps <= s)
        if side < 16:
            base = min(8 * base, 0.5)
    elif side < 16:
        base = 8e-3
    return base + abs(coefficients[0]) ** steps * 2.0 ** -22


def _product(x, y, sums):
    return (x.to(sums) @ y.to(sums)).double()


def model(g, steps=5, coefficients=orf.MUON, eps=1e-7, lo_scale=2.0 ** 11, sums=torch.float64):
    """[n, rows, cols] -> the same in 64 bits, before out's rounding."""
    a, b, c = coefficients
    tall = g.shape[1] > g.shape[2]
    x = (g.transpose(1, 2) if tall else g).double()
    x = x / (x.flatten(1).norm(dim=1)[:, None, None] + eps)
    m = x.shape[1]
    s = 2.0 ** min(6, int(math.log2(m) / 2 + 1e-9))
    off = 1 - torch.eye(m, dtype=torch.float64, device=x.device)

    def terms(x):
        x = x.float().double()
        hi = orf.half(x)
        return hi, orf.half((x - hi) * lo_scale) / lo_scale

    hi, lo = terms(x * s)
    for _ in range(steps):
        gram = _product(hi, hi.transpose(1, 2), sums)
        d, o = gram.diagonal(dim1=1, dim2=2).clone(), orf.half(gram * off)
        oo = _product(o, o, sums)
        p = orf.half((b * o + c / s ** 2 * (oo + o * (d[:, :, None] + d[:, None, :]))) * off)
        e = (b * d + c / s ** 2 * (oo.diagonal(dim1=1, dim2=2) + d * d)) / s ** 2
        x = (a + e[:, :, None]) * hi + a * lo + _product(p, hi, sums) / s ** 2
        hi, lo = terms(x)
    x = x / s
    return x.transpose(1, 2) if tall else x


def exact(g, steps=5, coefficients=orf.MUON, eps=1e-7):
    """The definition in 64 bits for a stack."""
    a, b, c = coefficients
    tall = g.shape[1] > g.shape[2]
    x = (g.transpose(1, 2) if tall else g).double()
    x = x / (x.flatten(1).norm(dim=1)[:, None, None] + eps)
    for _ in range(steps):
        s = x @ x.transpose(1, 2)
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.transpose(1, 2) if tall else x


def distances(x, y):
    return (x.double() - y.double()).flatten(1).norm(dim=1) / y.double().flatten(1).norm(dim=1)
