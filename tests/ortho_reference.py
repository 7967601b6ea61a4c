"""64-bit forms of the orthogonalised update, and how far the GPU's may be off.

`exact` is the definition.  `held` does the same steps and rounds to fp16 where the
kernels hold fp16 (X as two terms, X X^T and its polynomial without their diagonals),
everything else in 64 bits: what is left between it and a GPU's result are fp32 sums.

Bounds, of norms over a whole matrix.  A rounding to bf16 is off by at most 2^-8 of a
value, 2^-8 / sqrt(3) = 2.3e-3 of the norm where values spread over their binades.
  HELD   `held` against `exact`: at most 2e-3 (asserted on the CPU for the inputs here).
  EXACT  a GPU result against `exact`: the two are independent, sqrt(2.3^2 + 2^2) e-3 =
         3.05e-3; bound 2^-8 = 3.9e-3.
  CLOSE  a GPU result of one step against `held` rounded to bf16.  fp32 sums of up to a few
         thousand terms differ by some 1e-6 of their operands' norms; that moves one value in
         2^-11 / 1e-6 = 500 over an fp16 border, by 2^-10 of it: 2^-10 / sqrt(500) = 4.4e-5 of the
         norm for each of the three fp16 matrices, times 4.8 at most (b): below 4e-4.
         Two results that far apart round to bf16 differently in a share of 4e-4 / 2^-8
         of the elements, by 2^-8 each: sqrt(4e-4 2^-8) = 1.25e-3; bound 2e-3.
         After more steps there is no such bound: an element of hi on the other side of a
         border, 2^-10 of it away, moves a whole row of X X^T by 2^-10 / sqrt(n) of its entries, and
         2 / sqrt(n) of them over borders of their own (n = 256: one in eight), so that after
         a few steps the roundings of two results have nothing in common; both
         stay as near to `exact`.
  TWO    two GPU results of the same matrix whose sums were taken in another order:
         each within EXACT, independently: sqrt(2) EXACT.
  BLOCK  32 x 32 blocks against `exact`: an error that falls on few elements stays small in
         the norm of a matrix; here a block's error may be 1/8 of the norm that it has plus
         the norm of a block of the matrix's mean square (a wrong block is off by its own norm).
"""
import math

import torch

MUON = (3.4445, -4.7750, 2.0315)
HELD, EXACT, CLOSE, BLOCK = 2e-3, 2.0 ** -8, 2e-3, 1 / 8
TWO = math.sqrt(2) * EXACT


def start(g, eps):
    x = g.double()
    return x / (torch.sqrt((x * x).sum()) + eps)


def exact(g, steps=5, coefficients=MUON, eps=1e-7):
    """One matrix, in 64 bits."""
    a, b, c = coefficients
    tall = g.shape[0] > g.shape[1]
    x = start(g.T if tall else g, eps)
    for _ in range(steps):
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.T if tall else x


def half(x):
    return x.half().double()


def held(g, steps=5, coefficients=MUON, eps=1e-7):
    """One matrix with the kernels' fp16 roundings."""
    a, b, c = coefficients
    tall = g.shape[0] > g.shape[1]
    x = start(g.T if tall else g, eps)
    s = 2.0 ** min(6, int(math.log2(x.shape[0]) / 2 + 1e-9))
    x = x * s
    for _ in range(steps):
        hi = half(x)
        lo = half(x - hi)
        gram = hi @ hi.T
        d = gram.diagonal().clone()
        o = half(gram - torch.diag(d))
        oo = o @ o
        p = b * o + c / s ** 2 * (oo + o * (d[:, None] + d[None, :]))
        e = (b * d + c / s ** 2 * (oo.diagonal() + d * d)) / s ** 2
        p = half(p - torch.diag(p.diagonal()))
        x = (a + e[:, None]) * hi + a * lo + (p @ hi) / s ** 2
    x = x / s
    return x.T if tall else x


def gradient(rows, cols, dtype, seed, kind="tokens", device="cuda", n=None):
    """A weight gradient: of tokens (`few`: of 9 tokens), of channels of unequal size; or normal values."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=device)

    out = []
    for _ in range(1 if n is None else n):
        if kind == "normal":
            g = normal(rows, cols)
        else:
            tokens = min(9, rows, cols) if kind == "few" else 2 * min(rows, cols)
            g = (normal(tokens, rows) * torch.exp(normal(rows))).T @ (normal(tokens, cols) * torch.exp(0.5 * normal(cols)))
        out.append((1e-3 * g).to({"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[dtype]))
    return out[0] if n is None else torch.stack(out)


def distance(x, y):
    return ((x.double() - y.double()).norm() / y.double().norm()).item()


def check(got, g, what, **kw):
    """One matrix of the GPU against the definition, after one step also against `held`."""
    assert got.dtype == torch.bfloat16
    want = exact(g, **kw)
    assert torch.isfinite(got).all(), what
    d = distance(got, want)
    assert d <= EXACT, f"{what}: {d:.3g} from exact"
    if kw.get("steps") == 1:
        d = distance(got, held(g, **kw).bfloat16())
        assert d <= CLOSE, f"{what}: {d:.3g} from held"
    # blocks
    err, ref = got.double() - want, want
    R, C = err.shape
    pad = (0, -C % 32, 0, -R % 32)
    as_blocks = lambda t: torch.nn.functional.pad(t, pad).reshape((R + 31) // 32, 32, (C + 31) // 32, 32).pow(2).sum((1, 3)).sqrt()  # noqa: E731
    rms = ref.pow(2).mean().sqrt()
    worst = (as_blocks(err) / (as_blocks(ref) + 32 * rms)).max().item()
    assert worst <= BLOCK, f"{what}: a block is off by {worst:.3g}"
