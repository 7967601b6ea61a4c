"""Plain 64-bit forms of the operators around the MoE layer, and the error
bounds their GPU results are held to.

Bounds.  An output is rounded once to its 16-bit type: at most
u = finfo(type).eps / 2 of its value (bf16 2^-8, fp16 2^-11).  What comes before is
fp32: a sum that passes n accumulations of partial sums of magnitude A is off by at
most n 2^-23 A (a tensor-core accumulation may truncate, so a whole step each).
Where a factor of every product was rounded to 16 bits on its way into the
tensor cores (expanded affine weights, dg and du), the roundings are independent
and each uniform within u of its value at most, with variance u^2 / 3, so the
sum's error has the standard deviation u / sqrt(3) * sqrt(sum of squared
products); seven of them bound it (chance 3e-12 an element).  Inputs that pass
through an activation carry the bound times the activation's slope.
"""
import math

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e4m3(byte: int) -> float:
    e, m = (byte >> 3) & 15, byte & 7
    if byte & 127 == 127:
        return math.nan
    v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -v if byte & 128 else v


E4M3 = np.array([e4m3(b) for b in range(256)])


def unit(dtype: str) -> float:
    return torch.finfo(DT[dtype]).eps / 2


def make_weight(N, K, fmt, G, sdt, seed):
    """Random codes and scales: (dict of CPU tensors by field name, fp64 matrix)."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (N, K))
    word = np.zeros((N, K // 8), np.uint32)
    for i in range(8):
        word |= codes[:, i::8].astype(np.uint32) << np.uint32(4 * i)
    q = torch.from_numpy(word.view(np.int32))
    if fmt == "affine":
        s = torch.from_numpy(0.005 * (1 + rng.random((N, K // G)))).to(DT[sdt])
        b = torch.from_numpy(-0.04 - 0.03 * rng.random((N, K // G))).to(DT[sdt])
        S, B = (t.double().numpy().repeat(G, 1) for t in (s, b))
        return {"q": q, "s": s, "b": b}, codes * S + B
    if fmt == "nvfp4":
        # every positive byte but NaN, subnormals and zero among them, some negative
        s = rng.integers(0, 127, (N, K // G)) | (128 * (rng.random((N, K // G)) < 0.1))
        s = np.where(rng.random(s.shape) < 0.7, 56 + s % 8, s).astype(np.uint8)
        ms = np.array([0.013], np.float32)
        return ({"q": q, "s": torch.from_numpy(s), "b": torch.from_numpy(ms)},
                E2M1[codes] * E4M3[s].repeat(G, 1) * float(ms[0]))
    s = rng.integers(112, 124, (N, K // G)).astype(np.uint8)
    return {"q": q, "s": torch.from_numpy(s), "b": None}, E2M1[codes] * np.exp2(s.astype(np.float64) - 127).repeat(G, 1)


def silu(g):
    return g / (1 + torch.exp(-g))


def activate(act, g, u):
    if act == "swiglu":
        return silu(g) * u
    if act == "relu2":
        return torch.clamp(u, min=0) ** 2
    return u


def act_bound(act, g, u, eg, eu):
    """Bound of the activation's error for errors eg, eu of g and u: slopes at the
    values (|silu'| <= 1.1) and the second-order term, plus the fp32 activation
    itself (exp, divide, two products: 8 steps)."""
    if act == "swiglu":
        h = silu(g) * u
        return 1.1 * (u.abs() + eu) * eg + (silu(g).abs() + 1.1 * eg) * eu + (8 + g.abs()) * 2.0 ** -23 * h.abs()
    if act == "relu2":
        up = torch.clamp(u, min=0)
        return 2 * (up + eu) * eu + 2.0 ** -23 * up ** 2
    return eu


def product_bound(x, w, roundings, dtype, extra=0.0):
    """Error bound of x w^T in fp32 (fp64 tensors on the device): K / 16 tensor-core
    accumulations and the joins of partial sums; `roundings` 16-bit roundings of a
    factor; `extra` multiplies sum |x| |w| (offset arithmetic of the affine codes)."""
    K = x.shape[1]
    mag = x.abs() @ w.abs().T
    e = (K / 16 + 40 + extra) * 2.0 ** -23 * mag
    if roundings:
        e = e + 7 * math.sqrt(roundings / 3) * unit(dtype) * torch.sqrt((x ** 2) @ (w ** 2).T)
    return e


def check(got, want, bound, dtype, what):
    """Every element within its bound and the output's own rounding (fp16: or half
    of its smallest step, 2^-25).  A value from half a step above the type's largest
    one rounds to infinity (fp16: 65504 + 16): there infinity is the right answer,
    and either answer is within the bound of that border."""
    got = got.double()
    # half a step above the largest value (its step: 2 u of the binade's start)
    top = torch.finfo(DT[dtype]).max
    border = top + unit(dtype) * 2.0 ** math.floor(math.log2(top))
    large = want.abs() + bound >= border
    sure = want.abs() - bound >= border
    assert (got[sure] == torch.sign(want[sure]) * math.inf).all(), f"{what}: overflow"
    assert (got[large & torch.isinf(got)] * want[large & torch.isinf(got)] > 0).all(), f"{what}: sign of infinity"
    fine = ~(large & torch.isinf(got))
    got, want, bound = got[fine], want[fine], bound[fine]
    assert torch.isfinite(got).all(), f"{what}: not finite"
    tol = bound + unit(dtype) * (want.abs() + bound) + (2.0 ** -25 if dtype == "fp16" else 2.0 ** -134)
    over = ((got - want).abs() / tol).max().item() if got.numel() else 0.0
    assert over <= 1, f"{what}: {over:.3g} of the bound"
