"""Which kernel a 4-bit call takes (the rule of the streaming kernel's plan, restated),
and mean-square bounds beside the worst-case ones of ops_reference.

Mean squares.  A rounding to a 16-bit type is off by at most u = eps / 2 of the
value, evenly spread: its mean square is at most u^2 / 3 of the value's.  A
product whose weights were rounded adds the same of each of its terms.  fp32
errors are below 2^-23 a step, independent from step to step: the root of the
number of steps times 2^-23 of the partial sums' size, three of them.
"""
import math

import torch

from tests import ops_reference as ref

STREAM_ROWS, WARPS, ROOM = 16, 16, 226 * 1024


def stream_bytes(fmt, G, mats, K, T, depth=2):
    """Shared memory of the streaming kernel: rings, token rows, zeros, partial sums."""
    chunks, nt, wide = (K + 63) // 64, 2 if T > 8 else 1, not (fmt == "affine" and G == 32)
    scale = {"affine": 64 if wide else 128, "nvfp4": 64, "mxfp4": 32}[fmt]
    per = 4 // mats if nt == 1 else 2 if fmt == "affine" and wide else 2 // mats
    stage = mats * per * (512 + scale)
    row = chunks * 128 + (16 if wide else 64)
    return WARPS * depth * stage + T * row + per * 128 + 8 * WARPS * mats * nt * 128 + 16


def streams(fmt, G, mats, K, T):
    return T <= STREAM_ROWS and stream_bytes(fmt, G, mats, K, T) <= ROOM


def most_streamed_rows(fmt, G, mats, K):
    return max(T for T in range(STREAM_ROWS + 1) if T == 0 or streams(fmt, G, mats, K, T))


def bounds(x, w, fmt, G, dtype, mats, s_max=0.01):
    """(worst case, mean square per element) of the error of x w^T before the output's rounding."""
    xd = x.double()
    T, K = xd.shape
    streamed = streams(fmt, G, mats, K, T)
    rounded = 1 if fmt == "affine" and not streamed else 0
    # the streamed codes carry an offset of 128 (fp16: 64) that cancels per group: partial
    # sums of up to 143 (79) scales beside the weight, over the group's steps and three folds
    off = (143.0 if dtype == "bf16" else 79.0) * s_max
    offset = fmt == "affine" and streamed
    extra = off / w.abs().mean().item() * (min(G, 64) / 16 + 3) if offset else 0.0
    worst = ref.product_bound(xd, w, rounded, dtype, extra)
    terms = (xd ** 2) @ (w ** 2).T
    mean = (rounded * ref.unit(dtype) ** 2 / 3) * terms
    size = torch.sqrt(terms)
    steps = K / 16 + 40
    mean = mean + (3 * math.sqrt(steps) * 2.0 ** -23 * size) ** 2
    if offset:
        steps = K / min(G, 64) * (min(G, 64) / 16 + 3)
        mean = mean + (3 * math.sqrt(steps) * 2.0 ** -23 * off) ** 2 * (xd ** 2).mean(1, keepdim=True) * min(G, 64)
    return worst, mean


def check_mean(got, want, mean, dtype, what):
    """The error's mean square over all elements, a tenth for the sample's own spread."""
    u = ref.unit(dtype)
    allowed = (mean + u * u / 3 * want ** 2).mean() + (2.0 ** -24) ** 2 / 3 * (dtype == "fp16")
    err = ((got.double() - want) ** 2).mean()
    assert err <= 1.1 ** 2 * allowed, f"{what}: {math.sqrt(err / allowed):.3g} of the mean-square bound"
