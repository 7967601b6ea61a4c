"""Plain 64-bit forms of the tokens sorted by expert and back, written pick by pick,
and the inputs of their tests.

Bounds (u: half a step of the rows' type).  Sums are fp32: n additions of products, each
a fused multiply-add, are off by at most n 2^-24 of the sum of magnitudes (a term more
covers the second order); the result is rounded once more to its type.
"""
import numpy as np
import torch

from tests.ops_reference import DT


def make_ids(T, k, E, seed, drop=0.0, skew=1.0):
    """[T, k] int64: different experts in a row while there are enough, -1 for a share of `drop`."""
    rng = np.random.default_rng(seed)
    score = rng.gumbel(size=(T, E)) - skew * np.log1p(rng.permutation(E))
    ids = np.argsort(-score, axis=1)[:, :k].astype(np.int64)
    if k > E:
        ids = rng.integers(0, E, (T, k))
    ids[rng.random((T, k)) < drop] = -1
    return torch.from_numpy(ids)


def plan(ids, E):
    """(offsets, order, place) by counting, in plain Python."""
    flat = ids.reshape(-1).tolist()
    rows = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            rows[e].append(i)
    offsets, order, place = [0], [], [-1] * len(flat)
    for e in range(E):
        for i in rows[e]:
            place[i] = len(order)
            order.append(i)
        offsets.append(len(order))
    order += [-1] * (len(flat) - len(order))
    as_t = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return as_t(offsets), as_t(order), as_t(place).reshape(ids.shape)


def take(x, p, k):
    """rows (x's own type)."""
    _, order, _ = p
    out = torch.zeros(order.numel(), x.shape[1], dtype=x.dtype, device=x.device)
    here = order >= 0
    out[here] = x[(order[here] // k).long()]
    return out


def combine(y, w, p):
    """(out, bound of its fp32 error) in 64 bits; w None: ones."""
    place = p[2]
    T, k = place.shape
    out = torch.zeros(T, y.shape[1], dtype=torch.float64, device=y.device)
    mag = torch.zeros_like(out)
    for j in range(k):
        here = place[:, j] >= 0
        term = y[place[here, j].long()].double()
        if w is not None:
            term = term * w[here, j, None].double()
        out[here] += term
        mag[here] += term.abs()
    return out, (k + 1) * 2.0 ** -24 * mag


def combine_backward(d_out, y, w, p):
    """((d_y, bound), (d_w, bound)) in 64 bits."""
    _, order, place = p
    T, k = place.shape
    H = y.shape[1]
    e, d_y = d_out.double(), torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    here = order >= 0
    pick = order[here].long()
    d_y[here] = w.double().reshape(-1)[pick, None] * e[pick // k]
    d_w = torch.zeros(T, k, dtype=torch.float64, device=y.device)
    mag = torch.zeros_like(d_w)
    for j in range(k):
        at = place[:, j] >= 0
        prod = e[at] * y[place[at, j].long()].double()
        d_w[at, j] = prod.sum(1)
        mag[at, j] = prod.abs().sum(1)
    return (d_y, 2.0 ** -23 * d_y.abs()), (d_w, (H + 1) * 2.0 ** -24 * mag)


def rows(n, H, dtype, seed, pad=0, device="cuda"):
    """[n, H] normal values, a column range of a wider buffer when pad is given."""
    gen = torch.Generator(device=device).manual_seed(seed)
    return torch.randn(n, H + pad, generator=gen, device=device).to(DT[dtype])[:, pad:]
