"""Operators around the training of routed experts, as cases that can be timed.

Two operators and their parts, each in a plain form (elementary torch operations
in fp32, rounded once at the end) and as the library's own calls:

  dispatch  picks [T, k] of experts -> the tokens' rows sorted by expert:
            offsets[e] = the number of picks below expert e, order = the picks in a
            stable sort by expert, place = the row of every pick,
            rows[r] = x[order[r] / k].  A pick of -1 has no expert: its place is -1,
            it is sorted last, and its row is zero
  combine   out[t] = sum_j w[t, j] y[place[t, j]] over the present picks
  rows      both, and their gradients:
            d_y[r] = w[order[r]] d_out[order[r] / k],  d_w[t, j] = <d_out[t], y[place[t, j]]>,
            d_x[t] = sum_j d_rows[place[t, j]]
  ortho     a stack of matrices G, each brought near the orthogonal matrix of its
            singular vectors: X = G / (|G| + eps) and, `steps` times,
            A = X X^T,  X = a X + (b A + c A A) X
            (with |G| the Frobenius norm; a tall matrix from its other side)

A case is a dict: `op`, then `T`, `k`, `E`, `H` (token rows, picks a row,
experts, width), `dtype`, `ids` (type of the picks), `w` (type of the weights),
`drop` (share of absent picks) and `pad` (x is a column range of a buffer that
is `pad` columns wider); or `B`, `M`, `N` (matrices, rows, columns), `dtype` and
`steps`.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int32": torch.int32,
          "int64": torch.int64}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def listed():
    return [
        # one decoded token to its nine experts' rows, at the latent width: the smallest call
        dict(name="dispatch_t1", op="dispatch", T=1, k=9, E=496, H=1024, dtype="bf16", ids="int32", w="fp32", drop=0.0, pad=0),
        # a ragged batch of an odd width, with picks that a capacity limit dropped
        dict(name="dispatch_t77_odd", op="dispatch", T=77, k=6, E=130, H=1001, dtype="fp16", ids="int64", w="fp32", drop=0.1, pad=0),
        # a training batch's rows at the non-latent width
        dict(name="dispatch_t4096", op="dispatch", T=4096, k=8, E=256, H=6144, dtype="bf16", ids="int64", w="fp32", drop=0.0, pad=0),
        # sixteen streams decoded together: the experts' outputs of the latent layer back to the tokens
        dict(name="combine_t16", op="combine", T=16, k=9, E=496, H=1024, dtype="bf16", ids="int32", w="fp32", drop=0.0, pad=0),
        # a chunk of prefill, weights in the activations' type, some picks dropped
        dict(name="combine_t2000", op="combine", T=2000, k=8, E=256, H=6144, dtype="fp16", ids="int32", w="fp16", drop=0.05, pad=0),
        # a small fine-tuning step: to the experts, back, and all gradients; x a slice of a wider buffer
        dict(name="rows_t333", op="rows", T=333, k=9, E=496, H=1024, dtype="bf16", ids="int32", w="fp32", drop=0.03, pad=64),
        # a full training step's rows
        dict(name="rows_t8192", op="rows", T=8192, k=9, E=496, H=1024, dtype="bf16", ids="int32", w="fp32", drop=0.0, pad=0),
        # the update of a small projection: the fewest operations, where latency counts
        dict(name="ortho_64x256", op="ortho", B=1, M=64, N=256, dtype="bf16", steps=5),
        # the update of a latent projection
        dict(name="ortho_1024x4096", op="ortho", B=1, M=1024, N=4096, dtype="bf16", steps=5),
        # a tall matrix of odd sizes, momentum in 32 bits
        dict(name="ortho_1999x777", op="ortho", B=1, M=1999, N=777, dtype="fp32", steps=5),
        # sixteen experts' up matrices in one call
        dict(name="ortho_16x1856x1024", op="ortho", B=16, M=1856, N=1024, dtype="fp32", steps=5),
        # the weights of a gated block, the largest
        dict(name="ortho_8192x4096", op="ortho", B=1, M=8192, N=4096, dtype="bf16", steps=5),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    if rng.random() < 0.6:
        op = rng.choice(["dispatch", "combine", "rows"])
        most = 8192 * 9 * 1024
        while True:
            T, k, H = _log(rng, 1, 8192), rng.choice([1, 2, 4, 6, 8, 9]), _log(rng, 64, 8192)
            if rng.random() < 0.6:
                H = max(64, H // 32 * 32)
            if T * k * H <= most:
                break
        dtype = rng.choice(["bf16", "fp16"])
        return dict(op=op, T=T, k=k, E=_log(rng, max(k, 4), 512), H=H, dtype=dtype, ids=rng.choice(["int32", "int64"]),
                    w=rng.choice(["fp32", "fp32", dtype]), drop=rng.choice([0.0, 0.0, 0.05, 0.3]),
                    pad=rng.choice([0, 0, 8, 40]))
    most = _flops(dict(M=8192, N=4096, B=1, steps=5))
    while True:
        c = dict(op="ortho", B=rng.choice([1, 1, _log(rng, 2, 32)]), M=_log(rng, 32, 8192), N=_log(rng, 32, 8192),
                 dtype=rng.choice(["bf16", "fp16", "fp32"]), steps=rng.choice([5, 5, 5, 3, 6]))
        if _flops(c) <= most and c["B"] * c["M"] * c["N"] <= 8192 * 4096:
            return c


def _flops(c):
    m, n = min(c["M"], c["N"]), max(c["M"], c["N"])
    # a step: X X^T and A A are symmetric, one half of each; then B X
    return c["B"] * c["steps"] * (m * m * n + m * m * m + 2 * m * m * n)


def work(case):
    if case["op"] == "ortho":
        one = case["B"] * case["M"] * case["N"]
        return {"bytes": one * (4 if case["dtype"] == "fp32" else 2) + one * 2, "flops": _flops(case)}
    T, k, H = case["T"], case["k"], case["H"]
    P = T * k
    ids = P * (4 if case["ids"] == "int32" else 8)
    w = P * (4 if case["w"] == "fp32" else 2)
    tokens, rows, here = 2 * T * H, 2 * P * H, int(2 * P * H * (1 - case["drop"]))
    plan = 4 * (2 * P + case["E"] + 1)
    dispatch = {"bytes": tokens + ids + rows + plan, "flops": 0}
    combine = {"bytes": here + w + 4 * P + tokens, "flops": here}
    if case["op"] == "dispatch":
        return dispatch
    if case["op"] == "combine":
        return combine
    # d_out and y again are read, d_y and d_w written; d_rows read, d_x written
    grads = tokens + rows + w + here + tokens
    return {"bytes": dispatch["bytes"] + combine["bytes"] - 4 * P + grads, "flops": 4 * here}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1_000_003 * (seed + 1) + 7 * sum(v for v in case.values() if type(v) is int))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    dt = DTYPES[case["dtype"]]
    if case["op"] == "ortho":
        # a weight gradient of as many tokens as the short side, of channels of unequal size,
        # as momentum holds it
        B, M, N = case["B"], case["M"], case["N"]
        tokens = min(M, N)
        e = normal(B, tokens, M) * torch.exp(normal(B, 1, M))
        x = normal(B, tokens, N) * torch.exp(0.5 * normal(B, 1, N))
        return {"case": case, "g": (torch.bmm(e.transpose(1, 2), x) * (1e-3 / math.sqrt(tokens))).to(dt)}
    T, k, E, H = case["T"], case["k"], case["E"], case["H"]
    # picks without repetition in a row, of experts of unequal popularity
    popular = -1.1 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    popular = popular[torch.randperm(E, generator=gen, device="cuda")]
    chance = torch.rand(T, E, generator=gen, device="cuda").clamp(min=1e-20)
    ids = torch.topk(0.5 * popular - torch.log(-torch.log(chance).clamp(min=1e-20)), k, dim=1).indices
    absent = torch.rand(T, k, generator=gen, device="cuda") < case["drop"]
    d = {"case": case, "ids": torch.where(absent, torch.full_like(ids, -1), ids).to(DTYPES[case["ids"]])}
    if case["op"] != "combine":
        d["x"] = normal(T, H + case["pad"]).to(dt)[:, case["pad"]:]
    if case["op"] != "dispatch":
        score = torch.sigmoid(normal(T, k))
        d["w"] = (2.5 * score / score.sum(1, keepdim=True)).to(DTYPES[case["w"]])
        d["y"] = (0.3 * normal(T * k, H)).to(dt)
    if case["op"] == "rows":
        d["d_out"] = (0.05 * normal(T, H)).to(dt)
        d["d_rows"] = (0.05 * normal(T * k, H)).to(dt)
    return d


def prepare(case, seed):
    state = _inputs(case, seed)
    if case["op"] == "combine":
        state["plan"] = _plain_plan(state["ids"], case["E"])   # a user has it from the dispatch
    if own:
        import quantized_moe_decode_gemv_gb300 as pkg
        if case["op"] == "ortho":
            cfg = pkg.OrthoConfig(rows=case["M"], cols=case["N"], max_matrices=case["B"], dtype=case["dtype"],
                                  steps=case["steps"], coefficients=COEFFICIENTS, eps=EPS)
            state["ortho"] = pkg.Orthogonalizer(cfg)
        else:
            cfg = pkg.ExpertRowsConfig(n_experts=case["E"], top_k=case["k"], act_dtype=case["dtype"],
                                       max_tokens=case["T"])
            state["expert_rows"] = pkg.ExpertRows(cfg)
            if case["op"] == "combine":
                state["plan"] = pkg.RowPlan(*state["plan"])
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _plain_plan(ids, E):
    """(offsets [E + 1], order [T k], place [T, k]), int32."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    bounds = torch.arange(E + 1, device=ids.device)
    offsets = torch.searchsorted(key[order].contiguous(), bounds)
    order = torch.where(key[order] == E, torch.full_like(order, -1), order)
    place = torch.where(flat < 0, torch.full_like(place, -1), place)
    return offsets.int(), order.int(), place.int().reshape(ids.shape)


def _plain_rows(x, order, k):
    """x's row of every pick in order, zero where there is none."""
    here = (order >= 0)[:, None]
    return torch.where(here, x[order.clamp(min=0).long() // k], torch.zeros((), dtype=x.dtype, device=x.device))


def _plain_sum(y, place, w=None):
    picked = y.float()[place.clamp(min=0).long()]
    if w is not None:
        picked = picked * w.float()[:, :, None]
    return torch.where((place >= 0)[:, :, None], picked, torch.zeros((), device=y.device)).sum(1)


def _plain_ortho(g, steps):
    wide = g.shape[1] <= g.shape[2]
    x = g.float() if wide else g.float().transpose(1, 2)
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(steps):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return (x if wide else x.transpose(1, 2)).to(torch.bfloat16).contiguous()


def _plain(state):
    case = state["case"]
    if case["op"] == "ortho":
        return _plain_ortho(state["g"], case["steps"])
    dt = DTYPES[case["dtype"]]
    if case["op"] == "combine":
        return _plain_sum(state["y"], state["plan"][2], state["w"]).to(dt)
    offsets, order, place = _plain_plan(state["ids"], case["E"])
    out = {"rows": _plain_rows(state["x"], order, case["k"]), "offsets": offsets, "order": order, "place": place}
    if case["op"] == "dispatch":
        return out
    w, y, d_out = state["w"], state["y"], state["d_out"]
    out["out"] = _plain_sum(y, place, w).to(dt)
    pick = order.clamp(min=0).long()
    d_y = w.float().reshape(-1)[pick][:, None] * d_out.float()[pick // case["k"]]
    out["d_y"] = torch.where((order >= 0)[:, None], d_y, torch.zeros((), device=y.device)).to(dt)
    dots = (y.float()[place.clamp(min=0).long()] * d_out.float()[:, None, :]).sum(2)
    out["d_w"] = torch.where(place >= 0, dots, torch.zeros((), device=y.device)).to(w.dtype)
    out["d_x"] = _plain_sum(state["d_rows"], place).to(dt)
    return out


def run(state):
    if not own:
        return _plain(state)
    case = state["case"]
    if case["op"] == "ortho":
        return state["ortho"](state["g"])
    h = state["expert_rows"]
    if case["op"] == "combine":
        return h.combine(state["y"], state["w"], state["plan"])
    rows, plan = h.dispatch(state["x"], state["ids"])
    out = {"rows": rows, "offsets": plan.offsets, "order": plan.order, "place": plan.place}
    if case["op"] == "dispatch":
        return out
    out["out"] = h.combine(state["y"], state["w"], plan)
    d = h.combine_backward(state["d_out"], state["y"], state["w"], plan)
    out["d_y"], out["d_w"] = d.y, d.w
    out["d_x"] = h.dispatch_backward(state["d_rows"], plan)
    return out


# ---------------------------------------------------------------------------
# from the definition, in 64 bits
# ---------------------------------------------------------------------------

def _exact_ortho(g, steps):
    x = g.double()
    x = x / (torch.linalg.norm(x) + EPS)
    a, b, c = COEFFICIENTS
    one = torch.eye(min(x.shape), dtype=torch.float64, device=x.device)
    for _ in range(steps):
        # p(X) = (a + b X X^T + c (X X^T)^2) X = X (a + b X^T X + c (X^T X)^2), by the smaller of the two
        if x.shape[0] <= x.shape[1]:
            s = torch.einsum("ik,jk->ij", x, x)
            x = (a * one + torch.einsum("ij,jk->ik", s, b * one + c * s)) @ x
        else:
            s = torch.einsum("ki,kj->ij", x, x)
            x = x @ (a * one + torch.einsum("ij,jk->ik", s, b * one + c * s))
    return x


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "ortho":
        return torch.stack([_exact_ortho(g, case["steps"]) for g in d["g"]])
    T, k, E, H = case["T"], case["k"], case["E"], case["H"]
    ids = d["ids"].long()
    # a pick's row: the present picks of lower experts, and those of its own before it (row by row)
    flat = ids.reshape(-1)
    present = flat >= 0
    number = torch.bincount(flat[present], minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(number, 0)
    unique = torch.where(present, flat, torch.full_like(flat, E)) * (T * k) + torch.arange(T * k, device="cuda")
    order = torch.sort(unique).values % (T * k)
    place = torch.full((T * k,), -1, dtype=torch.int64, device="cuda")
    rows = int(offsets[E])
    place[order[:rows]] = torch.arange(rows, device="cuda")
    order[rows:] = -1
    place = place.reshape(T, k)
    valid = (place >= 0).double()

    def spread(tokens, weight):   # [T, H] -> [T k, H], a pick's share at its place
        out = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            mine = place[:, j] >= 0
            out[place[mine, j]] = tokens[mine] * weight[mine, j, None]
        return out

    def gather(rows64, weight):   # the reverse
        out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            mine = place[:, j] >= 0
            out[mine] += rows64[place[mine, j]] * weight[mine, j, None]
        return out

    if case["op"] == "combine":
        return gather(d["y"].double(), d["w"].double())
    out = {"rows": spread(d["x"].double(), valid), "offsets": offsets.int(), "order": order.int(), "place": place.int()}
    if case["op"] == "dispatch":
        return out
    w, y, d_out = d["w"].double(), d["y"].double(), d["d_out"].double()
    out["out"] = gather(y, w)
    out["d_y"] = spread(d_out, w)
    d_w = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        mine = place[:, j] >= 0
        d_w[mine, j] = torch.einsum("th,th->t", d_out[mine], y[place[mine, j]])
    out["d_w"] = d_w
    out["d_x"] = gather(d["d_rows"].double(), valid)
    return out
