"""Operators that a model puts around the MoE layer, as cases that can be timed.

Three operators, each in a plain form (elementary torch operations in fp32,
rounded once at the end) and as the library's own call:

  linear   out = x W^T (+ bias)                       4-bit weights W
  gated4   out = silu(x Wg^T) * (x Wu^T), or
           out = max(x Wu^T, 0)^2                      4-bit weights Wg, Wu
  block    the same two forms over 16-bit weights, forward alone (serving) or
           forward and backward (training: out, d_x, d_gate_w, d_up_w)

4-bit weights come in the library's three formats: affine codes with a scale
and a bias per group of 32, 64 or 128, NVFP4 (E2M1 codes, an E4M3 scale per 16,
one fp32 scale per matrix) and MXFP4 (E2M1 codes, an E8M0 scale per 32).

A case is a dict: `op`, `T` (token rows), `K` (input width), `N` (output
width), the formats, `act` and `pad` (x is a column range of a buffer that is
`pad` columns wider, as an output slice of a fused projection is).
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one decoded token through a latent output projection, quantised: the smallest
        # call, where latency counts
        dict(name="linear_t1_affine", op="linear", T=1, K=1024, N=4096, fmt="affine", G=64, dtype="bf16", act="none",
             bias=False, pad=0),
        # one decoded token through a large 4-bit gated block: a stream of weights
        dict(name="gated4_t1_nvfp4", op="gated4", T=1, K=4096, N=16384, fmt="nvfp4", G=16, dtype="bf16", act="swiglu",
             bias=False, pad=0),
        # a verification batch of drafted tokens through an attention output projection
        dict(name="linear_t5_mxfp4", op="linear", T=5, K=6144, N=6144, fmt="mxfp4", G=32, dtype="fp16", act="none",
             bias=True, pad=0),
        # sixteen streams decoded together through a squared-ReLU block, x a slice of a wider buffer
        dict(name="gated4_t16_affine", op="gated4", T=16, K=4096, N=3712, fmt="affine", G=32, dtype="bf16",
             act="relu2", bias=False, pad=64),
        # a ragged batch against an odd output width (a classifier or vocabulary slice)
        dict(name="linear_t77_odd", op="linear", T=77, K=1856, N=8191, fmt="affine", G=64, dtype="fp16", act="none",
             bias=True, pad=8),
        # a chunk of prefill mixed with decoding
        dict(name="gated4_t300_mxfp4", op="gated4", T=300, K=4096, N=8192, fmt="mxfp4", G=32, dtype="bf16",
             act="swiglu", bias=False, pad=0),
        # prefill
        dict(name="linear_t2048_affine", op="linear", T=2048, K=4096, N=16384, fmt="affine", G=128, dtype="bf16",
             act="none", bias=False, pad=0),
        # the shared expert's input half for one token, 16-bit weights
        dict(name="block_t1_relu2", op="block", T=1, K=4096, N=3712, dtype="bf16", act="relu2", train=False, pad=0),
        # a decode batch of 48 streams through a 16-bit gated block
        dict(name="block_t48_swiglu", op="block", T=48, K=6144, N=2048, dtype="fp16", act="swiglu", train=False, pad=0),
        # a small fine-tuning step: few tokens, so weights and weight gradients are most of the bytes
        dict(name="train_t9_swiglu", op="block", T=9, K=2048, N=5504, dtype="bf16", act="swiglu", train=True, pad=0),
        # a ragged training batch through the latent layer's shared expert
        dict(name="train_t333_relu2", op="block", T=333, K=4096, N=3712, dtype="fp16", act="relu2", train=True, pad=16),
        # a full training step's rows
        dict(name="train_t4096_swiglu", op="block", T=4096, K=4096, N=8192, dtype="bf16", act="swiglu", train=True, pad=0),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def _flops(c):
    per = 2 * c["T"] * c["K"] * c["N"] * (2 if c["act"] == "swiglu" else 1)
    return per * 3 if c.get("train") else per


def draw(rng):
    most = 2 * 2 * 3 * 4096 * 4096 * 8192
    while True:
        op = rng.choice(["linear", "gated4", "block", "block"])
        c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), pad=rng.choice([0, 0, 8, 72]))
        if op == "block":
            c["act"] = rng.choice(["swiglu", "swiglu", "relu2"])
            c["train"] = rng.random() < 0.5
            c["T"] = _log(rng, 1, 4096)
            c["K"] = 8 * _log(rng, 32, 768)
            c["N"] = 8 * _log(rng, 32, 1024)
        else:
            c["fmt"] = rng.choice(["affine", "affine", "nvfp4", "mxfp4"])
            c["G"] = {"affine": rng.choice([32, 64, 128]), "nvfp4": 16, "mxfp4": 32}[c["fmt"]]
            c["act"] = "none" if op == "linear" else rng.choice(["swiglu", "relu2"])
            c["bias"] = op == "linear" and rng.random() < 0.4
            c["T"] = _log(rng, 1, 2048)
            c["K"] = c["G"] * max(1, _log(rng, 256, 8192) // c["G"])
            c["N"] = _log(rng, 200, 16384)
        if _flops(c) <= (most if c.get("train") else most // 12):
            return c


def work(case):
    T, K, N = case["T"], case["K"], case["N"]
    n_mat = 2 if case["act"] == "swiglu" else 1
    io = 2 * T * K + 2 * T * N
    if case["op"] == "block":
        w = 2 * n_mat * K * N
        if case["train"]:
            # x, the weights and d_out read; out, d_x and the weights' gradients written
            return {"bytes": io + w + 2 * T * N + 2 * T * K + w, "flops": _flops(case)}
        return {"bytes": io + w, "flops": _flops(case)}
    per_group = {"affine": 4, "nvfp4": 1, "mxfp4": 1}[case["fmt"]]
    w = n_mat * (K * N // 2 + per_group * (K // case["G"]) * N) + (2 * N if case["bias"] else 0)
    return {"bytes": io + w, "flops": _flops(case)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _pack(codes):
    """[N, K] codes 0..15 -> int32 [N, K / 8], element 8 w + i in bits 4 i .. 4 i + 3 of word w."""
    c = codes.to(torch.int64).reshape(codes.shape[0], -1, 8)
    word = torch.zeros(c.shape[:2], dtype=torch.int64, device=c.device)
    for i in range(8):
        word |= c[:, :, i] << (4 * i)
    return torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32)


def _nearest_e2m1(v):
    edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    return torch.bucketize(v.abs(), edge) + 8 * (v < 0).to(torch.int64)


def _weight4(case, gen):
    """A normal matrix quantised to the case's format: {"q", "s", "b"}."""
    N, K, G = case["N"], case["K"], case["G"]
    w = torch.randn(N, K, generator=gen, device="cuda") * 0.02
    g = w.reshape(N, K // G, G)
    if case["fmt"] == "affine":
        dt = DTYPES[case["dtype"]]
        lo, hi = g.amin(2, keepdim=True), g.amax(2, keepdim=True)
        s, b = ((hi - lo) / 15).to(dt), lo.to(dt)
        q = torch.round((g - b.float()) / s.float()).clamp(0, 15)
        return {"q": _pack(q.reshape(N, K)), "s": s.reshape(N, -1).contiguous(), "b": b.reshape(N, -1).contiguous()}
    top = g.abs().amax(2, keepdim=True)
    if case["fmt"] == "nvfp4":
        scale = (w.abs().max() / (6 * 448)).reshape(1)
        s8 = (top / (6 * scale)).clamp(max=448).to(torch.float8_e4m3fn)
        real = s8.float() * scale
        q = _nearest_e2m1(g / torch.where(real > 0, real, torch.ones_like(real)))
        return {"q": _pack(q.reshape(N, K)), "s": s8.view(torch.uint8).reshape(N, -1).contiguous(), "b": scale.float()}
    e = torch.floor(torch.log2(top)) - 2
    q = _nearest_e2m1(g / torch.exp2(e))
    return {"q": _pack(q.reshape(N, K)), "s": (e + 127).to(torch.uint8).reshape(N, -1).contiguous(), "b": None}


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1_000_003 * (seed + 1) + case["T"] + 7 * case["K"] + 11 * case["N"])
    dt = DTYPES[case["dtype"]]
    T, K, N = case["T"], case["K"], case["N"]
    d = {"case": case}
    # activations after a norm: unit rows with a few channels several times larger
    wide = torch.randn(T, K + case["pad"], generator=gen, device="cuda")
    chan = torch.rand(K + case["pad"], generator=gen, device="cuda")
    wide = (wide * torch.where(chan < 0.01, 4.0, 1.0)).to(dt)
    d["x"] = wide[:, case["pad"]:]
    if case["op"] == "block":
        if case["act"] == "swiglu":
            d["gate_w"] = (torch.randn(N, K, generator=gen, device="cuda") * 0.02).to(dt)
        d["up_w"] = (torch.randn(N, K, generator=gen, device="cuda") * 0.02).to(dt)
        if case["train"]:
            d["d_out"] = (torch.randn(T, N, generator=gen, device="cuda") * 0.05).to(dt)
    else:
        if case["act"] == "swiglu":
            d["gate"] = _weight4(case, gen)
        d["up"] = _weight4(case, gen)
        d["bias"] = (torch.randn(N, generator=gen, device="cuda") * 0.1).to(dt) if case["bias"] else None
    return d


def prepare(case, seed):
    state = _inputs(case, seed)
    if own:
        import quantized_moe_decode_gemv_gb300 as pkg
        if case["op"] == "block":
            cfg = pkg.GatedConfig(in_features=case["K"], out_features=case["N"], act=case["act"],
                                  act_dtype=case["dtype"], max_tokens=case["T"], training=case["train"])
            state["block"] = pkg.GatedBlock(cfg)
        else:
            cfg = pkg.QLinearConfig(in_features=case["K"], out_features=case["N"], fmt=case["fmt"],
                                    group_size=case["G"], act_dtype=case["dtype"], scale_dtype=case["dtype"],
                                    act=case["act"], bias=case["bias"], max_tokens=case["T"])
            w = {n: state["up"][n] for n in ("q", "s", "b")}
            if case["act"] == "swiglu":
                w.update({"gate_" + n: state["gate"][n] for n in ("q", "s", "b")})
            w["bias"] = state["bias"]
            state = {"case": case, "x": state["x"], "linear": pkg.QLinear(cfg, w)}
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _codes(packed):
    shift = torch.arange(0, 32, 4, device=packed.device, dtype=torch.int32)
    return ((packed[:, :, None] >> shift) & 15).reshape(packed.shape[0], -1)


def _dequant(w, case):
    q = _codes(w["q"])
    N, K, G = case["N"], case["K"], case["G"]
    if case["fmt"] == "affine":
        return (q.float().reshape(N, K // G, G) * w["s"].float()[:, :, None] + w["b"].float()[:, :, None]).reshape(N, K)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    v = table[q.long()].reshape(N, K // G, G)
    if case["fmt"] == "nvfp4":
        s = w["s"].view(torch.float8_e4m3fn).float() * w["b"]
    else:
        s = torch.exp2(w["s"].float() - 127)
    return (v * s[:, :, None]).reshape(N, K)


def _plain(state):
    case, x = state["case"], state["x"].float()
    dt = DTYPES[case["dtype"]]
    if case["op"] != "block":
        u = x @ _dequant(state["up"], case).T
        if case["act"] == "swiglu":
            g = x @ _dequant(state["gate"], case).T
            u = g / (1 + torch.exp(-g)) * u
        elif case["act"] == "relu2":
            u = torch.clamp(u, min=0) ** 2
        if case["bias"]:
            u = u + state["bias"].float()
        return u.to(dt)
    up = state["up_w"].float()
    u = x @ up.T
    if case["act"] == "swiglu":
        gate = state["gate_w"].float()
        g = x @ gate.T
        sig = 1 / (1 + torch.exp(-g))
        h = g * sig * u
    else:
        h = torch.clamp(u, min=0) ** 2
    if not case["train"]:
        return h.to(dt)
    dh = state["d_out"].float()
    if case["act"] == "swiglu":
        du = dh * g * sig
        dg = dh * u * sig * (1 + g * (1 - sig))
        return {"out": h.to(dt), "d_x": (dg @ gate + du @ up).to(dt), "d_gate_w": (dg.T @ x).to(dt),
                "d_up_w": (du.T @ x).to(dt)}
    du = dh * 2 * torch.clamp(u, min=0)
    return {"out": h.to(dt), "d_x": (du @ up).to(dt), "d_up_w": (du.T @ x).to(dt)}


def run(state):
    if not own:
        return _plain(state)
    case = state["case"]
    if case["op"] != "block":
        return state["linear"](state["x"])
    block, x, gate_w, up_w = state["block"], state["x"], state.get("gate_w"), state["up_w"]
    if not case["train"]:
        return block(x, up_w, gate_w)
    out, saved = block.forward_train(x, up_w, gate_w)
    d = block.backward(state["d_out"], saved, x, up_w, gate_w)
    if case["act"] == "swiglu":
        return {"out": out, "d_x": d.x, "d_gate_w": d.gate_w, "d_up_w": d.up_w}
    return {"out": out, "d_x": d.x, "d_up_w": d.up_w}


# ---------------------------------------------------------------------------
# from the definition, in 64 bits
# ---------------------------------------------------------------------------

def _value_table(fmt):
    """The value of every code, by its bits: sign, two exponent bits (bias 1), one mantissa bit."""
    if fmt == "affine":
        return np.arange(16, dtype=np.float64)
    out = np.zeros(16)
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        mag = m * 0.5 if e == 0 else (1 + 0.5 * m) * 2.0 ** (e - 1)
        out[c] = -mag if c & 8 else mag
    return out


def _e4m3_table():
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = math.nan if (c & 127) == 127 else (-mag if c & 128 else mag)
    return out


def _matrix64(w, case):
    N, K, G = case["N"], case["K"], case["G"]
    by = w["q"].contiguous().view(torch.uint8).reshape(N, K // 2)
    table = torch.from_numpy(_value_table(case["fmt"])).cuda()
    m = torch.empty(N, K, dtype=torch.float64, device="cuda")
    m[:, 0::2] = table[(by % 16).long()]
    m[:, 1::2] = table[(by // 16).long()]
    if case["fmt"] == "affine":
        s, b = w["s"].double(), w["b"].double()
    elif case["fmt"] == "nvfp4":
        s, b = torch.from_numpy(_e4m3_table()).cuda()[w["s"].long()] * w["b"].double(), None
    else:
        s, b = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), w["s"].to(torch.int32) - 127), None
    for j in range(G):
        m[:, j::G] *= s
        if b is not None:
            m[:, j::G] += b
    return m


def exact(case, seed):
    d = _inputs(case, seed)
    x = d["x"].double()
    swiglu = case["act"] == "swiglu"
    if case["op"] == "block":
        wu = d["up_w"].double()
        wg = d["gate_w"].double() if swiglu else None
    else:
        wu = _matrix64(d["up"], case)
        wg = _matrix64(d["gate"], case) if swiglu else None
    u = torch.einsum("tk,nk->tn", x, wu)
    if swiglu:
        g = torch.einsum("tk,nk->tn", x, wg)
        p = torch.sigmoid(g)
        h = u * (g * p)
    elif case["act"] == "relu2":
        h = torch.where(u > 0, u * u, torch.zeros_like(u))
    else:
        h = u
    if case.get("bias"):
        h = h + d["bias"].double()
    if not case.get("train"):
        return h
    e = d["d_out"].double()
    if swiglu:
        du = e * (g * p)
        dg = e * u * (p + g * p * (1 - p))
        return {"out": h, "d_x": torch.einsum("tn,nk->tk", dg, wg) + torch.einsum("tn,nk->tk", du, wu),
                "d_gate_w": torch.einsum("tn,tk->nk", dg, x), "d_up_w": torch.einsum("tn,tk->nk", du, x)}
    du = torch.where(u > 0, 2 * u * e, torch.zeros_like(u))
    return {"out": h, "d_x": torch.einsum("tn,nk->tk", du, wu), "d_up_w": torch.einsum("tn,tk->nk", du, x)}
