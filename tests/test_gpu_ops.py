"""The operators around the MoE layer on the GPU against their plain 64-bit
forms (bounds: ops_reference)."""
import numpy as np
import pytest
import torch

from tests import ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


def rows(T, K, dtype, seed, pad=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    wide = (torch.randn(max(T, 1), K + pad, generator=g) * scale).to(ref.DT[dtype]).cuda()
    return wide[:T, pad:]


def make_linear(pkg, N, K, fmt, G, dtype, act, bias, max_tokens, seed=0, sdt=None):
    sdt = sdt or dtype
    w, dense = ref.make_weight(N, K, fmt, G, sdt, seed)
    fields = {n: t.cuda() if t is not None else None for n, t in w.items()}
    gate = None
    if act == "swiglu":
        wg, gate = ref.make_weight(N, K, fmt, G, sdt, seed + 1)
        fields.update({"gate_" + n: t.cuda() if t is not None else None for n, t in wg.items()})
        gate = torch.from_numpy(gate).cuda()
    if bias:
        fields["bias"] = torch.linspace(-2, 2, N).to(ref.DT[dtype]).cuda()
    cfg = pkg.QLinearConfig(in_features=K, out_features=N, fmt=fmt, group_size=G, act_dtype=dtype, scale_dtype=sdt,
                            act=act, bias=bias, max_tokens=max_tokens)
    op = pkg.QLinear(cfg, fields)
    return op, gate, torch.from_numpy(dense).cuda(), fields.get("bias")


def want_linear(x, gate, up, bias, fmt, G, dtype, act):
    """(fp64 result, bound).  Up to 16 rows the affine codes carry an offset M (128
    in bf16, 64 in fp16) that cancels per group: products of magnitude (M + 15) s
    beside the weight's, s <= 0.01 here against a mean |w| of 0.02 or more, at most
    (143 * 0.01 + 1.35) / 0.02 = 140 times, over the group's G / 16 accumulations
    and three folding steps; above, each affine weight is rounded once."""
    xd = x.double()
    stream = x.shape[0] <= 16
    extra = 140.0 * (min(G, 64) / 16 + 3) if fmt == "affine" and stream else 0.0
    roundings = 1 if fmt == "affine" and not stream else 0
    u = xd @ up.T
    eu = ref.product_bound(xd, up, roundings, dtype, extra)
    g, eg = u, eu
    if act == "swiglu":
        g = xd @ gate.T
        eg = ref.product_bound(xd, gate, roundings, dtype, extra)
    h = ref.activate(act, g, u)
    e = ref.act_bound(act, g, u, eg, eu)
    if bias is not None:
        h = h + bias.double()
        e = e + 2.0 ** -23 * h.abs()
    return h, e


FORMATS = [("affine", 32), ("affine", 64), ("affine", 128), ("nvfp4", 16), ("mxfp4", 32)]


@pytest.mark.parametrize("T", [1, 2, 8, 9, 16, 17, 100, 129, 300])
@pytest.mark.parametrize("fmt,G", FORMATS, ids=[f"{f}{g}" for f, g in FORMATS])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_linear(pkg, fmt, G, dtype, T):
    N, K = 333, 640
    op, _, w, b = make_linear(pkg, N, K, fmt, G, dtype, "none", True, 300)
    x = rows(T, K, dtype, T, pad=8)
    want, e = want_linear(x, None, w, b, fmt, G, dtype, "none")
    ref.check(op(x), want, e, dtype, "linear")
    assert op.device_status() == 0


@pytest.mark.parametrize("T", [1, 5, 12, 40, 260])
@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("fmt,G", FORMATS, ids=[f"{f}{g}" for f, g in FORMATS])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_linear_gated(pkg, fmt, G, dtype, act, T):
    N, K = 200, 384
    op, gate, up, _ = make_linear(pkg, N, K, fmt, G, dtype, act, False, 260, seed=3)
    x = rows(T, K, dtype, T)
    want, e = want_linear(x, gate, up, None, fmt, G, dtype, act)
    ref.check(op(x), want, e, dtype, act)


@pytest.mark.parametrize("N,K,fmt,G", [(1, 32, "affine", 32), (7, 16, "nvfp4", 16), (17, 96, "mxfp4", 32),
                                       (4097, 2080, "affine", 32), (520, 1040, "nvfp4", 16), (16, 8192, "affine", 128),
                                       (64, 65536, "mxfp4", 32)])
@pytest.mark.parametrize("T", [1, 6, 16, 33])
def test_linear_odd_sizes(pkg, N, K, fmt, G, T):
    op, _, w, _ = make_linear(pkg, N, K, fmt, G, "bf16", "none", False, 64, seed=5)
    x = rows(T, K, "bf16", T)
    want, e = want_linear(x, None, w, None, fmt, G, "bf16", "none")
    ref.check(op(x), want, e, "bf16", "odd sizes")


def test_linear_other_scale_type(pkg):
    for dtype, sdt in (("bf16", "fp16"), ("fp16", "bf16")):
        op, _, w, _ = make_linear(pkg, 96, 256, "affine", 64, dtype, "none", False, 32, sdt=sdt)
        for T in (3, 32):
            x = rows(T, 256, dtype, T)
            want, e = want_linear(x, None, w, None, "affine", 64, dtype, "none")
            ref.check(op(x), want, e, dtype, "scale type")


@pytest.mark.parametrize("T", [3, 40])
def test_rows_and_columns_beyond_are_left(pkg, T):
    """Output rows behind the last one and the columns between the rows keep what they held."""
    N, K = 75, 128
    op, _, w, _ = make_linear(pkg, N, K, "affine", 64, "bf16", "none", False, 64)
    x = rows(T, K, "bf16", 1)
    buf = torch.full((T + 5, N + 6), 7.0, dtype=torch.bfloat16, device="cuda")
    op(x, out=buf[:T, 3:3 + N])
    want, e = want_linear(x, None, w, None, "affine", 64, "bf16", "none")
    ref.check(buf[:T, 3:3 + N], want, e, "bf16", "strided out")
    buf[:T, 3:3 + N] = 7.0
    assert (buf == 7.0).all()


def test_linear_empty_batch(pkg):
    op, _, _, _ = make_linear(pkg, 75, 128, "affine", 64, "bf16", "none", False, 64)
    assert op(rows(0, 128, "bf16", 0)).shape == (0, 75)
    assert op.last_launch_count() == 0


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("fmt,G", [("nvfp4", 16), ("mxfp4", 32)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_nan_scale_reaches_its_row_only(pkg, fmt, G, dtype, T):
    N, K = 40, 128
    w, dense = ref.make_weight(N, K, fmt, G, dtype, 1)
    w["s"][21, 3] = 127 if fmt == "nvfp4" else 255
    cfg = pkg.QLinearConfig(in_features=K, out_features=N, fmt=fmt, group_size=G, act_dtype=dtype, max_tokens=64)
    op = pkg.QLinear(cfg, {n: t.cuda() if t is not None else None for n, t in w.items()})
    x = rows(T, K, dtype, 2)
    out = op(x)
    assert torch.isnan(out[:, 21]).all()
    keep = [i for i in range(N) if i != 21]
    d = torch.from_numpy(dense).cuda()[keep]
    want, e = want_linear(x, None, d, None, fmt, G, dtype, "none")
    ref.check(out[:, keep], want, e, dtype, "other rows")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [2, 40])
def test_mxfp4_wide_exponents(pkg, dtype, T):
    """Rows whose block exponents lie far from each other's, and far apart inside a
    row: a block 2^-40 below its row's largest is below the result's last bit."""
    N, K = 32, 128
    w, _ = ref.make_weight(N, K, "mxfp4", 32, dtype, 1)
    s = torch.full((N, 4), 120, dtype=torch.uint8)
    s[:, 1] = torch.arange(N).to(torch.uint8) + 60           # rows with a small block
    s[3] = torch.tensor([30, 31, 33, 40], dtype=torch.uint8)  # a whole row far below the others
    s[4] = torch.tensor([140, 139, 100, 141], dtype=torch.uint8)
    w["s"] = s
    codes = (w["q"].numpy().view(np.uint32)[:, :, None] >> np.arange(0, 32, 4, dtype=np.uint32)) & 15
    dense = ref.E2M1[codes.reshape(N, K)] * np.exp2(s.numpy().astype(np.float64) - 127).repeat(32, 1)
    cfg = pkg.QLinearConfig(in_features=K, out_features=N, fmt="mxfp4", group_size=32, act_dtype=dtype, max_tokens=64)
    op = pkg.QLinear(cfg, {n: t.cuda() if t is not None else None for n, t in w.items()})
    x = rows(T, K, dtype, 2, scale=2.0 ** -6 if dtype == "fp16" else 1.0)
    d = torch.from_numpy(dense).cuda()
    want = x.double() @ d.T
    # (a flushed or rounded small block is off by less than 2^-24 of its row's largest weight)
    e = ref.product_bound(x.double(), d, 0, dtype) + 2.0 ** -24 * x.double().abs().sum(1, keepdim=True) * d.abs().amax(1)
    ref.check(op(x), want, e, dtype, "exponents")


def test_infinities_and_nan_in_x_stay_in_their_row(pkg):
    for T in (4, 40):
        op, gate, up, _ = make_linear(pkg, 64, 128, "nvfp4", 16, "bf16", "swiglu", False, 64)
        x = rows(T, 128, "bf16", 3).clone()
        x[1, 5] = float("inf")
        x[2, 7] = float("nan")
        out = op(x)
        assert torch.isnan(out[2]).all() and not torch.isfinite(out[1]).all()
        rest = [i for i in range(T) if i not in (1, 2)]
        want, e = want_linear(x[rest], gate, up, None, "nvfp4", 16, "bf16", "swiglu")
        ref.check(out[rest], want, e, "bf16", "other rows")


# ---------------------------------------------------------------------------
# gated block
# ---------------------------------------------------------------------------

def make_block(pkg, T, K, N, dtype, act, training, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    dt = ref.DT[dtype]
    up = (torch.randn(N, K, generator=g) * 0.05).to(dt).cuda()
    gate = (torch.randn(N, K, generator=g) * 0.05).to(dt).cuda() if act == "swiglu" else None
    e = (torch.randn(max(T, 1), N + pad, generator=g) * 0.1).to(dt).cuda()[:T, pad:]
    cfg = pkg.GatedConfig(in_features=K, out_features=N, act=act, act_dtype=dtype, max_tokens=max(T, 1),
                          training=training)
    return pkg.GatedBlock(cfg), rows(T, K, dtype, seed + 1, pad=pad), up, gate, e


def want_block(x, up, gate, dtype, act):
    xd, ud = x.double(), up.double()
    u, eu = xd @ ud.T, ref.product_bound(xd, ud, 0, dtype)
    g, eg = (xd @ gate.double().T, ref.product_bound(xd, gate.double(), 0, dtype)) if gate is not None else (u, eu)
    return ref.activate(act, g, u), ref.act_bound(act, g, u, eg, eu), g, u, eg, eu


def want_grads(x, up, gate, e, g, u, eg, eu, dtype, act):
    """Gradients and bounds: dg, du carry the pre-activations' errors (|silu'| <= 1.1,
    |silu''| <= 0.5), about ten fp32 steps and one 16-bit rounding each."""
    ed, xd = e.double(), x.double()
    if act == "swiglu":
        p = 1 / (1 + torch.exp(-g))
        s, d = g * p, p * (1 + g * (1 - p))
        du, dg = ed * s, ed * u * d
        edu = ed.abs() * 1.1 * eg + 16 * 2.0 ** -23 * (1 + g.abs()) * du.abs()
        edg = ed.abs() * (1.1 * eu + 0.5 * (u.abs() + eu) * eg) + 16 * 2.0 ** -23 * (1 + g.abs()) * (ed * u).abs()
        pairs = [("g", dg, edg, gate.double()), ("u", du, edu, up.double())]
    else:
        du = 2 * ed * torch.clamp(u, min=0)
        edu = 2 * ed.abs() * eu + 2.0 ** -22 * du.abs()
        pairs = [("u", du, edu, up.double())]
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0   # half a step of an fp16 subnormal dg or du
    out = {}
    dx, edx = 0, 0
    for n, d, ed_, w in pairs:
        dx = dx + d @ w
        edx = edx + ref.product_bound(d, w.T.contiguous(), 1, dtype) + (ed_ + tiny) @ w.abs()
        out["d_" + n] = (d.T @ xd, ref.product_bound(d.T.contiguous(), xd.T.contiguous(), 1, dtype) +
                         (ed_ + tiny).T @ xd.abs())
    out["x"] = (dx, edx)
    return out


@pytest.mark.parametrize("T,K,N", [(1, 64, 32), (1, 4096, 264), (5, 1000, 520), (16, 512, 256), (17, 512, 256),
                                   (48, 776, 1000), (130, 320, 200), (257, 128, 8), (300, 8, 1024), (600, 1032, 1304)])
@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_block_forward(pkg, T, K, N, act, dtype):
    op, x, up, gate, _ = make_block(pkg, T, K, N, dtype, act, False, pad=8)
    want, e, *_ = want_block(x, up, gate, dtype, act)
    ref.check(op(x, up, gate), want, e, dtype, "block")
    assert op.device_status() == 0


@pytest.mark.parametrize("T,K,N", [(1, 64, 32), (2, 2048, 264), (16, 512, 256), (24, 264, 520), (33, 520, 1000), (48, 72, 136),
                                   (49, 72, 136), (200, 320, 200), (257, 136, 72), (515, 1032, 776)])
@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_block_backward(pkg, T, K, N, act, dtype):
    op, x, up, gate, e = make_block(pkg, T, K, N, dtype, act, True, seed=T, pad=8)
    out, saved = op.forward_train(x, up, gate)
    want, err, g, u, eg, eu = want_block(x, up, gate, dtype, act)
    ref.check(out, want, err, dtype, "out")
    d = op.backward(e, saved, x, up, gate)
    grads = want_grads(x, up, gate, e, g, u, eg, eu, dtype, act)
    ref.check(d.x, *grads["x"], dtype, "d_x")
    ref.check(d.up_w, *grads["d_u"], dtype, "d_up_w")
    if gate is not None:
        ref.check(d.gate_w, *grads["d_g"], dtype, "d_gate_w")
    else:
        assert d.gate_w is None
    assert op.device_status() == 0


@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("T", [6, 70])
def test_block_gradients_against_differences(pkg, act, T):
    """d/ds of sum(e * out) along random directions of every input, by central
    differences of the 64-bit form: its own error is below 1e-6 of the terms'
    sum, the gradients' is the element bounds' sum of squares (independent
    roundings, seven deviations)."""
    op, x, up, gate, e = make_block(pkg, T, 136, 88, "bf16", act, True, seed=9)
    _, saved = op.forward_train(x, up, gate)
    d = op.backward(e, saved, x, up, gate)
    _, _, g, u, eg, eu = want_block(x, up, gate, "bf16", act)
    bounds = want_grads(x, up, gate, e, g, u, eg, eu, "bf16", act)

    def loss(xx, uu, gg):
        uo = xx @ uu.T
        return (e.double() * ref.activate(act, xx @ gg.T if gg is not None else uo, uo)).sum()

    gen = torch.Generator(device="cuda").manual_seed(0)
    base = {"x": x.double(), "up_w": up.double(), "gate_w": gate.double() if gate is not None else None}
    for name, key in (("x", "x"), ("up_w", "d_u"), ("gate_w", "d_g")):
        if base[name] is None:
            continue
        v = torch.randn(base[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-5
        plus, minus = ({**base, name: base[name] + s * h * v} for s in (1, -1))
        slope = (loss(plus["x"], plus["up_w"], plus["gate_w"]) -
                 loss(minus["x"], minus["up_w"], minus["gate_w"])) / (2 * h)
        got = (getattr(d, name).double() * v).sum()
        want, bound = bounds[key]
        el = (bound + ref.unit("bf16") * want.abs()) * v
        tol = 7 * torch.sqrt((el ** 2).sum()) + 1e-6 * (want * v).abs().sum()
        assert (got - slope).abs() <= tol, (name, got.item(), slope.item(), tol.item())


def test_block_asked_gradients_only(pkg):
    op, x, up, gate, e = make_block(pkg, 40, 128, 64, "bf16", "swiglu", True)
    _, saved = op.forward_train(x, up, gate)
    whole = op.backward(e, saved, x, up, gate)
    for need in (("x",), ("gate_w",), ("up_w",), ("x", "up_w"), ()):
        d = op.backward(e, saved, x, up, gate, need=need)
        for n in d._fields:
            if n in need:
                assert torch.equal(getattr(d, n), getattr(whole, n)), n
            else:
                assert getattr(d, n) is None


def test_block_empty_batch(pkg):
    op, x, up, gate, e = make_block(pkg, 0, 128, 64, "bf16", "swiglu", True)
    out, saved = op.forward_train(x, up, gate)
    assert out.shape == (0, 64)
    d = op.backward(e, saved, x, up, gate)
    assert d.x.shape == (0, 128) and not d.gate_w.any() and not d.up_w.any()


def test_block_all_clipped(pkg):
    """Every unit of a squared-ReLU block below zero: zero output and gradients."""
    op, x, up, _, e = make_block(pkg, 20, 64, 64, "bf16", "relu2", True)
    x, up = x.abs(), -up.abs()
    out, saved = op.forward_train(x, up)
    d = op.backward(e, saved, x, up)
    assert not out.any() and not d.x.any() and not d.up_w.any()


def test_block_saturated_gate(pkg):
    """Gates of +-200: exp over- and underflows; silu and its slope are at their limits."""
    op, x, up, gate, e = make_block(pkg, 20, 64, 64, "bf16", "swiglu", True)
    x = torch.ones_like(x)
    gate = torch.zeros_like(gate)
    gate[:32, :], gate[32:, :] = 200 / 64, -200 / 64
    out, saved = op.forward_train(x, up, gate)
    d = op.backward(e, saved, x, up, gate)
    assert not out[:, 32:].any() and not d.gate_w[32:].any() and not d.up_w[32:].any()
    want, err, g, u, eg, eu = want_block(x, up, gate, "bf16", "swiglu")
    ref.check(out, want, err, "bf16", "out")
    grads = want_grads(x, up, gate, e, g, u, eg, eu, "bf16", "swiglu")
    ref.check(d.x, *grads["x"], "bf16", "d_x")


# ---------------------------------------------------------------------------
# streams, graphs, handles, a run together
# ---------------------------------------------------------------------------

def test_same_call_same_bits(pkg):
    for T in (7, 60):
        op, x, up, gate, e = make_block(pkg, T, 512, 264, "bf16", "swiglu", True)
        first = None
        for _ in range(3):
            out, saved = op.forward_train(x, up, gate)
            got = (out, *op.backward(e, saved, x, up, gate))
            if first is not None:
                assert all(torch.equal(a, b) for a, b in zip(first, got))
            first = got


@pytest.mark.parametrize("T", [5, 60])
def test_captured_and_replayed(pkg, T):
    lin, _, _, _ = make_linear(pkg, 128, 264 // 8 * 64, "affine", 64, "bf16", "none", False, 64)
    op, x, up, gate, e = make_block(pkg, T, 512, 264 // 8 * 64, "bf16", "swiglu", True)
    x = x.contiguous()

    def step():
        h, saved = op.forward_train(x, up, gate)
        return (lin(h), *op.backward(e, saved, x, up, gate))

    want0 = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want0, got))
    x.copy_(rows(T, 512, "bf16", 77))
    want1 = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want1, got))
    assert not torch.equal(want0[0], want1[0])


def test_two_handles_on_two_streams(pkg):
    pairs = [make_linear(pkg, 512, 512, "nvfp4", 16, "bf16", "none", False, 64, seed=s) for s in (0, 5)]
    x = rows(64, 512, "bf16", 1)
    want = [p[0](x) for p in pairs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pairs]
    for _ in range(5):
        outs = [p[0].forward(x, stream=s) for p, s in zip(pairs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_dense_layer_then_moe_layer(pkg):
    """A run as a decoder uses them: a 16-bit gated block and its 4-bit down
    projection, a 4-bit gated block and its down projection, then an MoE layer."""
    import moe_inputs as mi
    import oracle
    spec = mi.SPECS["tiny"]
    H, F, T = spec.hidden, 384, 6
    block, x, up, gate, _ = make_block(pkg, T, H, F, "bf16", "swiglu", False)
    down, _, wd, _ = make_linear(pkg, H, F, "affine", 64, "bf16", "none", False, T, seed=1)
    gated4, g4, u4, _ = make_linear(pkg, F, H, "mxfp4", 32, "bf16", "swiglu", False, T, seed=2)
    down4, _, wd4, _ = make_linear(pkg, H, F, "nvfp4", 16, "bf16", "none", False, T, seed=4)
    layer = mi.make_layer(spec, 0)
    moe = pkg.MoELayer(pkg.MoEConfig.from_spec(spec, max_tokens=T), pkg.upload_arrays(layer.arrays()))
    h1 = block(x, up, gate)
    y1 = down(h1)
    h2 = gated4(y1)
    y2 = down4(h2)
    y2 = (y2.float() / y2.float().pow(2).mean(1, keepdim=True).sqrt()).to(torch.bfloat16)
    out, ids, _, _ = moe.forward_ex(y2)
    for got, (want, e) in ((h1, want_block(x, up, gate, "bf16", "swiglu")[:2]),
                           (y1, want_linear(h1, None, wd, None, "affine", 64, "bf16", "none")),
                           (h2, want_linear(y1, g4, u4, None, "mxfp4", 32, "bf16", "swiglu"))):
        ref.check(got, want, e, "bf16", "step")
    r = oracle.oracle_forward(layer, y2.cpu().view(torch.int16).numpy().view(np.uint16))
    err = out.double().cpu().numpy() - r["out"]
    assert np.sqrt(np.mean(err ** 2)) <= 1e-2 * np.sqrt(np.mean(r["out"] ** 2))


def test_creates_and_failures_leak_nothing(pkg):
    lib = pkg.load_library()
    before = lib.moe_debug_live_allocations()
    w, _ = ref.make_weight(64, 128, "nvfp4", 16, "bf16", 0)
    fields = {n: t.cuda() for n, t in w.items()}
    cfg = pkg.QLinearConfig(in_features=128, out_features=64, fmt="nvfp4", group_size=16, max_tokens=64)
    gcfg = pkg.GatedConfig(in_features=128, out_features=64, max_tokens=64, training=True)
    makers = (lambda: pkg.QLinear(cfg, fields), lambda: pkg.GatedBlock(gcfg))
    for make in makers:
        op = make()
        n = lib.moe_debug_live_allocations() - before
        assert n > 0 and op.device_bytes() > 0
        op.close()
        assert lib.moe_debug_live_allocations() == before
        for i in range(1, n + 1):
            lib.moe_debug_fail_allocation(i)
            try:
                with pytest.raises(pkg.MoEError) as err:
                    make()
            finally:
                lib.moe_debug_fail_allocation(0)
            assert err.value.status == 7
            assert lib.moe_debug_live_allocations() == before


def test_refusals_with_tensors(pkg):
    op, _, _, _ = make_linear(pkg, 72, 128, "affine", 64, "bf16", "none", False, 16)
    x = rows(4, 128, "bf16", 0)
    bad = [x.float(), x.half(), x.cpu(), x[:, :64], rows(17, 128, "bf16", 0), x.t().contiguous().t(),
           rows(4, 128, "bf16", 0, pad=4), x[0], x.expand(4, 128)[:1].expand(4, 128)]
    for b in bad:
        with pytest.raises(pkg.MoEError):
            op(b)
    with pytest.raises(pkg.MoEError):
        op(x, out=torch.empty(3, 72, dtype=torch.bfloat16, device="cuda"))
    wide = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
    wide[:4, :128] = x
    assert torch.equal(op(wide[:4, :128], out=wide[:4, 128:200]), op(x))   # columns of one buffer
    for o in (wide[:4, 127:199], wide[:4, 56:128], wide[1:5, 56:128]):
        with pytest.raises(pkg.MoEError):
            op(wide[:4, :128], out=o)
    block, x, up, gate, e = make_block(pkg, 20, 128, 64, "bf16", "swiglu", True)
    out, saved = block.forward_train(x, up, gate)
    for call in (lambda: block(x, up), lambda: block(x, up, gate.t().contiguous()),
                 lambda: block(x, up.float(), gate),
                 lambda: block.backward(e[:3], saved, x, up, gate),
                 lambda: block.backward(e, (saved[0], None), x, up, gate),
                 lambda: block.backward(e, saved, x, up, gate, need=("w",)),
                 lambda: block.backward(e, (saved[0].half(), saved[1]), x, up, gate)):
        with pytest.raises(pkg.MoEError):
            call()
    serving = make_block(pkg, 20, 128, 64, "bf16", "swiglu", False)[0]
    with pytest.raises(pkg.MoEError) as err:
        serving.backward(e, saved, x, up, gate)
    assert err.value.status == 2
    relu = make_block(pkg, 20, 128, 64, "bf16", "relu2", False)[0]
    with pytest.raises(pkg.MoEError):
        relu(x, up, gate)


def test_calls_between_other_kernels(pkg):
    """Inputs rewritten right before each call and outputs read right after, with
    nothing waited for: the chained launches start early but may not run ahead."""
    T = 7
    lin, _, _, _ = make_linear(pkg, 264, 512, "nvfp4", 16, "bf16", "none", False, 64, seed=2)
    many, _, _, _ = make_linear(pkg, 264, 512, "affine", 64, "bf16", "relu2", False, 64, seed=3)
    block, x, up, gate, e = make_block(pkg, T, 264, 512, "bf16", "swiglu", True)
    inputs = [(rows(T, 264, "bf16", 50 + i), torch.randn_like(up) * 0.05) for i in range(12)]

    def step(xi, wi):
        x.copy_(xi)
        up.copy_(wi)
        h, saved = block.forward_train(x, up, gate)
        d = block.backward(e, saved, x, up, gate)
        y = lin(h)
        wide = h.repeat(6, 1)
        z = many(wide)
        wide.zero_()      # after the call read it
        return [t.clone() for t in (h, *d, y, z)]

    x = x.contiguous()
    torch.cuda.synchronize()
    fast = [step(*i) for i in inputs]
    torch.cuda.synchronize()
    for i, got in zip(inputs, fast):
        want = step(*i)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("T", [5, 70])
def test_block_rows_and_columns_beyond_are_left(pkg, T):
    block, x, up, gate, _ = make_block(pkg, T, 128, 72, "bf16", "swiglu", False)
    for pad in (4, 13):   # rows aligned to 8 bytes, and odd ones
        buf = torch.full((T + 3, 72 + 2 * pad), 7.0, dtype=torch.bfloat16, device="cuda")
        block(x, up, gate, out=buf[:T, pad:pad + 72])
        want, e, *_ = want_block(x, up, gate, "bf16", "swiglu")
        ref.check(buf[:T, pad:pad + 72], want, e, "bf16", "strided out")
        buf[:T, pad:pad + 72] = 7.0
        assert (buf == 7.0).all()


def test_strided_gradient_of_the_output(pkg):
    """d_out as a column range, aligned and not."""
    for pad in (0, 8, 3):
        block, x, up, gate, e = make_block(pkg, 30, 128, 72, "bf16", "swiglu", True, seed=4)
        _, saved = block.forward_train(x, up, gate)
        want = block.backward(e, saved, x, up, gate)
        wide = torch.zeros(30, 72 + pad, dtype=torch.bfloat16, device="cuda")
        wide[:, pad:] = e
        got = block.backward(wide[:, pad:], saved, x, up, gate)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_offsets_past_32_bits(pkg):
    """70000 rows of 32768 outputs: 2.3 billion elements."""
    T, N = 70000, 32768
    some = torch.tensor([0, 1, 65535, 65536, T - 2, T - 1], device="cuda")
    op, _, w, _ = make_linear(pkg, N, 64, "affine", 64, "bf16", "none", False, T)
    x = torch.randn(T, 64, device="cuda", dtype=torch.bfloat16)
    out = op(x)
    xd = x[some].double()
    want = xd @ w.T
    ref.check(out[some], want, ref.product_bound(xd, w, 1, "bf16"), "bf16", "linear")
    del out, op
    block, _, up, _, _ = make_block(pkg, T, 64, N, "bf16", "relu2", True)
    out, saved = block.forward_train(x, up)
    wantb, err, g, u, eg, eu = want_block(x[some], up, None, "bf16", "relu2")
    ref.check(out[some], wantb, err, "bf16", "out")
    e = torch.randn(T, N, device="cuda", dtype=torch.bfloat16) * 0.1
    d = block.backward(e, saved, x, up)
    grads = want_grads(x[some], up, None, e[some], g, u, eg, eu, "bf16", "relu2")
    ref.check(d.x[some], *grads["x"], "bf16", "d_x")
    # the weights' gradient over all rows, for some of them
    ns = torch.tensor([0, 5, 32760, N - 1], device="cuda")
    uu = x.double() @ up[ns].double().T
    du = 2 * e[:, ns].double() * torch.clamp(uu, min=0)
    edu = 2 * e[:, ns].double().abs() * ref.product_bound(x.double(), up[ns].double(), 0, "bf16") + 2.0 ** -22 * du.abs()
    bound = ref.product_bound(du.T.contiguous(), x.double().T.contiguous(), 1, "bf16") + edu.T @ x.double().abs()
    ref.check(d.up_w[ns], du.T @ x.double(), bound, "bf16", "d_up_w")


def test_two_threads(pkg):
    """Handles of their own, streams of their own, calls at the same time."""
    import threading
    made = [make_block(pkg, 60, 256, 264, "bf16", "swiglu", True, seed=s) for s in (0, 1)]
    want = []
    for op, x, up, gate, e in made:
        out, saved = op.forward_train(x, up, gate)
        want.append((out, *op.backward(e, saved, x, up, gate)))
    torch.cuda.synchronize()
    bad = []

    def work(i):
        op, x, up, gate, e = made[i]
        stream = torch.cuda.Stream()
        for _ in range(20):
            with torch.cuda.stream(stream):
                out, saved = op.forward_train(x, up, gate)
                got = (out, *op.backward(e, saved, x, up, gate))
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
