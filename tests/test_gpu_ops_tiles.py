"""The tensor-core kernels of the operators with several tiles a CTA (persistent
CTAs that carry their rings and accumulators from one tile to the next), against
the plain 64-bit forms, and call after call with the same bits."""
import pytest
import torch

from tests import ops_reference as ref
from tests.test_gpu_ops import make_block, rows, want_block, want_grads

pytestmark = pytest.mark.gpu

SMS = 152


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


def weight(N, K, fmt, G, dtype, seed):
    """Random codes and scales made on the GPU: (fields, fp64 matrix)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.int64)
    word = sum(codes[:, i::8] << (4 * i) for i in range(8))
    q = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32)
    if fmt == "affine":
        s = (0.005 * (1 + torch.rand(N, K // G, generator=g, device="cuda"))).to(ref.DT[dtype])
        b = (-0.04 - 0.03 * torch.rand(N, K // G, generator=g, device="cuda")).to(ref.DT[dtype])
        dense = codes.double() * s.double().repeat_interleave(G, 1) + b.double().repeat_interleave(G, 1)
        return {"q": q, "s": s, "b": b}, dense
    table = torch.from_numpy(ref.E2M1).cuda()
    if fmt == "nvfp4":
        s = torch.randint(40, 64, (N, K // G), generator=g, device="cuda", dtype=torch.int64)
        b = torch.tensor([0.013], device="cuda")
        dense = table[codes] * (torch.from_numpy(ref.E4M3).cuda()[s] * b.double()).repeat_interleave(G, 1)
        return {"q": q, "s": s.to(torch.uint8), "b": b}, dense
    s = torch.randint(116, 122, (N, K // G), generator=g, device="cuda", dtype=torch.int64)
    return {"q": q, "s": s.to(torch.uint8), "b": None}, table[codes] * torch.exp2(s.double() - 127).repeat_interleave(G, 1)


def linear(pkg, N, K, fmt, G, dtype, act, T, seed=0):
    w, up = weight(N, K, fmt, G, dtype, seed)
    gate = None
    if act == "swiglu":
        wg, gate = weight(N, K, fmt, G, dtype, seed + 1)
        w.update({"gate_" + n: t for n, t in wg.items()})
    cfg = pkg.QLinearConfig(in_features=K, out_features=N, fmt=fmt, group_size=G, act_dtype=dtype, scale_dtype=dtype,
                            act=act, max_tokens=T)
    return pkg.QLinear(cfg, w), gate, up


def check_linear(op, x, gate, up, fmt, dtype, act):
    """More rows than the stream takes: an affine weight is rounded once."""
    xd, r = x.double(), 1 if fmt == "affine" else 0
    u, eu = xd @ up.T, ref.product_bound(xd, up, r, dtype)
    g, eg = (xd @ gate.T, ref.product_bound(xd, gate, r, dtype)) if gate is not None else (u, eu)
    out = op(x)
    ref.check(out, ref.activate(act, g, u), ref.act_bound(act, g, u, eg, eu), dtype, act)
    for _ in range(3):
        assert torch.equal(out, op(x)), "another call, other bits"
    assert op.device_status() == 0


# K in 64-wide blocks: 28 to 31, every remainder of four (the last of 1888 half full)
FORMS = [("affine", 64, 1792), ("affine", 64, 1856), ("affine", 64, 1920), ("affine", 64, 1984), ("affine", 32, 1888),
         ("affine", 128, 1920), ("nvfp4", 16, 1856), ("nvfp4", 16, 1920), ("mxfp4", 32, 1920), ("mxfp4", 32, 1856)]


@pytest.mark.parametrize("T", [160, 208, 240, 256, 512, 2048])
@pytest.mark.parametrize("fmt,G,K", FORMS, ids=[f"{f}{g}-{k}" for f, g, k in FORMS])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_many_tiles_a_cta(pkg, act, fmt, G, K, T):
    N = 128 * (2 * SMS + 1) // ((T + 255) // 256) + 77   # two tiles a CTA and more, the last one ragged
    op, gate, up = linear(pkg, N, K, fmt, G, "bf16", act, T)
    check_linear(op, rows(T, K, "bf16", T), gate, up, fmt, "bf16", act)


@pytest.mark.parametrize("fmt,G,K,T", [("affine", 64, 1920, 256), ("affine", 64, 1856, 224), ("nvfp4", 16, 1904, 250),
                                       ("mxfp4", 32, 1920, 192), ("affine", 32, 1888, 210)])
def test_linear_relu2_fp16_many_tiles_a_cta(pkg, fmt, G, K, T):
    N = 128 * (2 * SMS + 1) + 5
    op, gate, up = linear(pkg, N, K, fmt, G, "fp16", "relu2", T, seed=7)
    check_linear(op, rows(T, K, "fp16", T, scale=0.25), gate, up, fmt, "fp16", "relu2")


@pytest.mark.parametrize("act,N,K,T", [("none", 4100, 128, 3000), ("swiglu", 4100, 64, 3000), ("relu2", 4100, 192, 3000),
                                       ("none", 4100, 320, 2999)])
def test_linear_short_products_many_tiles_a_cta(pkg, act, N, K, T):
    """One to five K blocks a tile: a decode group may have none or one pair of them."""
    op, gate, up = linear(pkg, N, K, "affine", 64, "bf16", act, T, seed=3)
    check_linear(op, rows(T, K, "bf16", 5), gate, up, "affine", "bf16", act)


@pytest.mark.parametrize("T,K,N", [(2048, 1032, 5504), (700, 264, 20000), (5000, 136, 1032)])
@pytest.mark.parametrize("act", ["swiglu", "relu2"])
def test_block_many_tiles_a_pair(pkg, act, T, K, N):
    op, x, up, gate, e = make_block(pkg, T, K, N, "bf16", act, True, seed=T)
    out, saved = op.forward_train(x, up, gate)
    want, err, g, u, eg, eu = want_block(x, up, gate, "bf16", act)
    ref.check(out, want, err, "bf16", "out")
    d = op.backward(e, saved, x, up, gate)
    grads = want_grads(x, up, gate, e, g, u, eg, eu, "bf16", act)
    ref.check(d.x, *grads["x"], "bf16", "d_x")
    ref.check(d.up_w, *grads["d_u"], "bf16", "d_up_w")
    if gate is not None:
        ref.check(d.gate_w, *grads["d_g"], "bf16", "d_gate_w")
    again, saved2 = op.forward_train(x, up, gate)
    d2 = op.backward(e, saved2, x, up, gate)
    assert torch.equal(out, again) and all(torch.equal(a, b) for a, b in zip(d, d2) if a is not None)
    assert op.device_status() == 0


@pytest.mark.parametrize("act,fmt,G,T,N,K", [("none", "affine", 64, 17, 7982, 4096), ("swiglu", "nvfp4", 16, 17, 7982, 4096),
                                             ("none", "mxfp4", 32, 40, 9976, 5760)])
def test_linear_split_and_many_units_a_cta(pkg, act, fmt, G, T, N, K):
    """Few rows: K divided over more units than there are CTAs, of unequal lengths."""
    op, gate, up = linear(pkg, N, K, fmt, G, "bf16", act, T, seed=5)
    check_linear(op, rows(T, K, "bf16", 1), gate, up, fmt, "bf16", act)
    assert op.last_launch_count() == 2   # the product and the join of its K splits
