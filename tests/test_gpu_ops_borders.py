"""4-bit calls on both sides of the border between the streaming kernel and the
tensor-core GEMM, which moves with the width of x, held to the model of the kernel
that runs and to mean-square bounds; streamed calls with several tiles a CTA."""
import pytest
import torch

from tests import ops_borders as ob
from tests import ops_reference as ref
from tests.test_gpu_ops import FORMATS, make_block, make_linear, rows, want_block

pytestmark = pytest.mark.gpu
IDS = [f"{f}{g}" for f, g in FORMATS]


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


def check(op, x, gate, up, bias, fmt, G, dtype, act):
    mats = 2 if gate is not None else 1
    xd = x.double()
    eu, mean = ob.bounds(x, up, fmt, G, dtype, mats)
    u = xd @ up.T
    g, eg = (xd @ gate.T, ob.bounds(x, gate, fmt, G, dtype, mats)[0]) if gate is not None else (u, eu)
    want, err = ref.activate(act, g, u), ref.act_bound(act, g, u, eg, eu)
    if bias is not None:
        want = want + bias.double()
        err = err + 2.0 ** -23 * want.abs()
    out = op(x)
    ref.check(out, want, err, dtype, act)
    if act == "none":
        ob.check_mean(out, want, mean, dtype, f"{fmt} T={x.shape[0]}")


@pytest.mark.parametrize("K", [4096, 6144, 8192, 14336, 65536])
@pytest.mark.parametrize("fmt,G", FORMATS, ids=IDS)
@pytest.mark.parametrize("act,dtype", [("none", "bf16"), ("none", "fp16"), ("swiglu", "bf16")])
def test_both_sides_of_the_border(pkg, act, dtype, fmt, G, K):
    N, mats = 123, 2 if act == "swiglu" else 1
    b = ob.most_streamed_rows(fmt, G, mats, K)
    op, gate, up, bias = make_linear(pkg, N, K, fmt, G, dtype, act, act == "none", b + 1, seed=K)
    scale = 2.0 ** -5 if act == "swiglu" else 2.0 ** -2   # wide sums: gates of order one
    for T in {1, max(b, 1), b + 1}:
        check(op, rows(T, K, dtype, T, scale=scale), gate, up, bias, fmt, G, dtype, act)
    assert op.device_status() == 0


@pytest.mark.parametrize("T", [1, 5, 16, 17, 48, 160])
@pytest.mark.parametrize("fmt,G", FORMATS, ids=IDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_mean_square_error(pkg, dtype, fmt, G, T):
    op, _, up, _ = make_linear(pkg, 777, 1280, fmt, G, dtype, "none", False, 160, seed=11)
    check(op, rows(T, 1280, dtype, T), None, up, None, fmt, G, dtype, "none")


@pytest.mark.parametrize("T", [1, 8, 9, 16])
@pytest.mark.parametrize("fmt,G", FORMATS, ids=IDS)
@pytest.mark.parametrize("act,dtype", [("swiglu", "bf16"), ("relu2", "fp16"), ("swiglu", "fp16")])
def test_streamed_gated_many_tiles_a_cta(pkg, act, dtype, fmt, G, T):
    op, gate, up, _ = make_linear(pkg, 7400, 448 if G == 64 else 384, fmt, G, dtype, act, False, 16, seed=2)
    x = rows(T, up.shape[1], dtype, T, scale=0.5)
    check(op, x, gate, up, None, fmt, G, dtype, act)
    first = op(x)
    assert all(torch.equal(first, op(x)) for _ in range(3))


@pytest.mark.parametrize("T", [1, 8, 9, 16])
@pytest.mark.parametrize("act", ["swiglu", "relu2"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_streamed_block_many_tiles_a_cta(pkg, dtype, act, T):
    op, x, up, gate, _ = make_block(pkg, T, 1288, 10008, dtype, act, True, seed=T)
    want, e, g, u, eg, eu = want_block(x, up, gate, dtype, act)
    out, saved = op.forward_train(x, up, gate)
    ref.check(out, want, e, dtype, "out")
    # the kept pre-activations are the fp32 sums themselves
    assert ((saved[1].double() - u).abs() <= eu + 2.0 ** -24 * u.abs()).all()
    if gate is not None:
        assert ((saved[0].double() - g).abs() <= eg + 2.0 ** -24 * g.abs()).all()
    assert torch.equal(out, op(x, up, gate))
