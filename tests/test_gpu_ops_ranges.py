"""Values at the ends of the operators' ranges."""
import pytest
import torch

from tests import ops_reference as ref
from tests.test_gpu_ops import FORMATS, make_block, make_linear, rows, want_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


@pytest.mark.parametrize("dtype,top,apart", [("bf16", 240, 110), ("fp16", 150, 24)])
@pytest.mark.parametrize("T", [4, 40])
def test_mxfp4_blocks_far_below_their_rows_largest(pkg, dtype, top, apart, T):
    """At the distance that is kept whole, and where x leaves only the small blocks."""
    N, K = 48, 256
    w, _ = ref.make_weight(N, K, "mxfp4", 32, dtype, 1)
    s = torch.full((N, K // 32), top - apart, dtype=torch.uint8)
    s[:, 0] = top
    w["s"] = s
    codes = (w["q"].to(torch.int64)[:, :, None] >> torch.arange(0, 32, 4)) & 15
    dense = (torch.from_numpy(ref.E2M1)[codes.reshape(N, K)] *
             torch.exp2(s.double() - 127).repeat_interleave(32, 1)).cuda()
    op = pkg.QLinear(pkg.QLinearConfig(in_features=K, out_features=N, fmt="mxfp4", group_size=32, act_dtype=dtype,
                                       max_tokens=64), {n: t.cuda() if t is not None else None for n, t in w.items()})
    x = rows(T, K, dtype, 2).clone()
    x[:, :32] = 0
    want, e = want_linear(x, None, dense, None, "mxfp4", 32, dtype, "none")
    ref.check(op(x), want, e, dtype, "small blocks")


@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** -100])
@pytest.mark.parametrize("T", [4, 40])
@pytest.mark.parametrize("fmt,G", FORMATS, ids=[f"{f}{g}" for f, g in FORMATS])
def test_large_and_small_rows(pkg, fmt, G, T, scale):
    op, _, w, _ = make_linear(pkg, 96, 512, fmt, G, "bf16", "none", False, 64, seed=6)
    x = rows(T, 512, "bf16", 4, scale=scale)
    want, e = want_linear(x, None, w, None, fmt, G, "bf16", "none")
    ref.check(op(x), want, e, "bf16", "range")


def test_no_graph_is_recorded(pkg):
    """The operators are no autograd functions: inputs that require gradients are taken
    as they are, outputs carry no graph, and nobody's .grad is touched."""
    op, _, _, _ = make_linear(pkg, 64, 128, "affine", 64, "bf16", "none", False, 32)
    block, x, up, gate, e = make_block(pkg, 20, 128, 64, "bf16", "swiglu", True)
    plain = block.forward_train(x, up, gate)
    x, up, gate = (t.detach().clone().requires_grad_() for t in (x, up, gate))
    out, saved = block.forward_train(x, up, gate)
    d = block.backward(e, saved, x, up, gate)
    y = op(x)
    for t in (out, *saved, *d, y):
        assert not t.requires_grad and t.grad_fn is None
    assert x.grad is None and up.grad is None and gate.grad is None
    assert torch.equal(out, plain[0])
