"""A routed layer's experts trained with the operators together: tokens to the experts' rows, each
expert's gated block on its rows, back with weights; the gradients the same way; the
experts' weight gradients orthogonalised in one call.  Against 64 bits."""
import pytest
import torch

from tests import ops_reference as ref
from tests import ortho_reference as orf
from tests import rows_reference as rr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


def norm_of(err):
    return err.double().pow(2).sum().sqrt().item()


@pytest.mark.parametrize("act,dtype,drop", [("swiglu", "bf16", 0.0), ("relu2", "fp16", 0.1)])
def test_a_training_step_of_routed_experts(pkg, act, dtype, drop):
    T, k, E, K, N = 150, 3, 7, 128, 96
    dt, u = ref.DT[dtype], ref.unit(dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, e = normal(T, K).to(dt), normal(T, N).to(dt)
    ids = rr.make_ids(T, k, E - 1, 3, drop).cuda()     # (the last expert has no token)
    w = torch.rand(T, k, generator=gen, device="cuda")
    up = (normal(E, N, K) * K ** -0.5).to(dt)
    gate = (normal(E, N, K) * K ** -0.5).to(dt) if act == "swiglu" else None

    rows_op = pkg.ExpertRows(pkg.ExpertRowsConfig(n_experts=E, top_k=k, act_dtype=dtype, max_tokens=T))
    block = pkg.GatedBlock(pkg.GatedConfig(in_features=K, out_features=N, act=act, act_dtype=dtype, max_tokens=T * k, training=True))
    rows, plan = rows_op.dispatch(x, ids)
    bounds = plan.offsets.tolist()
    y, d_rows = torch.zeros(T * k, N, dtype=dt, device="cuda"), torch.zeros(T * k, K, dtype=dt, device="cuda")
    saved = []
    for i in range(E):
        a, b = bounds[i], bounds[i + 1]
        saved.append(block.forward_train(rows[a:b], up[i], None if gate is None else gate[i], out=y[a:b])[1])
    out = rows_op.combine(y, w, plan)
    d = rows_op.combine_backward(e, y, w, plan)
    d_up, d_gate = torch.empty_like(up), None if gate is None else torch.empty_like(gate)
    for i in range(E):
        a, b = bounds[i], bounds[i + 1]
        g = block.backward(d.y[a:b], saved[i], rows[a:b], up[i], None if gate is None else gate[i])
        d_rows[a:b] = g.x
        d_up[i] = g.up_w
        if gate is not None:
            d_gate[i] = g.gate_w
    d_x = rows_op.dispatch_backward(d_rows, plan)
    ortho = pkg.Orthogonalizer(pkg.OrthoConfig(rows=N, cols=K, max_matrices=E, dtype=dtype))
    update = ortho(d_up)

    # the same in 64 bits, with autograd
    x64, w64, up64 = (t.double().requires_grad_() for t in (x, w, up))
    gate64 = None if gate is None else gate.double().requires_grad_()
    here = (ids >= 0)
    hu = torch.einsum("tk,tjnk->tjn", x64, up64[ids.clamp(min=0)])
    if act == "swiglu":
        h = ref.silu(torch.einsum("tk,tjnk->tjn", x64, gate64[ids.clamp(min=0)])) * hu
    else:
        h = torch.clamp(hu, min=0) ** 2
    out64 = (h * (w64 * here)[:, :, None]).sum(1)
    out64.backward(e.double())
    # Norms: each result passes at most four roundings to 16 bits one after the other (the block's
    # output, the sum over experts, d_y, dg and du, the block's gradient, the sum of d_x), each
    # u / sqrt(3) of the norm of what it rounds; sums over picks have norms of at least 1 / sqrt(2) of
    # their terms' root mean square here (independent signs).  Six of them: 6 u.
    for got, want, what in ((out, out64, "out"), (d.w, w64.grad, "d_w"), (d_up, up64.grad, "d_up"), (d_x, x64.grad, "d_x")) + (
            () if gate is None else ((d_gate, gate64.grad, "d_gate"),)):
        assert norm_of(got.double() - want) <= 6 * u * norm_of(want), what
    assert not d_up[E - 1].any() and not update[E - 1].any() and (d.w[~here] == 0).all()
    for i in range(E - 1):
        orf.check(update[i], d_up[i], f"update {i}")
        # the update follows the gradient: <update, d_up> is the sum of singular values times about 1
        assert (update[i].double() * d_up[i].double()).sum() > 0.5 * torch.linalg.svdvals(d_up[i].double()).sum()
    for op in (rows_op, block, ortho):
        assert op.device_status() == 0


def test_the_layers_own_routing(pkg):
    """ids and weights as the layer gives them: its picks brought to rows and back are the tokens
    times the sum of their weights."""
    import moe_inputs as mi
    spec = mi.SPECS["tiny"]
    layer = pkg.MoELayer(pkg.MoEConfig.from_spec(spec, max_tokens=8), pkg.upload_arrays(mi.make_layer(spec, 0).arrays()))
    x = rr.rows(8, spec.hidden, "bf16", 0)
    _, ids, w, _ = layer.forward_ex(x)
    op = pkg.ExpertRows(pkg.ExpertRowsConfig(n_experts=spec.n_experts, top_k=spec.top_k, max_tokens=8))
    rows, plan = op.dispatch(x, ids)
    assert plan.offsets[-1].item() == 8 * spec.top_k
    want = x.double() * w.double().sum(1, keepdim=True)
    bound = (spec.top_k + 1) * 2.0 ** -24 * x.double().abs() * w.double().abs().sum(1, keepdim=True)
    ref.check(op.combine(rows, w, plan), want, bound, "bf16", "out")
    layer.close()
