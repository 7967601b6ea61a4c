"""Rows that begin at every place of a 16-byte word, of every small width and around a piece's 256
columns, with elements before, between and behind them that stay as they are."""
import pytest
import torch

from tests import rows_reference as rr

pytestmark = pytest.mark.gpu

T, K, E = 5, 3, 4
WIDTHS = [*range(1, 18), *range(247, 266), 511, 513, 769]
GUARD = 77.0


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


def place(n, H, shift, gap, values=None):
    """(buffer, rows): n rows of H that begin `shift` elements into a word, gap elements between them."""
    flat = torch.full((64 + n * (H + gap),), GUARD, dtype=torch.bfloat16, device="cuda")
    rows = torch.as_strided(flat, (n, H), (H + gap, 1), 16 + shift)
    assert rows.data_ptr() % 16 == 2 * shift
    if values is not None:
        rows.copy_(values)
    return flat, rows


def untouched(flat, rows):
    """Everything of the buffer but the rows."""
    mine = flat.clone()
    torch.as_strided(mine, rows.shape, rows.stride(), rows.storage_offset()).fill_(GUARD)
    return bool((mine == GUARD).all())


@pytest.mark.parametrize("shift", range(8))
@pytest.mark.parametrize("gap", [0, 3])
def test_rows_at_every_place(pkg, shift, gap):
    op = pkg.ExpertRows(pkg.ExpertRowsConfig(n_experts=E, top_k=K, act_dtype="bf16", max_tokens=400))
    ids = rr.make_ids(T, K, E, 1, 0.2)
    cpu = rr.plan(ids, E)
    p = tuple(t.cuda() for t in cpu)
    plan, ids = pkg.RowPlan(*p), ids.cuda()
    w = torch.rand(T, K, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") - 0.4
    for H in WIDTHS:
        x, y, e = rr.rows(T, H, "bf16", 3), rr.rows(T * K, H, "bf16", 4), rr.rows(T, H, "bf16", 5)
        other = (shift + 3) % 8
        xf, xs = place(T, H, other, gap + 1, x)
        yf, ys = place(T * K, H, other, gap + 1, y)
        for inputs in ((x, y, e), (xs, ys, None)):
            gx, gy, ge = inputs
            # to the rows: in one launch, and by a plan
            want = rr.take(x, p, K)
            for call in (lambda out: op.dispatch(gx, ids, out=out), lambda out: op.take(gx, plan, out=out)):
                flat, out = place(T * K, H, shift, gap)
                call(out)
                assert torch.equal(out, want) and untouched(flat, out), H
            # back, with weights and without
            for weights, call in ((w, lambda out: op.combine(gy, w, plan, out=out)),
                                  (None, lambda out: op.dispatch_backward(gy, plan, out=out))):
                flat, out = place(T, H, shift, gap)
                call(out)
                want, bound = rr.combine(y, weights, p)
                assert ((out.double() - want).abs() <= bound + 2.0 ** -8 * want.abs()).all() and untouched(flat, out), H
            # gradients: y and d_out read from every place
            ef, es = place(T, H, shift, gap, e)
            (d_y, by), (d_w, bw) = rr.combine_backward(e, y, w, p)
            got = op.combine_backward(es if ge is None else ge, gy, w, plan)
            assert ((got.y.double() - d_y).abs() <= by + 2.0 ** -8 * d_y.abs()).all(), H
            assert ((got.w.double() - d_w).abs() <= bw + 2.0 ** -24 * d_w.abs()).all(), H
        assert untouched(xf, xs) and untouched(yf, ys) and torch.equal(xs, x) and torch.equal(ys, y)
    assert op.device_status() == 0


@pytest.mark.parametrize("shift", range(8))
def test_gradient_rows_at_every_place(pkg, shift):
    """d_y by the C entry, into rows of any place; y and d_out from others."""
    op, lib = pkg.ExpertRows(pkg.ExpertRowsConfig(n_experts=E, top_k=K, act_dtype="bf16", max_tokens=T)), pkg.load_library()
    p = tuple(t.cuda() for t in rr.plan(rr.make_ids(T, K, E, 6, 0.2), E))
    w = torch.rand(T, K, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")
    for H in WIDTHS:
        y, e = rr.rows(T * K, H, "bf16", 8), rr.rows(T, H, "bf16", 9)
        (want, bound), (want_w, bound_w) = rr.combine_backward(e, y, w, p)
        ef, es = place(T, H, (shift + 5) % 8, 2, e)
        flat, out = place(T * K, H, shift, 1)
        d_w = torch.full((T, K), GUARD, device="cuda")
        s = torch.cuda.current_stream().cuda_stream
        status = lib.moe_rows_combine_backward(op.handle, es.data_ptr(), es.stride(0), T, H, y.data_ptr(), H, w.data_ptr(), 2, p[0].data_ptr(),
                                               p[2].data_ptr(), out.data_ptr(), out.stride(0), d_w.data_ptr(), s)
        assert status == 0
        assert ((out.double() - want).abs() <= bound + 2.0 ** -8 * want.abs()).all() and untouched(flat, out), H
        assert ((d_w.double() - want_w).abs() <= bound_w + 2.0 ** -24 * want_w.abs()).all(), H
    assert op.device_status() == 0
