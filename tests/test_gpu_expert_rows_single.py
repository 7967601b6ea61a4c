"""One token's rows beside others in one buffer: a single row has no stride of its own, and meets nothing
that lies in other columns."""
import pytest
import torch

from tests import rows_reference as rr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


@pytest.mark.parametrize("H", [64, 33])
@pytest.mark.parametrize("row", [0, 1, 2])
def test_column_ranges_of_one_buffer(pkg, H, row):
    k, E = 3, 5
    op = pkg.ExpertRows(pkg.ExpertRowsConfig(n_experts=E, top_k=k, act_dtype="bf16", max_tokens=4))
    ids = torch.tensor([[4, 0, 2]])
    p = tuple(t.cuda() for t in rr.plan(ids, E))
    plan, w = pkg.RowPlan(*p), torch.rand(1, k, device="cuda")
    wide = torch.full((k, 4 * H), 7.0, dtype=torch.bfloat16, device="cuda")
    x, rows, out, d_x = (wide[row:row + 1, :H], wide[:, H:2 * H], wide[row:row + 1, 2 * H:3 * H], wide[row:row + 1, 3 * H:])
    x.copy_(rr.rows(1, H, "bf16", 1))
    want = rr.take(x, p, k)
    op.dispatch(x, ids.cuda(), out=rows)
    assert torch.equal(rows, want)
    rows.fill_(7)
    op.take(x, plan, out=rows)
    assert torch.equal(rows, want)
    op.combine(rows, w, plan, out=out)
    want, bound = rr.combine(rows, w, p)
    assert ((out.double() - want).abs() <= bound + 2.0 ** -8 * want.abs()).all()
    op.dispatch_backward(rows, plan, out=d_x)
    want, bound = rr.combine(rows, None, p)
    assert ((d_x.double() - want).abs() <= bound + 2.0 ** -8 * want.abs()).all()
    rest = torch.ones_like(wide, dtype=torch.bool)
    rest[:, H:2 * H] = False
    rest[row] = False
    assert (wide[rest] == 7).all() and op.device_status() == 0


def test_rows_that_do_meet_are_refused(pkg):
    """The same row, one that begins inside another's columns, one that reaches into the next row's."""
    k, E, H = 3, 5, 64
    op = pkg.ExpertRows(pkg.ExpertRowsConfig(n_experts=E, top_k=k, act_dtype="bf16", max_tokens=4))
    ids = torch.tensor([[4, 0, 2]], device="cuda")
    wide = torch.zeros(k, 3 * H, dtype=torch.bfloat16, device="cuda")
    flat, rows = wide.view(-1), wide[:, H:2 * H]
    plan = op.plan(ids)
    for at in (3 * H + H, 3 * H + H - 8, 3 * H + H + 8, 3 * H + 2 * H - 1, H - 1 + 1):
        x = flat[at:at + H].view(1, H)
        for call in (lambda: op.dispatch(x, ids, out=rows), lambda: op.take(x, plan, out=rows), lambda: op.dispatch_backward(rows, plan, out=x)):
            with pytest.raises(pkg.MoEError):
                call()
    for at in (0, 2 * H, 3 * H, 5 * H, 5 * H + H):       # beside them: 5 H to 6 H, and its wrap to the next row's first columns
        x = flat[at:at + H].view(1, H)
        op.take(x, plan, out=rows)
    assert op.device_status() == 0
