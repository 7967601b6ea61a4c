"""Every kind of plan of the orthogonalised update on the GPU: tiles of 128 x 128 and of 256 x 256 on
pairs, wide and tall, alone, stacked and in several groups, K split or not."""
import pytest
import torch

from tests import ortho_reference as orf
from tests.test_ortho_plans_host import SHAPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


def handle(pkg, rows, cols, n, **kw):
    return pkg.Orthogonalizer(pkg.OrthoConfig(rows=rows, cols=cols, max_matrices=n, dtype="bf16", **kw))


@pytest.mark.parametrize("rows,cols,n", SHAPES)
def test_plans(pkg, rows, cols, n):
    g = torch.stack([orf.gradient(rows, cols, "bf16", i, "normal" if i % 2 else "tokens") for i in range(min(n, 5))])
    g = g[torch.arange(n, device="cuda") % g.shape[0]].contiguous()
    looked_at = sorted({0, 1, n // 2, n - 1} & set(range(n)))
    one, five = handle(pkg, rows, cols, n, steps=1), handle(pkg, rows, cols, n)
    got = one(g)
    for i in looked_at:
        orf.check(got[i], g[i], f"matrix {i}, one step", steps=1)
    got = five(g)
    for i in looked_at:
        orf.check(got[i], g[i], f"matrix {i}")
    assert torch.equal(got, got[torch.arange(n, device="cuda") % min(n, 5)])
    for _ in range(3):
        assert torch.equal(five(g), got)
    assert one.device_status() == 0 and five.device_status() == 0


@pytest.mark.parametrize("rows,cols,n", [(7168, 2048, 1), (760, 9000, 2), (4000, 300, 4), (2100, 1100, 19)])
def test_plans_captured_with_fewer_matrices_between(pkg, rows, cols, n):
    """A graph of the full stack, replayed after calls of other sizes on the same handle: counters and
    partial sums of one call mean nothing to the next."""
    g = torch.stack([orf.gradient(rows, cols, "bf16", i) for i in range(min(n, 3))])
    g = g[torch.arange(n, device="cuda") % g.shape[0]].contiguous()
    op = handle(pkg, rows, cols, n)
    want, less = op(g).clone(), op(g[:1]).clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = op(g)
    for _ in range(3):
        assert torch.equal(op(g[:1]), less)
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert op.device_status() == 0
