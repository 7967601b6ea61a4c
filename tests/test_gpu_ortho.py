"""Orthogonalised updates on the GPU, against 64-bit forms."""
import pytest
import torch

from tests import ortho_reference as orf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


def handle(pkg, rows, cols, n=1, dtype="bf16", **kw):
    return pkg.Orthogonalizer(pkg.OrthoConfig(rows=rows, cols=cols, max_matrices=n, dtype=dtype, **kw))


SHAPES = [(1, 1), (1, 100), (100, 1), (2, 3), (5, 4), (16, 16), (31, 33), (33, 31), (32, 64), (64, 256), (127, 129), (128, 128),
          (130, 128), (129, 1000), (1000, 129), (255, 257), (300, 640), (640, 300), (512, 512), (777, 1999), (1999, 777),
          (1024, 1024), (2051, 1030), (1500, 4100), (4100, 2050)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_shapes(pkg, rows, cols, dtype):
    op = handle(pkg, rows, cols, dtype=dtype)
    g = orf.gradient(rows, cols, dtype, 1)
    orf.check(op(g), g, f"{rows} x {cols}")
    assert op.device_status() == 0 and op.last_launch_count() == (2 if rows * ((cols + 7) // 8) <= 4096 else 3)


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_one_step(pkg, rows, cols):
    """Before roundings part: near the 64-bit form with the kernels' roundings."""
    for kind in ("tokens", "few"):
        g = orf.gradient(rows, cols, "fp32", 9, kind)
        orf.check(handle(pkg, rows, cols, dtype="fp32", steps=1)(g), g, f"{rows} x {cols}", steps=1)


@pytest.mark.parametrize("kind", ["tokens", "few", "normal"])
@pytest.mark.parametrize("rows,cols", [(96, 400), (700, 300), (1100, 1100)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_kinds(pkg, kind, rows, cols, dtype):
    op = handle(pkg, rows, cols, dtype=dtype)
    g = orf.gradient(rows, cols, dtype, 2, kind)
    orf.check(op(g), g, kind)


@pytest.mark.parametrize("n,rows,cols", [(3, 130, 70), (20, 64, 300), (2, 513, 1030), (33, 40, 40), (5, 1024, 600), (19, 1000, 1100)])
def test_stacks(pkg, n, rows, cols):
    """A stack's matrices come out as each alone; fewer than the handle holds, too."""
    op, one = handle(pkg, rows, cols, n + 1, "fp32"), handle(pkg, rows, cols, 1, "fp32")
    g = orf.gradient(rows, cols, "fp32", 3, n=n)
    got = op(g)
    for i in range(n):
        orf.check(got[i], g[i], f"matrix {i}")
        alone = one(g[i])
        assert orf.distance(got[i], alone) <= orf.TWO
    for a, b in zip(op(g[:2]), got):
        assert orf.distance(a, b) <= orf.TWO
    assert op(g[:0]).shape == (0, rows, cols)
    assert torch.equal(op(g), got)          # the same again


@pytest.mark.parametrize("steps,coefficients", [(1, orf.MUON), (3, orf.MUON), (8, orf.MUON), (5, (1.5, -0.5, 0.0)), (4, (2.0, -1.5, 0.5))])
def test_steps_and_coefficients(pkg, steps, coefficients):
    op = handle(pkg, 200, 330, dtype="fp32", steps=steps, coefficients=coefficients)
    g = orf.gradient(200, 330, "fp32", 4, "normal")
    orf.check(op(g), g, "steps", steps=steps, coefficients=coefficients)


def test_it_orthogonalises(pkg):
    """Cubic steps to the end: X X^T = 1 up to the roundings of bf16 rows and fp16 steps."""
    op = handle(pkg, 96, 500, dtype="fp32", steps=30, coefficients=(1.5, -0.5, 0.0))
    x = op(orf.gradient(96, 500, "fp32", 5, "normal")).double()
    # an element of X X^T: off by two roundings of 2^-8 / sqrt(3) of unit rows, in random
    # directions (sqrt(2 / 500) of them, seven times that); the diagonal by twice 2^-8
    off = x @ x.T - torch.eye(96, device="cuda", dtype=torch.float64)
    assert off.abs().max() <= 2 * 2.0 ** -8 + 1e-3


@pytest.mark.parametrize("scale", [1e-41, 1e-30, 1e-18, 1e-3, 1e15, 1e34, 5e37])
def test_any_magnitude(pkg, scale):
    g = (orf.gradient(70, 90, "fp32", 6, "normal").double() * (scale * 1e3)).float()   # (1e-41: subnormal numbers)
    assert torch.isfinite(g).all()
    orf.check(handle(pkg, 70, 90, dtype="fp32", eps=0.0)(g), g, f"{scale}", eps=0.0)
    if scale < 1e-10:    # eps is far above the norm: what is left is small, and linear in the matrix
        got, want = handle(pkg, 70, 90, dtype="fp32")(g), orf.exact(g)
        # X's second fp16 term, 8 X here, ends at 2^-24: half of that is rounded away at the
        # start and in each step, and what is missing is multiplied by 3.4445 from there on
        lost = 2.0 ** -25 / 8 * sum(3.4445 ** i for i in range(6))
        assert (got.double() - want).abs().max() <= 2.0 ** -8 * want.abs().max() + lost


def test_one_large_element_among_zeros(pkg):
    """Rank one, its norm in one element; and the zero matrix."""
    op = handle(pkg, 300, 200, 2, "bf16")
    g = torch.zeros(2, 300, 200, dtype=torch.bfloat16, device="cuda")
    g[0, 217, 33] = -3.0
    got = op(g)
    x = 1.0
    for _ in range(5):
        x = 3.4445 * x - 4.775 * x ** 3 + 2.0315 * x ** 5
    assert abs(got[0, 217, 33].item() + x) <= 2.0 ** -8 * abs(x) + 2.0 ** -10
    got[0, 217, 33] = 0
    assert not got.any()


def test_values_that_are_not_finite_stay_in_their_matrix(pkg):
    op = handle(pkg, 140, 150, 3, "fp32")
    g = orf.gradient(140, 150, "fp32", 7, n=3)
    clean = op(g)
    for bad in (float("nan"), float("inf"), -float("inf")):
        g[1, 139, 2] = bad
        got = op(g)
        assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2]) and got[1].isnan().all()


@pytest.mark.parametrize("rows,cols", [(200, 96), (96, 200), (61, 45)])
def test_strided_matrices(pkg, rows, cols):
    """Column ranges of wide buffers, matrices beside each other, one matrix for all."""
    op = handle(pkg, rows, cols, 3, "bf16")
    g = orf.gradient(rows, cols, "bf16", 8, n=3)
    want = op(g)
    wide = torch.full((3, rows, cols + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :, 8:8 + cols] = g
    assert torch.equal(op(wide[:, :, 8:8 + cols]), want)
    odd = torch.zeros(3, rows, cols + 3, dtype=torch.bfloat16, device="cuda")
    odd[:, :, 1:1 + cols] = g
    assert torch.equal(op(odd[:, :, 1:1 + cols]), want)
    beside = torch.cat(list(g), dim=1).reshape(rows, 3, cols).transpose(0, 1)     # [3, rows, cols], rows 3 cols apart
    assert beside.stride(1) == 3 * cols and torch.equal(op(beside), want)
    same = op(g[1:2].expand(3, rows, cols))
    assert all(torch.equal(m, want[1]) for m in same)
    for pad, at in ((32, 16), (5, 3)):
        out = torch.full((3, rows + 1, cols + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        part = out[:, :rows, at:at + cols]
        assert op(g, out=part) is part and torch.equal(part, want)
        part.fill_(7)
        assert (out == 7).all()
    assert torch.equal(op(g[2]), want[2]) and op(g[2]).shape == (rows, cols)


def test_refusals(pkg):
    op = handle(pkg, 64, 96, 2, "bf16")
    g = orf.gradient(64, 96, "bf16", 0, n=2)
    buf = torch.zeros(3, 64, 96, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: op(g.float()), lambda: op(g[0].T), lambda: op(g[:, :63]), lambda: op(g.cpu()), lambda: op(buf),
                 lambda: op(g[0, 0]), lambda: op(g.transpose(1, 2).contiguous().transpose(1, 2)), lambda: op(g, out=g),
                 lambda: op(g, out=buf[:1]), lambda: op(g, out=buf[:2].half()), lambda: op(buf[:2], out=buf[1:]),
                 lambda: op(g, out=buf[:1].expand(2, 64, 96)), lambda: op(g[0, :1].expand(64, 96))):
        with pytest.raises(pkg.MoEError):
            call()
    want = op(g)
    torch.cuda.synchronize()
    lib = pkg.load_library()
    bad = [(g.data_ptr() + 1, 96, 6144, 2, buf.data_ptr(), 96, 6144), (g.data_ptr(), 95, 6144, 2, buf.data_ptr(), 96, 6144),
           (g.data_ptr(), 96, -6144, 2, buf.data_ptr(), 96, 6144), (g.data_ptr(), 96, 6144, 2, buf.data_ptr(), 96, 6143),
           (g.data_ptr(), 96, 6144, 3, buf.data_ptr(), 96, 6144), (g.data_ptr(), 96, 6144, -1, buf.data_ptr(), 96, 6144),
           (None, 96, 6144, 2, buf.data_ptr(), 96, 6144), (g.data_ptr(), 96, 6144, 2, None, 96, 6144)]
    for args in bad:
        assert lib.moe_ortho_forward(op.handle, *args, None) == 1, args
        assert lib.moe_ortho_last_error(op.handle)
    assert torch.equal(op(g), want)


@pytest.mark.parametrize("rows,cols", [(50, 80), (600, 520)])
def test_captured_and_replayed(pkg, rows, cols):
    op = handle(pkg, rows, cols, dtype="fp32")
    g = orf.gradient(rows, cols, "fp32", 1)
    op(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = op(g)
        twice = op(got.float())
    for seed in (2, 3):
        g.copy_(orf.gradient(rows, cols, "fp32", seed))
        graph.replay()
        torch.cuda.synchronize()
        want = op(g)
        assert torch.equal(got, want) and torch.equal(twice, op(want.float()))


def test_two_handles_on_two_streams(pkg):
    ops = [handle(pkg, 300, 900), handle(pkg, 900, 300)]
    g = [orf.gradient(300, 900, "bf16", 1), orf.gradient(900, 300, "bf16", 2)]
    want = [op(x) for op, x in zip(ops, g)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for op, s, x in zip(ops, streams, g):
            with torch.cuda.stream(s):
                got.append([op(x) for _ in range(3)])
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for gs, w in zip(got, want) for a in gs)


def test_large_matrices_beside_each_other_and_other_work(pkg):
    """Two handles whose CTAs fill the GPU, on two streams, and products of torch on a third: each
    launch waits until all of its CTAs are resident, none for the other's."""
    shapes = [(1500, 4100), (4100, 2050)]
    ops = [handle(pkg, *s) for s in shapes]
    g = [orf.gradient(*s, "bf16", i) for i, s in enumerate(shapes)]
    want = [op(x) for op, x in zip(ops, g)]
    a = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    with torch.cuda.stream(streams[2]):
        for _ in range(40):
            b = a @ a
    got = []
    for _ in range(6):
        for op, s, x in zip(ops, streams, g):
            with torch.cuda.stream(s):
                got.append(op(x))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])
    assert torch.isfinite(b).all() and all(op.device_status() == 0 for op in ops)


def test_inputs_of_a_given_stream_may_be_dropped(pkg):
    op = handle(pkg, 256, 512)
    g = orf.gradient(256, 512, "bf16", 1)
    want = op(g)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        mine = g.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = op.forward(mine, stream=stream)
        del mine
        over = [torch.full_like(g, float("nan")) for _ in range(3)]
        torch.cuda.synchronize()
        assert len(over) == 3 and torch.equal(got, want)


def test_offsets_past_32_bits(pkg):
    """2.2e9 elements in a stack: its last matrix comes out as alone."""
    n, side = 2100, 1024
    op, one = handle(pkg, side, side, n), handle(pkg, side, side)
    g = torch.randn(n, side, side, device="cuda", dtype=torch.bfloat16)
    got = op(g)
    for i in (0, n - 1):
        orf.check(got[i], g[i], f"matrix {i}")
        assert orf.distance(one(g[i]), got[i]) <= orf.TWO
    assert op.device_status() == 0


def test_a_failed_create_leaves_nothing(pkg):
    lib = pkg.load_library()
    live = lib.moe_debug_live_allocations()
    for n in range(1, 12):
        lib.moe_debug_fail_allocation(n)
        with pytest.raises(pkg.MoEError) as err:
            handle(pkg, 64, 64)
        assert err.value.status == 7 and lib.moe_debug_live_allocations() == live
    lib.moe_debug_fail_allocation(0)
    op = handle(pkg, 64, 64)
    assert lib.moe_debug_live_allocations() == live + 11
    op.close()
    assert lib.moe_debug_live_allocations() == live
