"""Tokens sorted by expert and back on the GPU, against 64-bit forms written pick by pick."""
import pytest
import torch

from tests import ops_reference as ref
from tests import rows_reference as rr

pytestmark = pytest.mark.gpu

CASES = [
    # T, k, E, H, dtype, drop, pad
    (1, 1, 1, 8, "bf16", 0.0, 0), (1, 9, 496, 1024, "bf16", 0.0, 0), (1, 16, 16, 24, "fp16", 0.0, 0),
    (2, 3, 5, 1, "bf16", 0.0, 0), (5, 4, 7, 7, "fp16", 0.2, 0), (33, 8, 1024, 130, "bf16", 0.1, 2),
    (77, 6, 130, 1001, "fp16", 0.1, 0), (300, 2, 3, 64, "bf16", 0.5, 8), (300, 10, 60, 520, "fp16", 0.0, 8),
    (455, 9, 496, 1024, "bf16", 0.03, 64), (456, 9, 31, 40, "bf16", 0.0, 3), (1025, 4, 1024, 16, "bf16", 0.05, 0),
    (3001, 7, 257, 72, "fp16", 0.02, 0), (20000, 9, 496, 8, "bf16", 0.01, 0), (40, 5, 9, 4104, "bf16", 0.3, 0),
    (600, 3, 8, 8200, "fp16", 0.0, 0), (16, 2, 1, 32, "bf16", 0.0, 0),
    (128, 8, 40, 48, "bf16", 0.1, 0), (129, 8, 1024, 48, "bf16", 0.1, 0), (16384, 8, 77, 16, "fp16", 0.02, 0),
    (16385, 8, 1000, 16, "bf16", 0.1, 0), (100, 16, 64, 2056, "bf16", 0.05, 8), (700, 16, 20, 520, "fp16", 0.0, 0),
    (200, 3, 12, 1, "fp16", 0.2, 0), (300, 4, 12, 255, "bf16", 0.3, 1), (300, 4, 12, 257, "fp16", 0.3, 2), (330, 9, 50, 2049, "bf16", 0.1, 5),
    (90, 5, 12, 4097, "fp16", 0.3, 0),
]


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


def handle(pkg, T, k, E, dtype):
    return pkg.ExpertRows(pkg.ExpertRowsConfig(n_experts=E, top_k=min(k, E), act_dtype=dtype, max_tokens=max(T, 1)))


def case(T, k, E, H, dtype, drop, pad, seed=0):
    k = min(k, E)
    ids = rr.make_ids(T, k, E, seed, drop)
    return k, ids, rr.plan(ids, E)


def on_gpu(p):
    return tuple(t.cuda() for t in p)


@pytest.mark.parametrize("T,k,E,H,dtype,drop,pad", CASES)
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
def test_dispatch(pkg, T, k, E, H, dtype, drop, pad, id_type):
    op = handle(pkg, T, k, E, dtype)
    k, ids, p = case(T, k, E, H, dtype, drop, pad)
    ids = ids.to(id_type).cuda()
    x = rr.rows(T, H, dtype, 1, pad)
    alone = op.plan(ids)
    got, plan = op.dispatch(x, ids)
    assert all(torch.equal(a, b.cuda()) for a, b in zip(plan, p))
    assert all(torch.equal(a, b) for a, b in zip(plan, alone))
    want = rr.take(x, on_gpu(p), k)
    assert torch.equal(got, want)
    assert torch.equal(op.take(x, plan), want)
    assert op.device_status() == 0


@pytest.mark.parametrize("T,k,E,H,dtype,drop,pad", CASES)
@pytest.mark.parametrize("w_type", ["fp32", "own"])
def test_combine_and_gradients(pkg, T, k, E, H, dtype, drop, pad, w_type):
    op = handle(pkg, T, k, E, dtype)
    k, ids, p = case(T, k, E, H, dtype, drop, pad, seed=2)
    p = on_gpu(p)
    plan = pkg.RowPlan(*p)
    y, e = rr.rows(T * k, H, dtype, 3, pad), rr.rows(T, H, dtype, 4, pad)
    w = torch.rand(T, k, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda") - 0.3
    if w_type == "own":
        w = w.to(ref.DT[dtype])
    want, bound = rr.combine(y, w, p)
    ref.check(op.combine(y, w, plan), want, bound, dtype, "out")
    want, bound = rr.combine(y, None, p)
    ref.check(op.dispatch_backward(y, plan), want, bound, dtype, "d_x")
    (d_y, by), (d_w, bw) = rr.combine_backward(e, y, w, p)
    got = op.combine_backward(e, y, w, plan)
    ref.check(got.y, d_y, by, dtype, "d_y")
    if w_type == "own":
        ref.check(got.w, d_w, bw, dtype, "d_w")
    else:
        assert ((got.w.double() - d_w).abs() <= bw + 2.0 ** -24 * d_w.abs()).all()
    only_y, only_w = op.combine_backward(e, y, w, plan, need=("y",)), op.combine_backward(e, y, w, plan, need=("w",))
    assert only_y.w is None and torch.equal(only_y.y, got.y)
    assert only_w.y is None and torch.equal(only_w.w, got.w)
    assert op.device_status() == 0


def test_gradients_against_differences(pkg):
    """d_x, d_y and d_w of a run to the rows and back, against central differences of the
    same run in 64 bits: <d, step> for a random direction of each input."""
    T, k, E, H = 37, 3, 5, 48
    op = handle(pkg, T, k, E, "bf16")
    _, ids, p = case(T, k, E, H, "bf16", 0.1, 0, seed=6)
    p = on_gpu(p)
    plan = pkg.RowPlan(*p)
    x, e = rr.rows(T, H, "bf16", 7), rr.rows(T, H, "bf16", 8)
    w = torch.rand(T, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    y = op.take(x, plan)
    d = op.combine_backward(e, y, w, plan)
    d_x = op.dispatch_backward(d.y, plan)

    def loss(x64, w64):
        out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            here = p[2][:, j] >= 0
            out[here] += w64[here, j, None] * x64[here]
        return (out * e.double()).sum()

    sx, sw = torch.randn(T, H, device="cuda").double(), torch.randn(T, k, device="cuda").double()
    h = 2.0 ** -10   # (the loss is linear in each: differences are exact up to 64-bit rounding)
    want = (loss(x.double() + h * sx, w.double()) - loss(x.double() - h * sx, w.double())) / (2 * h)
    got = (d_x.double() * sx).sum()
    # d_x: two roundings to bf16 (d_y, then their sum) of terms that |w e| bounds
    tol = (2 * 2.0 ** -8 * (w.double().abs().sum(1, keepdim=True) * e.double().abs()) * sx.abs()).sum()
    assert abs(got - want) <= tol
    want = (loss(x.double(), w.double() + h * sw) - loss(x.double(), w.double() - h * sw)) / (2 * h)
    got = (d.w.double() * sw).sum()
    tol = ((H + 2) * 2.0 ** -24 * (e.double().abs() * x.double().abs()).sum(1, keepdim=True) * sw.abs()).sum()
    assert abs(got - want) <= tol + 1e-9


def test_no_tokens(pkg):
    op = handle(pkg, 4, 2, 6, "bf16")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    rows, plan = op.dispatch(x, torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert rows.shape == (0, 64) and plan.order.numel() == 0 and plan.place.shape == (0, 2)
    assert plan.offsets.tolist() == [0] * 7
    w = torch.empty(0, 2, device="cuda")
    assert op.take(x, plan).shape == (0, 64) and op.combine(rows, w, plan).shape == (0, 64)
    d = op.combine_backward(x, rows, w, plan)
    assert d.y.shape == (0, 64) and d.w.shape == (0, 2) and op.dispatch_backward(rows, plan).shape == (0, 64)


@pytest.mark.parametrize("T", [3, 700])
def test_no_pick_has_an_expert(pkg, T):
    op = handle(pkg, T, 4, 9, "fp16")
    ids = torch.full((T, 4), -1, device="cuda")
    x, w = rr.rows(T, 96, "fp16", 0), torch.full((T, 4), float("nan"), device="cuda")
    rows, plan = op.dispatch(x, ids)
    assert not rows.any() and (plan.order == -1).all() and (plan.place == -1).all() and not plan.offsets.any()
    y = torch.full((4 * T, 96), float("inf"), dtype=torch.float16, device="cuda")
    assert not op.combine(y, w, plan).any() and not op.dispatch_backward(y, plan).any()
    d = op.combine_backward(x, y, w, plan)
    assert not d.y.any() and not d.w.any() and op.device_status() == 0


def test_one_expert_twice_and_one_for_all(pkg):
    op = handle(pkg, 500, 3, 4, "bf16")
    for ids in (torch.tensor([[1, 1, 0]]).repeat(500, 1), torch.full((500, 3), 3), torch.tensor([[2, -1, 2]])):
        p = rr.plan(ids, 4)
        x = rr.rows(ids.shape[0], 56, "bf16", 1)
        rows, plan = op.dispatch(x, ids.cuda())
        assert all(torch.equal(a, b.cuda()) for a, b in zip(plan, p))
        assert torch.equal(rows, rr.take(x, on_gpu(p), 3))
        want, bound = rr.combine(rows, None, on_gpu(p))
        ref.check(op.dispatch_backward(rows, plan), want, bound, "bf16", "d_x")


def test_values_that_are_not_finite_stay_in_their_rows(pkg):
    T, k, E, H = 40, 3, 8, 136
    op = handle(pkg, T, k, E, "bf16")
    _, ids, p = case(T, k, E, H, "bf16", 0.2, 0)
    p, plan = on_gpu(p), pkg.RowPlan(*on_gpu(p))
    y = rr.rows(T * k, H, "bf16", 1)
    w = torch.rand(T, k, device="cuda")
    r0 = int(p[2][p[2] >= 0][5])
    clean = op.combine(y, w, plan)
    y[r0, 3] = float("nan")
    y[r0, 4] = float("inf")
    got = op.combine(y, w, plan)
    t0 = int(p[1][r0]) // k
    changed = (got != clean) | got.isnan()
    assert got[t0, 3].isnan() and got[t0, 4].isinf() and changed.sum() == 2
    # a weight of a pick without an expert is not looked at
    w2 = torch.where(p[2] < 0, torch.full_like(w, float("nan")), w)
    assert torch.equal(op.combine(y, w2, plan).nan_to_num(7.0), got.nan_to_num(7.0))


def test_ids_out_of_range_are_reported(pkg):
    op = handle(pkg, 20, 2, 5, "bf16")
    ids = rr.make_ids(20, 2, 5, 0)
    x = rr.rows(20, 64, "bf16", 1)
    for bad, kind in ((5, torch.int32), (-2, torch.int64), (2 ** 40, torch.int64), (-2 ** 31, torch.int32)):
        mine = ids.clone()
        mine[7, 1] = bad
        rows, plan = op.dispatch(x, mine.to(kind).cuda())
        assert op.device_status() == 11 and op.device_status() == 0
        mine[7, 1] = -1
        p = rr.plan(mine, 5)
        assert all(torch.equal(a, b.cuda()) for a, b in zip(plan, p))
        assert torch.equal(rows, rr.take(x, on_gpu(p), 2))
    # a place past the rows: reported, and without an expert (the bounds check is the kernel's own)
    p = rr.plan(ids, 5)
    p[2][3, 0] = 40
    bad = pkg.RowPlan(*on_gpu(p))
    p[2][3, 0] = -1
    y, w = rr.rows(40, 64, "bf16", 2), torch.ones(20, 2, device="cuda")
    want, bound = rr.combine(y, w, on_gpu(p))
    ref.check(op.combine(y, w, bad), want, bound, "bf16", "out")
    assert op.device_status() == 11 and op.device_status() == 0


@pytest.mark.parametrize("H", [96, 33])
def test_strided_rows_and_given_outputs(pkg, H):
    """Inputs and outputs as column ranges of one wide buffer; what lies between stays."""
    T, k, E = 45, 2, 6
    op = handle(pkg, T, k, E, "fp16")
    _, ids, p = case(T, k, E, H, "fp16", 0.1, 0, seed=3)
    gp, plan = on_gpu(p), pkg.RowPlan(*on_gpu(p))
    wide = torch.full((T * k, 3 * H + 5), 9.0, dtype=torch.float16, device="cuda")
    x = rr.rows(T, H, "fp16", 4)
    rows, _ = op.dispatch(x, ids.cuda(), out=wide[:, H:2 * H])
    assert rows.data_ptr() == wide[:, H:].data_ptr() and torch.equal(wide[:, H:2 * H], rr.take(x, gp, k))
    assert (wide[:, :H] == 9).all() and (wide[:, 2 * H:] == 9).all()
    w = torch.rand(T, k, device="cuda")
    out = wide[:T, 2 * H:3 * H]
    want, bound = rr.combine(wide[:, H:2 * H], w, gp)
    op.combine(wide[:, H:2 * H], w, plan, out=out)      # columns beside its input
    ref.check(out, want, bound, "fp16", "out")
    assert (wide[:, :H] == 9).all() and (wide[T:, 2 * H:] == 9).all() and (wide[:, 3 * H:] == 9).all()
    assert torch.equal(wide[:, H:2 * H], rr.take(x, gp, k))


def test_refusals(pkg):
    op = handle(pkg, 8, 2, 5, "bf16")
    ids, x = rr.make_ids(8, 2, 5, 0).cuda(), rr.rows(8, 64, "bf16", 1)
    rows, plan = op.dispatch(x, ids)
    w = torch.ones(8, 2, device="cuda")
    other = rr.rows(8, 64, "fp16", 1)
    big = handle(pkg, 9, 2, 5, "bf16").plan(torch.zeros(9, 2, dtype=torch.int32, device="cuda"))
    for call in (
        lambda: op.dispatch(x, ids[:, :1].contiguous()), lambda: op.dispatch(x, ids.short()),
        lambda: op.dispatch(x, ids.cpu()), lambda: op.dispatch(x, ids.T.contiguous().T), lambda: op.dispatch(other, ids),
        lambda: op.dispatch(x.float(), ids), lambda: op.dispatch(x[:7], ids), lambda: op.dispatch(x[:, ::2], ids),
        lambda: op.dispatch(x.expand(8, 64)[:1].expand(8, 64), ids), lambda: op.dispatch(x[:, :0], ids),
        lambda: op.dispatch(x, ids, out=rows[:15]), lambda: op.dispatch(x, ids, out=rows[:, :63]),
        lambda: op.dispatch(torch.zeros(9, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(9, 2, dtype=torch.int32, device="cuda")),
        lambda: op.take(x, (plan.offsets[:-1], plan.order, plan.place)), lambda: op.take(x, (plan.offsets, plan.order.long(), plan.place)),
        lambda: op.combine(rows, None, plan), lambda: op.combine(rows, w[:7], plan), lambda: op.combine(rows, w.double(), plan),
        lambda: op.combine(rows[:15], w, plan), lambda: op.combine(rows, w, plan, out=rows[:8]),
        lambda: op.combine_backward(x, rows[:, :32], w, plan), lambda: op.combine_backward(x, rows, w, plan, need=("x",)),
        lambda: op.take(torch.zeros(9, 64, dtype=torch.bfloat16, device="cuda"), big),
    ):
        with pytest.raises(pkg.MoEError):
            call()
    assert torch.equal(op.take(x, plan), rows) and op.device_status() == 0


def test_overlaps_are_refused_by_the_c_entries(pkg):
    T, k, E, H = 6, 2, 5, 64
    op, lib = handle(pkg, T, k, E, "bf16"), pkg.load_library()
    buf = torch.zeros(1 << 16, device="cuda")
    at = {n: buf.data_ptr() + 4096 * i for i, n in
          enumerate(("x", "ids", "offsets", "order", "place", "rows", "y", "w", "out", "e", "d_y", "d_w"))}

    def dispatch(**o):
        p = {**at, **o}
        return lib.moe_rows_dispatch(op.handle, p["x"], H, T, H, p["ids"], 4, p["offsets"], p["order"], p["place"], p["rows"], H, None)

    def combine(**o):
        p = {**at, **o}
        return lib.moe_rows_combine(op.handle, p["y"], H, T, H, p["w"], 2, p["place"], p["out"], H, None)

    def grad(**o):
        p = {**at, **o}
        return lib.moe_rows_combine_backward(op.handle, p["e"], H, T, H, p["y"], H, p["w"], 2, p["offsets"], p["place"],
                                             p["d_y"], H, p["d_w"], None)

    assert dispatch() == 0 and combine() == 0 and grad() == 0
    for a, b in (("rows", "x"), ("rows", "ids"), ("rows", "place"), ("order", "ids"), ("place", "order"), ("offsets", "x")):
        assert dispatch(**{a: at[b]}) == 1, (a, b)
    for a in ("y", "w", "place"):
        assert combine(out=at[a]) == 1, a
    for o in ("d_y", "d_w"):
        for a in ("e", "y", "w", "place", "offsets"):
            assert grad(**{o: at[a]}) == 1, (o, a)
    assert grad(d_w=at["d_y"]) == 1
    assert dispatch(x=at["x"] + 1) == 1 and dispatch(ids=at["ids"] + 2) == 1 and combine(w=at["w"] + 2) == 1
    assert combine(y=None) == 1 and grad(w=None) == 1 and dispatch(place=None) == 1
    torch.cuda.synchronize()
    assert op.device_status() == 0


def step(op, x, ids, w, e):
    rows, plan = op.dispatch(x, ids)
    out = op.combine(rows, w, plan)
    d = op.combine_backward(e, rows, w, plan)
    return (rows, *plan, out, *d, op.dispatch_backward(d.y, plan))


@pytest.mark.parametrize("T", [5, 900])
def test_captured_and_replayed(pkg, T):
    k, E, H = 4, 17, 72
    op = handle(pkg, T, k, E, "bf16")
    ids, x, e = rr.make_ids(T, k, E, 0, 0.1).cuda(), rr.rows(T, H, "bf16", 1), rr.rows(T, H, "bf16", 2)
    w = torch.rand(T, k, device="cuda")
    step(op, x, ids, w, e)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(op, x, ids, w, e)
    for seed in (3, 4):
        ids.copy_(rr.make_ids(T, k, E, seed, 0.1))
        x.copy_(rr.rows(T, H, "bf16", seed))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step(op, x, ids, w, e)))


def test_two_handles_on_two_streams(pkg):
    T, k, E, H = 1500, 6, 300, 256
    ops = [handle(pkg, T, k, E, "bf16") for _ in range(2)]
    data = [(rr.rows(T, H, "bf16", s), rr.make_ids(T, k, E, s).cuda(), torch.rand(T, k, device="cuda"), rr.rows(T, H, "bf16", s + 5))
            for s in range(2)]
    want = [step(ops[0], *d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for op, s, d in zip(ops, streams, data):
            with torch.cuda.stream(s):
                got.append(step(op, *d))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_inputs_of_a_given_stream_may_be_dropped(pkg):
    T, k, E, H = 64, 3, 10, 512
    op = handle(pkg, T, k, E, "bf16")
    x, ids, w, e = rr.rows(T, H, "bf16", 1), rr.make_ids(T, k, E, 0).cuda(), torch.rand(T, k, device="cuda"), rr.rows(T, H, "bf16", 2)
    rows, plan = op.dispatch(x, ids)
    want = (rows, op.combine(rows, w, plan), *op.combine_backward(e, rows, w, plan), op.dispatch_backward(rows, plan))
    side = torch.cuda.Stream()
    for _ in range(3):
        mine = [t.clone() for t in (x, ids, w, e)]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        r, p = op.dispatch(mine[0], mine[1], stream=side)
        got = (r, op.combine(r, mine[2], p, stream=side), *op.combine_backward(mine[3], r, mine[2], p, stream=side),
               op.dispatch_backward(r, p, stream=side.cuda_stream))
        del mine
        over = [torch.full_like(t, 3) for t in (x, ids, w, e) for _ in range(3)]
        torch.cuda.synchronize()
        assert len(over) == 12 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_between_other_kernels(pkg):
    """Kernels of torch write the inputs right before and read the outputs right after."""
    T, k, E, H = 300, 4, 33, 1024
    op = handle(pkg, T, k, E, "bf16")
    w, e = torch.rand(T, k, device="cuda"), rr.rows(T, H, "bf16", 2)
    src = [(rr.rows(T, H, "bf16", s), rr.make_ids(T, k, E, s).cuda()) for s in range(6)]
    want = [[t.clone() for t in step(op, x, ids, w, e)] for x, ids in src]
    x, ids = torch.empty_like(src[0][0]), torch.empty_like(src[0][1])
    got = []
    for sx, si in src:
        x.copy_(sx)
        ids.copy_(si)
        got.append([t + 0 for t in step(op, x, ids, w, e)])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_offsets_past_32_bits(pkg):
    """6 GB of rows: the last rows are right."""
    T, k, E, H = 46000, 8, 256, 8192
    op = handle(pkg, T, k, E, "bf16")
    ids = (torch.arange(T * k, device="cuda") * 7 % E).reshape(T, k)
    x = rr.rows(T, H, "bf16", 1)
    rows, plan = op.dispatch(x, ids)
    order = torch.argsort(ids.reshape(-1), stable=True)
    assert torch.equal(plan.order.long(), order)
    tail = order[-3000:]
    assert torch.equal(rows[-3000:], x[tail // k])
    assert torch.equal(rows[:3000], x[order[:3000] // k])
    w = torch.full((T, k), 0.125, device="cuda")
    out = op.combine(rows, w, plan)
    assert torch.equal(out, x)        # eight equal rows: exact
    d = op.combine_backward(out, rows, w, plan, need=("y",))
    assert torch.equal(d.y[-3000:], (x[tail // k].float() * 0.125).bfloat16())
    assert op.device_status() == 0


@pytest.mark.parametrize("T,k,E", [(1 << 20, 16, 1024), (200001, 7, 300)])
def test_millions_of_picks(pkg, T, k, E):
    op = handle(pkg, T, k, E, "bf16")
    gen = torch.Generator(device="cuda").manual_seed(0)
    ids = torch.randint(-1, E, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    x = torch.arange(T, device="cuda", dtype=torch.int32).view(torch.int16).reshape(T, 2).view(torch.bfloat16)   # a row's number
    rows, plan = op.dispatch(x, ids)
    key = torch.where(ids < 0, E, ids).reshape(-1)
    order = torch.argsort(key, stable=True)
    n = int((key < E).sum())
    assert plan.offsets.tolist() == torch.searchsorted(key[order].contiguous(), torch.arange(E + 1, device="cuda", dtype=torch.int32)).tolist()
    assert torch.equal(plan.order[:n].long(), order[:n]) and (plan.order[n:] == -1).all()
    assert torch.equal(plan.place.reshape(-1)[order[:n]].long(), torch.arange(n, device="cuda"))
    assert (plan.place[ids < 0] == -1).all()
    assert torch.equal(rows[:n].view(torch.int16), x[order[:n] // k].view(torch.int16)) and not rows[n:].view(torch.int16).any()
    assert op.device_status() == 0


def test_a_failed_create_leaves_nothing(pkg):
    lib = pkg.load_library()
    live = lib.moe_debug_live_allocations()
    for n in (1, 2):
        lib.moe_debug_fail_allocation(n)
        with pytest.raises(pkg.MoEError) as err:
            handle(pkg, 5000, 2, 8, "bf16")
        assert err.value.status == 7 and lib.moe_debug_live_allocations() == live
    lib.moe_debug_fail_allocation(0)
    op = handle(pkg, 5000, 2, 8, "bf16")
    assert lib.moe_debug_live_allocations() == live + 2 and op.device_bytes() > 0
    op.close()
    assert lib.moe_debug_live_allocations() == live
