"""The operators on streams of their own: what a call on a given stream uses may be
dropped right after it, and calls after a join of streams wait for both."""
import pytest
import torch

from tests.test_gpu_ops import make_block, make_linear, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import quantized_moe_decode_gemv_gb300 as p
    p.load_library()
    return p


@pytest.mark.parametrize("T", [8, 64])
def test_inputs_of_a_given_stream_may_be_dropped(pkg, T):
    """The side stream is busy for some milliseconds; memory of the dropped inputs is
    asked for again and overwritten before the call has run."""
    op, _, _, _ = make_linear(pkg, 320, 512, "affine", 64, "bf16", "none", False, 64)
    block, bx, up, gate, e = make_block(pkg, T, 512, 320, "bf16", "swiglu", True)
    x = rows(T, 512, "bf16", 3)
    want = op(x)
    h, saved = block.forward_train(x, up, gate)
    grads = block.backward(e, saved, x, up, gate)
    side = torch.cuda.Stream()
    for _ in range(4):
        mine = [t.clone() for t in (x, up, gate, e)]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)   # about ten milliseconds
        got = op.forward(mine[0], stream=side)
        got_h, got_saved = block.forward_train(mine[0], mine[1], mine[2], stream=side)
        got_d = block.backward(mine[3], got_saved, mine[0], mine[1], mine[2], stream=side)
        shapes = [t.shape for t in mine]
        del mine
        over = [torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda") for s in shapes for _ in range(3)]
        torch.cuda.synchronize()
        assert len(over) == 12 and torch.equal(got, want) and torch.equal(got_h, h)
        assert all(torch.equal(a, b) for a, b in zip(got_d, grads))


def test_a_call_after_a_join_waits_for_both_streams(pkg):
    """x is written on a side stream that the call's stream waits for: directly, and captured."""
    for T in (8, 64):
        op, _, _, _ = make_linear(pkg, 320, 512, "nvfp4", 16, "bf16", "none", False, 64)
        block, _, up, gate, _ = make_block(pkg, T, 320, 512, "bf16", "swiglu", False)
        src = [rows(T, 512, "bf16", s) for s in range(4)]
        x, side = torch.empty_like(src[0]), torch.cuda.Stream()
        want = []
        for s in src:
            y = op(s)
            want.append((y, block(y, up, gate)))
        torch.cuda.synchronize()

        def step(s):
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            y0 = op(s)            # work of the call's own stream, to be waited for too
            with torch.cuda.stream(side):
                torch.cuda._sleep(2_000_000)
                x.copy_(s)
            main.wait_stream(side)
            y = op(x)
            return y0, y, block(y, up, gate)

        for s, (wy, wz) in zip(src, want):
            y0, y, z = step(s)
            assert torch.equal(y0, wy) and torch.equal(y, wy) and torch.equal(z, wz)
        held = src[0].clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(held)
        for s, (wy, wz) in zip(src, want):
            held.copy_(s)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got[0], wy) and torch.equal(got[1], wy) and torch.equal(got[2], wz)


def test_captured_on_a_given_stream(pkg):
    """The capture's own stream and one forked from it, by object and by number; inputs made
    inside and outside the capture."""
    T = 40
    op, _, _, _ = make_linear(pkg, 320, 512, "mxfp4", 32, "bf16", "none", False, 64)
    block, x, up, gate, e = make_block(pkg, T, 512, 320, "bf16", "swiglu", True)
    x = x.contiguous()

    def want_of():
        h, saved = block.forward_train(x, up, gate)
        return op(x), h, *block.backward(e, saved, x, up, gate)

    want = want_of()
    torch.cuda.synchronize()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        inside = x + 0
        side.wait_stream(main)
        y = op.forward(inside, stream=side.cuda_stream)
        h, saved = block.forward_train(x, up, gate, stream=main)
        d = block.backward(e, saved, x, up, gate, stream=main.cuda_stream)
        main.wait_stream(side)
        del inside
    for seed in (1, 2):
        x.copy_(rows(T, 512, "bf16", seed))
        torch.cuda.synchronize()
        want = want_of()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (y, h, *d)))
