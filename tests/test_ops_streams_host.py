"""What the Python handles of the operators do with a given stream, on stand-ins
for the library, its tensors and streams (no GPU needed)."""
import contextlib
import types

import pytest
import torch

import quantized_moe_decode_gemv_gb300 as pkg
from quantized_moe_decode_gemv_gb300 import _ops

DEVICE = torch.device("cuda", 0)


class Tensor:
    """A [rows, cols] tensor of the device that notes the streams it is used on."""

    def __init__(self, rows, cols, dtype=torch.bfloat16):
        self.shape, self.dtype, self.device, self.used = (rows, cols), dtype, DEVICE, []

    def stride(self):
        return self.shape[1], 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def record_stream(self, stream):
        self.used.append(stream)


def handle(cls, **fields):
    h = cls.__new__(cls)
    cuda = types.SimpleNamespace(stream=lambda s: contextlib.nullcontext(), ExternalStream=lambda s, device: (s, device))
    h._torch, h.device, h.handle, h._dtype = types.SimpleNamespace(cuda=cuda), DEVICE, None, torch.bfloat16
    h._empty = lambda shape, dtype, device: Tensor(*shape, dtype)
    h._raw_stream = lambda index: 7
    for n, v in fields.items():
        setattr(h, n, v)
    return h


def linear():
    return handle(_ops.QLinear, _K=64, _N=32, _call=lambda *a: 0)


def block(gated):
    return handle(_ops.GatedBlock, _K=64, _N=32, _gated=gated, _f32=torch.float32, _call_forward=lambda *a: 0,
                  _call_backward=lambda *a: 0)


STREAM = types.SimpleNamespace(cuda_stream=99)


@pytest.mark.parametrize("stream,used", [(STREAM, [STREAM]), (None, [])])
def test_linear_marks_what_a_given_stream_uses(stream, used):
    x, out = Tensor(3, 64), Tensor(3, 32)
    linear().forward(x, stream=stream)
    assert x.used == used
    linear().forward(x, out=out, stream=stream)
    assert out.used == used


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("stream,used", [(STREAM, [STREAM]), (None, [])])
def test_block_marks_what_a_given_stream_uses(gated, stream, used):
    op, x, d, up = block(gated), Tensor(3, 64), Tensor(3, 32), Tensor(32, 64)
    gate = Tensor(32, 64) if gated else None
    out, saved = op.forward_train(x, up, gate, stream=stream)
    mine = [x, up] + ([gate] if gated else [])
    assert all(t.used == used for t in mine)
    for t in mine:
        t.used.clear()
    op.backward(d, saved, x, up, gate, stream=stream)
    assert all(t.used == used for t in mine + [d] + [s for s in saved if s is not None])


def test_the_package_exports_the_handles():
    assert pkg.QLinear is _ops.QLinear and pkg.GatedBlock is _ops.GatedBlock
