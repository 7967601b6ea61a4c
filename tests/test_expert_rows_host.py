"""Refusals of the tokens-by-expert operator on the host, and its plain forms on hand-worked
values (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

import quantized_moe_decode_gemv_gb300 as pkg
from quantized_moe_decode_gemv_gb300 import _capi, _train_ops
from tests import rows_reference as rr
from tests.test_ops_streams_host import STREAM, Tensor, handle


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_capi.LIB_PATH):
        pytest.fail("libmoe_gb300.so is not built; run __graft_entry__.build()")
    return _capi.load_library()


@pytest.mark.parametrize("kw,want", [
    ({}, "MOE_OK"), ({"n_experts": 1, "top_k": 1}, "MOE_OK"), ({"n_experts": 1024, "top_k": 16}, "MOE_OK"),
    ({"n_experts": 0}, "MOE_ERR_INVALID_ARG"), ({"max_tokens": 0}, "MOE_ERR_INVALID_ARG"),
    ({"top_k": 0}, "MOE_ERR_TOPK_GT_E"), ({"top_k": 9}, "MOE_ERR_TOPK_GT_E"),
    ({"n_experts": 1025}, "MOE_ERR_UNSUPPORTED"), ({"n_experts": 64, "top_k": 17}, "MOE_ERR_UNSUPPORTED"),
    ({"act_dtype": "fp32"}, "MOE_ERR_UNSUPPORTED"), ({"max_tokens": 1 << 23}, "MOE_OK"),
    ({"max_tokens": (1 << 23) + 1}, "MOE_ERR_UNSUPPORTED"),
])
def test_config_refusals(lib, kw, want):
    c = pkg.ExpertRowsConfig(**{**dict(n_experts=8, top_k=2, max_tokens=4), **kw}).to_c()
    assert _capi.STATUS_NAMES[lib.moe_rows_validate(ctypes.byref(c))] == want, lib.moe_rows_last_error(None)


def test_null_arguments(lib):
    assert lib.moe_rows_validate(None) == 1
    h = ctypes.c_void_p(5)
    c = pkg.ExpertRowsConfig(n_experts=8, top_k=2).to_c()
    assert lib.moe_rows_create(ctypes.byref(c), None) == 1
    assert lib.moe_rows_create(None, ctypes.byref(h)) == 1 and not h.value
    assert lib.moe_rows_plan(None, None, 4, 0, None, None, None, None) == 1
    assert lib.moe_rows_dispatch(None, None, 0, 0, 1, None, 4, None, None, None, None, 0, None) == 1
    assert lib.moe_rows_take(None, None, 0, 0, 1, None, None, None, 0, None) == 1
    assert lib.moe_rows_combine(None, None, 0, 0, 1, None, 2, None, None, 0, None) == 1
    assert lib.moe_rows_combine_backward(None, None, 0, 0, 1, None, 0, None, 2, None, None, None, 0, None, None) == 1
    assert lib.moe_rows_destroy(None) == 0 and lib.moe_rows_device_status(None, None) == 1
    assert lib.moe_rows_device_bytes(None) == 0 and lib.moe_rows_last_launch_count(None) == 0


@pytest.mark.parametrize("field", ["n_experts", "top_k", "max_tokens"])
def test_sizes_beyond_32_bits(field):
    for v in (2 ** 32 + 2, 2 ** 31):
        with pytest.raises(pkg.MoEError) as err:
            pkg.ExpertRowsConfig(**{**dict(n_experts=8, top_k=2), field: v}).to_c()
        assert err.value.status == 1
    with pytest.raises(pkg.MoEError):
        pkg.ExpertRowsConfig(n_experts=8, top_k=2, act_dtype="int8").to_c()


class Any(Tensor):
    """A stand-in tensor of any shape."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        super().__init__(shape[0], shape[-1], dtype)
        self.shape = shape


def op():
    fn = lambda *a: 0  # noqa: E731
    lib = type("Lib", (), {n: staticmethod(fn) for n in ("moe_rows_plan", "moe_rows_dispatch", "moe_rows_take", "moe_rows_combine",
                                                         "moe_rows_combine_backward")})
    h = handle(_train_ops.ExpertRows, _k=2, _E=5, _i32=torch.int32, _id_bytes={torch.int32: 4, torch.int64: 8}, _lib=lib,
               _w_types={torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}, config=pkg.ExpertRowsConfig(5, 2, max_tokens=4))
    h._empty = lambda shape, dtype, device: Any(*shape, dtype=dtype)
    return h


@pytest.mark.parametrize("stream,used", [(STREAM, [STREAM]), (None, [])])
def test_what_a_given_stream_uses_is_marked(stream, used):
    h, x, ids, w = op(), Any(3, 64), Any(3, 2, dtype=torch.int32), Any(3, 2, dtype=torch.float32)
    mine = [x, ids]
    rows, plan = h.dispatch(x, ids, stream=stream)
    assert all(t.used == used for t in mine)
    d_out, out = Any(3, 64), Any(3, 64)
    h.combine(rows, w, plan, out=out, stream=stream)
    assert all(t.used == used for t in (rows, w, out, *plan))
    for t in (rows, w, *plan):
        t.used.clear()
    h.combine_backward(d_out, rows, w, plan, stream=stream)
    assert all(t.used == used for t in (d_out, rows, w, *plan))
    for t in (rows, x, *plan):
        t.used.clear()
    h.dispatch_backward(rows, plan, stream=stream)
    h.take(x, plan, stream=stream)
    assert rows.used == used and x.used == used and all(t.used == 2 * used for t in plan)


def test_more_tokens_than_the_handle_serves():
    with pytest.raises(pkg.MoEError) as err:
        op().plan(Any(5, 2, dtype=torch.int32))
    assert err.value.status == 1


def test_plain_forms_on_hand_worked_values():
    ids = torch.tensor([[2, 0], [-1, 2], [0, 2]])
    p = rr.plan(ids, 4)
    assert p[0].tolist() == [0, 2, 2, 5, 5]
    assert p[1].tolist() == [1, 4, 0, 3, 5, -1]
    assert p[2].tolist() == [[2, 0], [-1, 3], [1, 4]]
    x = torch.tensor([[1.0], [2.0], [3.0]]).bfloat16()
    rows = rr.take(x, p, 2)
    assert rows[:, 0].tolist() == [1, 3, 1, 2, 3, 0]
    w = torch.tensor([[0.5, 2.0], [9.0, 0.25], [1.0, 4.0]])
    out, _ = rr.combine(rows, w, p)
    assert out[:, 0].tolist() == [2.5, 0.5, 15.0]
    (d_y, _), (d_w, _) = rr.combine_backward(torch.tensor([[1.0], [10.0], [100.0]]).bfloat16(), rows, w, p)
    assert d_y[:, 0].tolist() == [2.0, 100.0, 0.5, 2.5, 400.0, 0.0]
    assert d_w.tolist() == [[1, 1], [0, 20], [300, 300]]


def test_chained_kernels_promise_no_constant_inputs():
    """As for the other operators: inputs may be written until the kernel's wait."""
    path = os.path.join(os.path.dirname(_capi.__file__), "csrc", "moe_rows.cuh")
    text = re.sub(r"//[^\n]*", "", open(path).read())
    kernels = re.split(r"__global__", text)[1:]
    assert len(kernels) == 8
    for kernel in kernels:
        head, body = kernel.split("{", 1)
        assert "griddepcontrol.wait" in body and "__restrict__" not in head


def test_chunks_are_waited_for_before_their_totals():
    """The plan of several chunks begins while they are counted, and waits before it adds them."""
    text = open(os.path.join(os.path.dirname(_capi.__file__), "csrc", "moe_rows.cuh")).read()
    body = text[text.index("void rw_plan("):]
    assert body.index("griddepcontrol.wait") < body.index("A.totals[") < body.index("rw_starts(A, write")
    # and whoever counts has waited for the ids before it lets the plan begin
    for kernel in ("k_rows_count(", "k_rows_scan("):
        k = text[text.index("void __launch_bounds__(RW_CHUNK, 1) " + kernel):]
        assert k.index("griddepcontrol.wait") < k.index("griddepcontrol.launch_dependents") < k.index("A.totals")
