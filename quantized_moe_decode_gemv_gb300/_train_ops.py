"""Python handles of the operators around the training of routed experts
(include/moe_layer.h): tokens sorted by expert and back, orthogonalised updates.

Argument checks and marshalling, as in ``_ops``; the arithmetic runs in the CUDA
library.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Any, NamedTuple, Tuple

from ._capi import DTYPE, MOE_OK, MoEError, load_library, moe_ortho_config, moe_rows_config, torch_act_dtype
from ._ops import _INVALID_ARG, _SHAPE, _Handle, _int32, _name_of


def _device_of(torch, device):
    """A CUDA device with its index; the current one for None."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if device.type != "cuda":
        raise MoEError(_INVALID_ARG, f"the operator runs on a CUDA device, not on {device}")
    return torch.device("cuda", torch.cuda.current_device()) if device.index is None else device


def _create(handle, torch, c, device) -> None:
    """Validates the C config (before a device is looked for) and creates the handle on its device."""
    status = handle._fn("validate")(ctypes.byref(c))
    if status == MOE_OK:
        handle.device = _device_of(torch, device)
        h = ctypes.c_void_p()
        with torch.cuda.device(handle.device):
            status = handle._fn("create")(ctypes.byref(c), ctypes.byref(h))
    if status != MOE_OK:
        raise MoEError(status, handle._fn("last_error")(None).decode())
    handle.handle = h.value


# ---------------------------------------------------------------------------
# tokens sorted by expert and back
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class ExpertRowsConfig:
    """Mirror of ``moe_rows_config``."""
    n_experts: int
    top_k: int
    act_dtype: str = "bf16"
    max_tokens: int = 16

    def to_c(self) -> moe_rows_config:
        return moe_rows_config(
            n_experts=_int32(self.n_experts, "n_experts"), top_k=_int32(self.top_k, "top_k"),
            act_dtype=_name_of(DTYPE, self.act_dtype, "act_dtype"), max_tokens=_int32(self.max_tokens, "max_tokens"))


class RowPlan(NamedTuple):
    """Where every pick's row is: int32 tensors offsets [E + 1], order [T k], place [T, k]."""
    offsets: Any
    order: Any
    place: Any


class RowGrads(NamedTuple):
    """Gradients of ``combine`` (None where not asked for)."""
    y: Any
    w: Any


class ExpertRows(_Handle):
    """A batch's tokens as rows sorted by expert, the experts' rows back to the tokens with
    weights, and the gradients of both.

    ``ids`` [T, k] (int32 or int64, -1: no expert) name each token's experts.  Sorted rows
    come as [T k, H]: expert e's are ``offsets[e] : offsets[e + 1]``, rows from
    ``offsets[E]`` on are zero.  ``offsets`` stay on the GPU; reading them on the host, to call an
    operator for each expert's rows, waits for it.

    No autograd function: ``requires_grad`` is not looked at, outputs carry no graph; a
    training loop keeps the plan and calls the backward methods.
    """

    _prefix = "moe_rows"

    def __init__(self, config: ExpertRowsConfig, device=None):
        import torch
        self._setup(torch, load_library())
        self.config = config
        _create(self, torch, config.to_c(), device)
        self._dtype, self._k, self._E = torch_act_dtype(config.act_dtype), config.top_k, config.n_experts
        self._i32, self._id_bytes = torch.int32, {torch.int32: 4, torch.int64: 8}
        self._w_types = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

    # A decode call's kernel takes a few microseconds: arguments are checked by plain comparisons,
    # and reasons are found when one fails.

    def _ids(self, ids) -> int:
        shape = ids.shape
        if len(shape) != 2 or shape[1] != self._k:
            raise MoEError(_SHAPE, f"ids must be [T, {self._k}], not {list(shape)}")
        if ids.dtype not in self._id_bytes or ids.device != self.device or not ids.is_contiguous():
            raise MoEError(_INVALID_ARG, f"ids must be a contiguous int32 or int64 tensor on {self.device}")
        if shape[0] > self.config.max_tokens:
            raise MoEError(_INVALID_ARG, f"{shape[0]} tokens, max_tokens is {self.config.max_tokens}")
        return shape[0]

    def _width(self, x, rows: int, what: str) -> int:
        shape = x.shape
        if len(shape) != 2 or shape[0] != rows:
            raise MoEError(_SHAPE, f"{what} must be [{rows}, H], not {list(shape)}")
        return shape[1]

    def _bad_plan(self, plan, T):
        for t, shape, what in zip(plan, ((self._E + 1,), (T * self._k,), (T, self._k)), RowPlan._fields):
            if t.shape != shape:
                raise MoEError(_SHAPE, f"the plan's {what} must be {list(shape)}, not {list(t.shape)}")
        raise MoEError(_INVALID_ARG, f"the plan must be three contiguous int32 tensors on {self.device}")

    def _plan(self, plan) -> int:
        """T of a plan, its tensors checked."""
        offsets, order, place = plan
        T, i32, device = place.shape[0], self._i32, self.device
        if not (place.shape == (T, self._k) and order.shape == (T * self._k,) and offsets.shape == (self._E + 1,) and
                place.dtype is i32 and order.dtype is i32 and offsets.dtype is i32 and place.device == device and
                order.device == device and offsets.device == device and place.is_contiguous() and order.is_contiguous() and
                offsets.is_contiguous()):
            self._bad_plan(plan, T)
        if T > self.config.max_tokens:
            raise MoEError(_INVALID_ARG, f"a plan of {T} tokens, max_tokens is {self.config.max_tokens}")
        return T

    def _weights(self, w, T: int) -> int:
        if w.shape != (T, self._k):
            raise MoEError(_SHAPE, f"w must be [{T}, {self._k}], not {list(w.shape)}")
        if w.dtype not in self._w_types or w.device != self.device or not w.is_contiguous():
            raise MoEError(_INVALID_ARG, f"w must be a contiguous fp32, bf16 or fp16 tensor on {self.device}")
        return self._w_types[w.dtype]

    def _given(self, out, rows: int, H: int) -> int:
        """Row stride of an output that the caller gives."""
        ld = self._stride(out, H, "out")
        if out.shape[0] != rows:
            raise MoEError(_SHAPE, f"out has {out.shape[0]} rows, not {rows}")
        return ld

    def _new_plan(self, T: int) -> RowPlan:
        k, empty, i32, device = self._k, self._empty, self._i32, self.device
        return RowPlan(empty((self._E + 1,), dtype=i32, device=device), empty((T * k,), dtype=i32, device=device),
                       empty((T, k), dtype=i32, device=device))

    def _new(self, rows: int, H: int):
        return self._empty((rows, H), dtype=self._dtype, device=self.device)

    def plan(self, ids, stream=None) -> RowPlan:
        """The plan of ids [T, k] alone."""
        T = self._ids(ids)
        s, where = self._stream(stream, ids)
        with where:
            p = self._new_plan(T)
        status = self._lib.moe_rows_plan(self.handle, ids.data_ptr(), self._id_bytes[ids.dtype], T, p[0].data_ptr(),
                                         p[1].data_ptr(), p[2].data_ptr(), s)
        if status:
            self._fail(status)
        return p

    def dispatch(self, x, ids, out=None, stream=None):
        """(rows [T k, H], plan) of x [T, H] (rows may be strided) and ids [T, k]."""
        T = self._ids(ids)
        H = ldo = self._width(x, T, "x")
        ldx = self._stride(x, H, "x")
        if out is not None:
            ldo = self._given(out, T * self._k, H)
        s, where = self._stream(stream, x, ids, out)
        with where:
            if out is None:
                out = self._new(T * self._k, H)
            p = self._new_plan(T)
        status = self._lib.moe_rows_dispatch(self.handle, x.data_ptr(), ldx, T, H, ids.data_ptr(), self._id_bytes[ids.dtype],
                                             p[0].data_ptr(), p[1].data_ptr(), p[2].data_ptr(), out.data_ptr(), ldo, s)
        if status:
            self._fail(status)
        return out, p

    def take(self, x, plan, out=None, stream=None):
        """rows [T k, H] of x [T, H] by a plan that is there already."""
        T = self._plan(plan)
        H = ldo = self._width(x, T, "x")
        ldx = self._stride(x, H, "x")
        if out is not None:
            ldo = self._given(out, T * self._k, H)
        s, where = self._stream(stream, x, out, *plan)
        if out is None:
            with where:
                out = self._new(T * self._k, H)
        status = self._lib.moe_rows_take(self.handle, x.data_ptr(), ldx, T, H, plan[0].data_ptr(), plan[2].data_ptr(),
                                         out.data_ptr(), ldo, s)
        if status:
            self._fail(status)
        return out

    def _combine(self, y, w, plan, out, stream, what):
        T = self._plan(plan)
        H = ldo = self._width(y, T * self._k, what)
        ldy = self._stride(y, H, what)
        wt = 2 if w is None else self._weights(w, T)
        if out is not None:
            ldo = self._given(out, T, H)
        s, where = self._stream(stream, y, w, out, *plan)
        if out is None:
            with where:
                out = self._new(T, H)
        status = self._lib.moe_rows_combine(self.handle, y.data_ptr(), ldy, T, H, None if w is None else w.data_ptr(), wt,
                                            plan[2].data_ptr(), out.data_ptr(), ldo, s)
        if status:
            self._fail(status)
        return out

    def combine(self, y, w, plan, out=None, stream=None):
        """out [T, H]: a token's rows of y [T k, H], weighted by w [T, k] (fp32 or 16-bit) and summed."""
        if w is None:
            raise MoEError(_INVALID_ARG, "w is missing")
        return self._combine(y, w, plan, out, stream, "y")

    def dispatch_backward(self, d_rows, plan, out=None, stream=None):
        """d_x [T, H] for the gradient d_rows [T k, H] of ``dispatch``'s (or ``take``'s) rows."""
        return self._combine(d_rows, None, plan, out, stream, "d_rows")

    def combine_backward(self, d_out, y, w, plan, need=("y", "w"), stream=None) -> RowGrads:
        """Gradients of the tensors named in ``need`` for the gradient d_out [T, H] of ``combine``'s out."""
        for n in need:
            if n not in RowGrads._fields:
                raise MoEError(_INVALID_ARG, f"need names {', '.join(RowGrads._fields)}")
        T = self._plan(plan)
        P = T * self._k
        H = self._width(d_out, T, "d_out")
        ldd = self._stride(d_out, H, "d_out")
        if self._width(y, P, "y") != H:
            raise MoEError(_SHAPE, f"y is {y.shape[1]} wide, d_out {H}")
        ldy = self._stride(y, H, "y")
        wt = self._weights(w, T)
        s, where = self._stream(stream, d_out, y, w, *plan)
        with where:
            d_y = self._new(P, H) if "y" in need else None
            d_w = self._empty((T, self._k), dtype=w.dtype, device=self.device) if "w" in need else None
        status = self._lib.moe_rows_combine_backward(
            self.handle, d_out.data_ptr(), ldd, T, H, y.data_ptr(), ldy, w.data_ptr(), wt, plan[0].data_ptr(),
            plan[2].data_ptr(), None if d_y is None else d_y.data_ptr(), H, None if d_w is None else d_w.data_ptr(), s)
        if status:
            self._fail(status)
        return RowGrads(d_y, d_w)


# ---------------------------------------------------------------------------
# orthogonalised updates
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class OrthoConfig:
    """Mirror of ``moe_ortho_config``."""
    rows: int
    cols: int
    max_matrices: int = 1
    dtype: str = "bf16"          # of the matrices: "bf16", "fp16" or "fp32"
    steps: int = 5
    coefficients: Tuple[float, float, float] = (3.4445, -4.7750, 2.0315)
    eps: float = 1e-7

    def to_c(self) -> moe_ortho_config:
        if len(self.coefficients) != 3:
            raise MoEError(_INVALID_ARG, f"three coefficients (of X, X^3 and X^5), not {len(self.coefficients)}")
        a, b, c = (float(v) for v in self.coefficients)
        return moe_ortho_config(
            rows=_int32(self.rows, "rows"), cols=_int32(self.cols, "cols"), dtype=_name_of(DTYPE, self.dtype, "dtype"),
            steps=_int32(self.steps, "steps"), max_matrices=_int32(self.max_matrices, "max_matrices"), a=a, b=b, c=c,
            eps=float(self.eps))


class Orthogonalizer(_Handle):
    """Matrices [rows, cols], alone or stacked as [n, rows, cols], each brought near the
    orthogonal matrix of its singular vectors (all singular values to about 1), as bf16.

    For weight gradients or momentum of any of the three types; a tall matrix is taken
    from its other side, nothing is transposed in memory.  Products have fp16 operands and fp32
    sums, whatever the type: with the default coefficients and a smaller side of 64 and more the
    result is off by about 2e-3 of its norm in five steps, bf16's rounding included, 3e-3 in
    eight; include/moe_layer.h has the bounds for all sizes, steps and coefficients.
    """

    _prefix = "moe_ortho"

    def __init__(self, config: OrthoConfig, device=None):
        import torch
        self._setup(torch, load_library())
        self.config = config
        _create(self, torch, config.to_c(), device)
        self._dtype = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[config.dtype]
        self._bf16, self._R, self._C, self._call = torch.bfloat16, config.rows, config.cols, self._lib.moe_ortho_forward

    def _stack(self, t, dtype, what: str):
        """(number, row stride, matrix stride) of a matrix or a stack of them."""
        shape = t.shape
        if len(shape) not in (2, 3) or shape[-2] != self._R or shape[-1] != self._C:
            raise MoEError(_SHAPE, f"{what} must be [{self._R}, {self._C}] or a stack of them, not {list(shape)}")
        if t.dtype is not dtype:
            raise MoEError(_INVALID_ARG, f"{what} must be {dtype}, not {t.dtype}")
        if t.device != self.device:
            raise MoEError(_INVALID_ARG, f"{what} is on {t.device}, the handle on {self.device}")
        n = shape[0] if len(shape) == 3 else 1
        stride = t.stride()
        if stride[-1] != 1 and self._C > 1 and n:
            raise MoEError(_INVALID_ARG, f"{what} needs consecutive columns")
        if n > self.config.max_matrices:
            raise MoEError(_INVALID_ARG, f"{what} has {n} matrices, max_matrices is {self.config.max_matrices}")
        return n, stride[-2], stride[0] if len(shape) == 3 else 0

    def forward(self, g, out=None, stream=None):
        """out (bf16, g's shape) of g; rows and matrices of both may be strided."""
        n, ldg, step_g = self._stack(g, self._dtype, "g")
        s, where = self._stream(stream, g, out)
        if out is None:
            with where:
                out = self._empty(g.shape, dtype=self._bf16, device=self.device)
        elif out.shape != g.shape:
            raise MoEError(_SHAPE, f"out must be {list(g.shape)}, not {list(out.shape)}")
        _, ldo, step_o = self._stack(out, self._bf16, "out")
        status = self._call(self.handle, g.data_ptr(), ldg, step_g, n, out.data_ptr(), ldo, step_o, s)
        if status:
            self._fail(status)
        return out

    __call__ = forward
