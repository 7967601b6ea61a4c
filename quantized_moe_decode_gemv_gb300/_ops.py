"""Python handles of the operators around the MoE layer (include/moe_layer.h):
the linear operators with 4-bit weights and the 16-bit gated block.

Argument checks and marshalling; the arithmetic runs in the CUDA library.
Outputs are allocated on the stream of the call: with ``stream=None`` the
current one, otherwise the given one, where a consumer on another stream has to
order itself after the call as after any kernel.  The caller orders a given stream
after what writes the inputs; tensors handed to such a call are marked as used on
it (``Tensor.record_stream``), so they may be dropped right after the call.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import operator
from typing import Any, Dict, NamedTuple, Optional, Tuple

from ._capi import (ACT, DTYPE, MOE_OK, QLINEAR_ACT, WFMT, MoEError, load_library, moe_gated_config,
                    moe_qlinear_config, moe_qlinear_weights, torch_act_dtype)

_INVALID_ARG, _SHAPE = 1, 5
_HERE = contextlib.nullcontext()


def _name_of(table: Dict[str, int], key: str, what: str) -> int:
    if key not in table:
        raise MoEError(_INVALID_ARG, f"unknown {what} {key!r} (one of {', '.join(table)})")
    return table[key]


def _int32(value, what: str) -> int:
    """``value`` for a C int32 field (ctypes would keep its low 32 bits)."""
    v = operator.index(value)
    if not -2 ** 31 <= v < 2 ** 31:
        raise MoEError(_INVALID_ARG, f"{what} {v} does not fit 32 bits")
    return v


class _Handle:
    """What the operator handles share: device, streams, status, lifetime.

    A decode call's kernel takes a few microseconds, so its wrapper has to stay
    below that: tensors are checked by plain comparisons, and the current stream
    is read by torch's raw accessor where there is one.
    """

    _prefix = ""

    def _setup(self, torch, lib):
        self._torch, self._lib, self.handle = torch, lib, None
        self._empty = torch.empty
        self._raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

    def _fn(self, name: str):
        return getattr(self._lib, f"{self._prefix}_{name}")

    def _fail(self, status: int) -> None:
        raise MoEError(status, self._fn("last_error")(self.handle).decode())

    def _stride(self, x, cols: int, what: str) -> int:
        """Row stride of a [T, cols] tensor of the handle's type on its device (a single row has none)."""
        shape = x.shape
        if len(shape) != 2 or shape[1] != cols:
            raise MoEError(_SHAPE, f"{what} must be [T, {cols}], not {list(shape)}")
        if x.dtype is not self._dtype:
            raise MoEError(_INVALID_ARG, f"{what} must be {self._dtype}, not {x.dtype}")
        if x.device != self.device:
            raise MoEError(_INVALID_ARG, f"{what} is on {x.device}, the handle on {self.device}")
        row, col = x.stride()
        if col != 1 and cols > 1 and shape[0]:
            raise MoEError(_INVALID_ARG, f"{what} needs consecutive columns")
        if shape[0] <= 1:
            return cols
        if shape[0] >= 2 ** 31:   # (the C entry refuses more rows than max_tokens)
            raise MoEError(_INVALID_ARG, f"{what} has {shape[0]} rows")
        if row < cols:
            raise MoEError(_INVALID_ARG, f"{what} has overlapping rows")
        return row

    def _matrix(self, w, rows: int, cols: int, what: str) -> int:
        if w is None:
            raise MoEError(_INVALID_ARG, f"{what} is missing")
        if w.shape != (rows, cols):
            raise MoEError(_SHAPE, f"{what} must be [{rows}, {cols}], not {list(w.shape)}")
        if w.dtype is not self._dtype or w.device != self.device or not w.is_contiguous():
            raise MoEError(_INVALID_ARG, f"{what} must be a contiguous {self._dtype} tensor on {self.device}")
        return w.data_ptr()

    def _stream(self, stream, *tensors):
        """(stream handle, context in which outputs are allocated) of a call that uses ``tensors``."""
        if stream is None:
            if self._raw_stream is not None:
                return self._raw_stream(self.device.index), _HERE
            return self._torch.cuda.current_stream(self.device).cuda_stream, _HERE
        if not hasattr(stream, "cuda_stream"):
            stream = self._torch.cuda.ExternalStream(int(stream), device=self.device)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)   # not the allocation's own: freed memory waits for it
        return int(stream.cuda_stream), self._torch.cuda.stream(stream)

    def device_status(self, stream=None) -> int:
        """Synchronises the stream and returns the status recorded by the kernels since the last call."""
        return self._fn("device_status")(self.handle, ctypes.c_void_p(self._stream(stream)[0]))

    def device_bytes(self) -> int:
        return int(self._fn("device_bytes")(self.handle))

    def last_launch_count(self) -> int:
        return int(self._fn("last_launch_count")(self.handle))

    def close(self) -> None:
        """Frees the handle (also when it is collected); waits for the device, so not during a graph capture."""
        if getattr(self, "handle", None):
            handle, self.handle = self.handle, None
            self._fn("destroy")(handle)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------
# linear operators with 4-bit weights
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class QLinearConfig:
    """Mirror of ``moe_qlinear_config``."""
    in_features: int
    out_features: int
    fmt: str = "affine"          # "affine", "nvfp4" or "mxfp4"
    group_size: int = 64
    act_dtype: str = "bf16"
    scale_dtype: str = "bf16"
    act: str = "none"            # "none", "swiglu" or "relu2"
    bias: bool = False
    max_tokens: int = 16

    def to_c(self) -> moe_qlinear_config:
        return moe_qlinear_config(
            in_features=_int32(self.in_features, "in_features"),
            out_features=_int32(self.out_features, "out_features"), group_size=_int32(self.group_size, "group_size"),
            weight_format=_name_of(WFMT, self.fmt, "fmt"), act_dtype=_name_of(DTYPE, self.act_dtype, "act_dtype"),
            scale_dtype=_name_of(DTYPE, self.scale_dtype, "scale_dtype"), act=_name_of(QLINEAR_ACT, self.act, "act"),
            has_bias=int(bool(self.bias)), max_tokens=_int32(self.max_tokens, "max_tokens"))


class QLinear(_Handle):
    """``out = x W^T (+ bias)``, ``silu(x Wg^T) * (x W^T)`` or ``max(x W^T, 0)^2`` with 4-bit weights.

    ``weights``: device tensors by C field name -- ``q`` int32 [N, K/8], ``s``,
    ``b`` (affine: scale dtype [N, K/G]; nvfp4: uint8 [N, K/16] and fp32 [1];
    mxfp4: uint8 [N, K/32] and None), ``gate_q``, ``gate_s``, ``gate_b`` for
    "swiglu", ``bias`` [N].  They are copied and may be freed afterwards.

    No autograd function: ``requires_grad`` is not looked at, and ``out`` carries no graph.
    """

    _prefix = "moe_qlinear"

    def __init__(self, config: QLinearConfig, weights: Dict[str, Any], stream=None):
        import torch
        self._setup(torch, load_library())
        self.config = config
        c = config.to_c()
        w = {n: weights.get(n) for n, _ in moe_qlinear_weights._fields_}
        unknown = set(weights) - set(w)
        if unknown:
            raise MoEError(_INVALID_ARG, f"unknown weights {sorted(unknown)}")
        cw = moe_qlinear_weights(**{n: (None if t is None else t.data_ptr()) for n, t in w.items()})
        status = self._fn("validate")(ctypes.byref(c), ctypes.byref(cw))
        if status != MOE_OK:
            raise MoEError(status, self._fn("last_error")(None).decode())
        self._check_weights(w)
        self.device = w["q"].device
        self._dtype = torch_act_dtype(config.act_dtype)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            status = self._fn("create")(ctypes.byref(c), ctypes.byref(cw), ctypes.c_void_p(self._stream(stream)[0]),
                                        ctypes.byref(h))
        if status != MOE_OK:
            raise MoEError(status, self._fn("last_error")(None).decode())
        self.handle = h.value
        self._call, self._K, self._N = self._lib.moe_qlinear_forward, config.in_features, config.out_features

    def _check_weights(self, w) -> None:
        torch, c = self._torch, self.config
        N, K, G = c.out_features, c.in_features, c.group_size
        words = (torch.int32, torch.uint32)
        if c.fmt == "affine":
            sdt = (torch_act_dtype(c.scale_dtype),)
            form = {"q": ((N, K // 8), words), "s": ((N, K // G), sdt), "b": ((N, K // G), sdt)}
        else:
            form = {"q": ((N, K // 8), words), "s": ((N, K // G), (torch.uint8,)),
                    "b": ((1,), (torch.float32,)) if c.fmt == "nvfp4" else None}
        if c.act == "swiglu":
            form.update({"gate_" + n: f for n, f in list(form.items())})
        if c.bias:
            form["bias"] = ((N,), (torch_act_dtype(c.act_dtype),))
        device = w["q"].device
        for n, f in form.items():
            t = w[n]
            if f is None or t is None:
                continue
            if tuple(t.shape) != f[0] or t.dtype not in f[1]:
                raise MoEError(_SHAPE, f"{n} must be {f[1][0]} {list(f[0])}, not {t.dtype} {list(t.shape)}")
            if t.device != device or not t.is_cuda or not t.is_contiguous():
                raise MoEError(_INVALID_ARG, f"{n} must be contiguous and on one CUDA device")

    def forward(self, x, out=None, stream=None):
        """out [T, N] of x [T, K] (rows may be strided); ``out`` may be given, rows strided too."""
        ldx = self._stride(x, self._K, "x")
        T = x.shape[0]
        s, where = self._stream(stream, x, out)
        if out is None:
            if stream is None:
                out = self._empty((T, self._N), dtype=self._dtype, device=self.device)
            else:
                with where:
                    out = self._empty((T, self._N), dtype=self._dtype, device=self.device)
            ldo = self._N
        else:
            ldo = self._stride(out, self._N, "out")
            if out.shape[0] != T:
                raise MoEError(_SHAPE, f"out has {out.shape[0]} rows, x {T}")
        status = self._call(self.handle, x.data_ptr(), ldx, T, out.data_ptr(), ldo, s)
        if status:
            self._fail(status)
        return out

    __call__ = forward


# ---------------------------------------------------------------------------
# gated block with 16-bit weights
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class GatedConfig:
    """Mirror of ``moe_gated_config``."""
    in_features: int
    out_features: int
    act: str = "swiglu"          # "swiglu" or "relu2" (no gate matrix)
    act_dtype: str = "bf16"
    max_tokens: int = 16
    training: bool = False

    def to_c(self) -> moe_gated_config:
        return moe_gated_config(
            in_features=_int32(self.in_features, "in_features"),
            out_features=_int32(self.out_features, "out_features"), act=_name_of(ACT, self.act, "act"),
            act_dtype=_name_of(DTYPE, self.act_dtype, "act_dtype"),
            max_tokens=_int32(self.max_tokens, "max_tokens"), training=int(bool(self.training)))


class GatedGrads(NamedTuple):
    """Gradients of one backward call (None where not asked for, or no gate)."""
    x: Any
    gate_w: Any
    up_w: Any


class GatedBlock(_Handle):
    """``silu(x Wg^T) * (x Wu^T)`` or ``max(x Wu^T, 0)^2`` over the caller's 16-bit weights, and its backward pass.

    No autograd function: ``requires_grad`` is not looked at, outputs carry no graph
    and no ``.grad`` is written; a training loop calls ``backward`` and hands its
    results on.
    """

    _prefix = "moe_gated"

    def __init__(self, config: GatedConfig, device=None):
        import torch
        self._setup(torch, load_library())
        self.config = config
        c = config.to_c()
        status = self._fn("validate")(ctypes.byref(c))
        if status != MOE_OK:
            raise MoEError(status, self._fn("last_error")(None).decode())
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if self.device.type != "cuda":
            raise MoEError(_INVALID_ARG, f"a gated block runs on a CUDA device, not on {self.device}")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._dtype = torch_act_dtype(config.act_dtype)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            status = self._fn("create")(ctypes.byref(c), ctypes.byref(h))
        if status != MOE_OK:
            raise MoEError(status, self._fn("last_error")(None).decode())
        self.handle = h.value
        self._call_forward, self._call_backward = self._lib.moe_gated_forward, self._lib.moe_gated_backward
        self._K, self._N, self._gated, self._f32 = config.in_features, config.out_features, config.act == "swiglu", torch.float32

    def _weights(self, up_w, gate_w) -> Tuple[int, Optional[int]]:
        pu = self._matrix(up_w, self._N, self._K, "up_w")
        if self._gated:
            return pu, self._matrix(gate_w, self._N, self._K, "gate_w")
        if gate_w is not None:
            raise MoEError(_SHAPE, "a squared-ReLU block takes no gate matrix")
        return pu, None

    def _forward(self, x, up_w, gate_w, out, stream, save: bool):
        N, device, empty = self._N, self.device, self._empty
        ldx = self._stride(x, self._K, "x")
        pu, pg = self._weights(up_w, gate_w)
        s, where = self._stream(stream, x, up_w, gate_w, out)
        T, ldo, g, u = x.shape[0], N, None, None
        if out is not None:
            ldo = self._stride(out, N, "out")
            if out.shape[0] != T:
                raise MoEError(_SHAPE, f"out has {out.shape[0]} rows, x {T}")
        with where:
            if out is None:
                out = empty((T, N), dtype=self._dtype, device=device)
            if save:
                u = empty((T, N), dtype=self._f32, device=device)
                if pg is not None:
                    g = empty((T, N), dtype=self._f32, device=device)
        status = self._call_forward(self.handle, x.data_ptr(), ldx, T, pg, pu, out.data_ptr(), ldo,
                                    None if g is None else g.data_ptr(), None if u is None else u.data_ptr(), s)
        if status:
            self._fail(status)
        return out, (g, u)

    def forward(self, x, up_w, gate_w=None, out=None, stream=None):
        """out [T, N] of x [T, K] (rows may be strided) and up_w, gate_w [N, K]."""
        return self._forward(x, up_w, gate_w, out, stream, False)[0]

    __call__ = forward

    def forward_train(self, x, up_w, gate_w=None, out=None, stream=None):
        """(out, saved): ``saved`` are the fp32 pre-activations (gate, up) that ``backward`` takes."""
        return self._forward(x, up_w, gate_w, out, stream, True)

    def backward(self, d_out, saved, x, up_w, gate_w=None, need=("x", "gate_w", "up_w"), stream=None) -> GatedGrads:
        """Gradients of the tensors named in ``need`` for the gradient ``d_out`` [T, N] of ``forward_train``'s out."""
        f32, device, dtype, empty = self._f32, self.device, self._dtype, self._empty
        for n in need:
            if n not in GatedGrads._fields:
                raise MoEError(_INVALID_ARG, f"need names {', '.join(GatedGrads._fields)}")
        K, N, T = self._K, self._N, x.shape[0]
        ldd, ldx = self._stride(d_out, N, "d_out"), self._stride(x, K, "x")
        pu, pg = self._weights(up_w, gate_w)
        if d_out.shape[0] != T:
            raise MoEError(_SHAPE, f"d_out has {d_out.shape[0]} rows, x {T}")
        ps = [None, None]
        for i, t in enumerate(saved):
            if i == 0 and pg is None:
                continue
            if (t is None or t.dtype is not f32 or t.shape != (T, N) or t.device != device or
                    not t.is_contiguous()):
                raise MoEError(_INVALID_ARG, "saved must be what forward_train returned for x")
            ps[i] = t.data_ptr()
        s, where = self._stream(stream, d_out, x, up_w, gate_w, *(saved if pg is not None else saved[1:]))
        with where:
            d_x = empty((T, K), dtype=dtype, device=device) if "x" in need else None
            d_g = empty((N, K), dtype=dtype, device=device) if pg is not None and "gate_w" in need else None
            d_u = empty((N, K), dtype=dtype, device=device) if "up_w" in need else None
        p = [None if t is None else t.data_ptr() for t in (d_x, d_g, d_u)]
        status = self._call_backward(self.handle, d_out.data_ptr(), ldd, T, x.data_ptr(), ldx, pg, pu, ps[0], ps[1],
                                     p[0], K, p[1], p[2], s)
        if status:
            self._fail(status)
        return GatedGrads(d_x, d_g, d_u)
