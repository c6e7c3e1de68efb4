"""ctypes binding of the 8-bit linear-layer calls of libns.so (include/ns.h,
ns_q8_*): argument checks and marshalling only.

A quantised matrix is a pair (q, scale): int8 values, rows x cols, and one
fp32 scale per row; `Q8Rows` names the two. Every call takes lists, one entry
per layer.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Sequence

from . import _binding
from ._binding import NS_BF16, NS_FP32, _check

Q8_ABSMAX, Q8_POW2 = 0, 1
Q8_MATMUL, Q8_GRAD_INPUT, Q8_GRAD_WEIGHT = 0, 1, 2
Q8_MAX_K = 131071

_i64, _vp = ctypes.c_int64, ctypes.c_void_p


class RowsStruct(ctypes.Structure):
    """ns_q8_rows"""
    _fields_ = [("rows", _i64), ("cols", _i64), ("values", _vp), ("ld_values", _i64), ("q", _vp), ("ld_q", _i64),
                ("scale", _vp)]


class LayerStruct(ctypes.Structure):
    """ns_q8_layer"""
    _fields_ = [("tokens", _i64), ("out_features", _i64), ("in_features", _i64),
                ("xq", _vp), ("ld_xq", _i64), ("x_scale", _vp),
                ("wq", _vp), ("ld_wq", _i64), ("w_scale", _vp),
                ("dy", _vp), ("ld_dy", _i64), ("out", _vp), ("ld_out", _i64)]


class Q8Rows(NamedTuple):
    """An 8-bit matrix: row r stands for q[r] * scale[r]."""
    q: "torch.Tensor"       # int8, rows x cols  # noqa: F821
    scale: "torch.Tensor"   # float32, rows      # noqa: F821


_declared: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    global _declared
    if _declared is None:
        L = _binding.lib()
        i32, size = ctypes.c_int32, ctypes.c_size_t
        rows, layers = ctypes.POINTER(RowsStruct), ctypes.POINTER(LayerStruct)
        L.ns_q8_quantize.argtypes = [rows, i32, i32, i32, _vp]
        L.ns_q8_dequantize.argtypes = [rows, i32, i32, _vp]
        L.ns_q8_matmul.argtypes = [layers, i32, i32, _vp, size, _vp]
        L.ns_q8_grad_input.argtypes = [layers, i32, _vp, size, _vp]
        L.ns_q8_grad_weight.argtypes = [layers, i32, ctypes.c_float, i32, _vp, size, _vp]
        L.ns_q8_workspace_bytes.argtypes = [i32, layers, i32, i32, ctypes.POINTER(size)]
        for name in ("quantize", "dequantize", "matmul", "grad_input", "grad_weight", "workspace_bytes"):
            getattr(L, "ns_q8_" + name).restype = ctypes.c_int
        _declared = L
    return _declared


def _code(dtype) -> int:
    import torch
    if dtype == torch.bfloat16:
        return NS_BF16
    if dtype == torch.float32:
        return NS_FP32
    raise TypeError(f"unsupported dtype {dtype}; use bfloat16 or float32")


class _Call:
    """What the tensors of one call share: their device, and the stream."""

    def __init__(self, stream):
        self.stream, self.device, self.seen = stream, None, []

    def matrix(self, t, name: str, dtype) -> None:
        if t.dim() != 2:
            raise ValueError(f"{name} must be 2-D")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
        if t.numel() and t.shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"the rows of {name} must be contiguous")
        if t.shape[0] > 1 and t.numel() and t.stride(0) < t.shape[1]:
            raise ValueError(f"the rows of {name} overlap")
        self.on_device(t, name)

    def rows(self, pair, name: str):
        q, scale = pair
        import torch
        self.matrix(q, name, torch.int8)
        if scale.dim() != 1 or scale.shape[0] != q.shape[0] or scale.dtype != torch.float32:
            raise ValueError(f"{name} needs one float32 scale per row")
        if scale.numel() > 1 and scale.stride(0) != 1:
            raise ValueError(f"the scales of {name} must be contiguous")
        self.on_device(scale, name)
        return q, scale

    def on_device(self, t, name: str) -> None:
        if self.device is None:
            self.device = t.device
        if t.device != self.device or self.device.type != "cuda":
            raise ValueError(f"{name}: all tensors of a call must be on the same CUDA device")
        self.seen.append(t)

    def enter(self):
        """The stream, with the device and (so that what the call allocates
        belongs to it) that stream current."""
        import contextlib

        import torch
        stack = contextlib.ExitStack()
        if torch.cuda.current_device() != self.device.index:
            stack.enter_context(torch.cuda.device(self.device))
        if self.stream is None:
            return stack, torch.cuda.current_stream()
        if self.stream.device != self.device:
            raise ValueError("the stream is on another device than the tensors")
        if self.stream != torch.cuda.current_stream():
            # memory that the caller frees early stays theirs until the
            # stream has used it
            for t in self.seen:
                t.record_stream(self.stream)
        stack.enter_context(torch.cuda.stream(self.stream))
        return stack, self.stream


def _ptr(t):
    return t.data_ptr() if t.numel() else None


def _ld(t) -> int:
    return t.stride(0) if t.shape[0] > 1 else max(1, t.shape[1])


def quantize_rows(tensors: Sequence, pow2: bool = False, stream=None):
    """Rows to 8 bits (ns_q8_quantize): a list of 2-D bf16 or fp32 tensors (all
    of one dtype; rows contiguous, at any pitch) to a list of `Q8Rows`, whose q
    lies at a pitch of a multiple of 16 bytes. pow2: scales that are powers of
    two, with which products with bf16 values are exact. For a layer's
    input this is its checkpoint for q8_grad_weight; for its weights, the
    channels' form for q8_matmul and q8_grad_input."""
    import torch
    tensors = list(tensors)
    if not tensors:
        return []
    dt = tensors[0].dtype
    code = _code(dt)
    call = _Call(stream)
    for t in tensors:
        call.matrix(t, "every matrix", dt)
    stack, s = call.enter()
    with stack:
        out = []
        arr = (RowsStruct * len(tensors))()
        for i, t in enumerate(tensors):
            rows, cols = t.shape
            q = torch.empty((rows, -(-cols // 16) * 16), dtype=torch.int8, device=t.device)[:, :cols]
            scale = torch.empty(rows, dtype=torch.float32, device=t.device)
            if cols == 0:
                scale.fill_(2.0 ** -126)
            out.append(Q8Rows(q, scale))
            arr[i] = RowsStruct(rows, cols, _ptr(t), _ld(t), _ptr(q), _ld(q), _ptr(scale))
        _check(lib().ns_q8_quantize(arr, len(tensors), Q8_POW2 if pow2 else Q8_ABSMAX, code, s.cuda_stream))
    return out


def dequantize_rows(matrices: Sequence, dtype=None, stream=None):
    """The values of 8-bit matrices ((q, scale) pairs) as a list of tensors of
    `dtype` (default bf16) (ns_q8_dequantize)."""
    import torch
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _code(dtype)
    call = _Call(stream)
    pairs = [call.rows(m, "every matrix") for m in matrices]
    if not pairs:
        return []
    stack, s = call.enter()
    with stack:
        out = []
        arr = (RowsStruct * len(pairs))()
        for i, (q, scale) in enumerate(pairs):
            v = torch.empty(q.shape, dtype=dtype, device=q.device)
            out.append(v)
            arr[i] = RowsStruct(q.shape[0], q.shape[1], _ptr(v), _ld(v), _ptr(q), _ld(q), _ptr(scale))
        _check(lib().ns_q8_dequantize(arr, len(pairs), code, s.cuda_stream))
    return out


def _product(call: _Call, op: int, layers, outs, dtype, code: int, beta: float = 0.0):
    """Runs one product over `layers`, a list of (tokens, out, in, x pair or
    None, w pair or None, dy or None); `outs` holds the outputs, or None for
    new ones."""
    import torch
    n = len(layers)
    stack, s = call.enter()
    with stack:
        arr = (LayerStruct * n)()
        made = [] if outs is None else outs
        for i, (t, o, k, x, w, dy) in enumerate(layers):
            if outs is None:
                shape = (t, o) if op == Q8_MATMUL else (t, k)
                made.append(torch.empty(shape, dtype=dtype, device=call.device))
            a, out = arr[i], made[i]
            a.tokens, a.out_features, a.in_features = t, o, k
            if x is not None:
                a.xq, a.ld_xq, a.x_scale = _ptr(x[0]), _ld(x[0]), _ptr(x[1])
            if w is not None:
                a.wq, a.ld_wq, a.w_scale = _ptr(w[0]), _ld(w[0]), _ptr(w[1])
            if dy is not None:
                a.dy, a.ld_dy = _ptr(dy), _ld(dy)
            a.out, a.ld_out = _ptr(out), _ld(out)
        L = lib()
        need = ctypes.c_size_t(0)
        _check(L.ns_q8_workspace_bytes(op, arr, n, code, ctypes.byref(need)))
        # a block of the caching allocator: the call's own until it has run on
        # this stream, also inside a captured graph
        ws = torch.empty(need.value, dtype=torch.uint8, device=call.device) if need.value else None
        wp = None if ws is None else ws.data_ptr()
        if op == Q8_MATMUL:
            rc = L.ns_q8_matmul(arr, n, code, wp, need.value, s.cuda_stream)
        elif op == Q8_GRAD_INPUT:
            rc = L.ns_q8_grad_input(arr, n, wp, need.value, s.cuda_stream)
        else:
            rc = L.ns_q8_grad_weight(arr, n, beta, code, wp, need.value, s.cuda_stream)
        _check(rc)
    return made


def _outputs(call: _Call, out, shapes, dtype):
    if out is None:
        return None
    out = list(out)
    if len(out) != len(shapes):
        raise ValueError("one output per layer is needed")
    for t, shape in zip(out, shapes):
        call.matrix(t, "an output", dtype)
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"an output is {tuple(t.shape)}, its layer needs {tuple(shape)}")
    return out


def _same_length(*lists):
    if len({len(v) for v in lists}) != 1:
        raise ValueError("one entry per layer is needed in every list")


def q8_matmul(xs: Sequence, ws: Sequence, dtype=None, out=None, stream=None):
    """Y = X W^T of 8-bit layers (ns_q8_matmul): `xs` holds (q, scale) pairs of
    tokens x in, `ws` of out x in. Returns a list of tokens x out tensors of
    `dtype` (default bf16), new ones or those of `out`."""
    import torch
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _code(dtype)
    xs, ws = list(xs), list(ws)
    _same_length(xs, ws)
    if not xs:
        return []
    call = _Call(stream)
    layers = []
    for x, w in zip(xs, ws):
        x, w = call.rows(x, "x"), call.rows(w, "w")
        if x[0].shape[1] != w[0].shape[1]:
            raise ValueError(f"x has {x[0].shape[1]} columns, w {w[0].shape[1]}")
        layers.append((x[0].shape[0], w[0].shape[0], x[0].shape[1], x, w, None))
    outs = _outputs(call, out, [(t, o) for t, o, *_ in layers], dtype)
    return _product(call, Q8_MATMUL, layers, outs, dtype, code)


def q8_grad_input(dys: Sequence, ws: Sequence, out=None, stream=None):
    """dX = dY W of 8-bit layers (ns_q8_grad_input): `dys` holds bf16 tensors of
    tokens x out, `ws` (q, scale) pairs of out x in. Returns a list of
    tokens x in bf16 tensors, new ones or those of `out`."""
    import torch
    dys, ws = list(dys), list(ws)
    _same_length(dys, ws)
    if not dys:
        return []
    call = _Call(stream)
    layers = []
    for dy, w in zip(dys, ws):
        call.matrix(dy, "dy", torch.bfloat16)
        w = call.rows(w, "w")
        if dy.shape[1] != w[0].shape[0]:
            raise ValueError(f"dy has {dy.shape[1]} columns, w {w[0].shape[0]} rows")
        layers.append((dy.shape[0], dy.shape[1], w[0].shape[1], None, w, dy))
    outs = _outputs(call, out, [(t, k) for t, _, k, *_ in layers], torch.bfloat16)
    return _product(call, Q8_GRAD_INPUT, layers, outs, torch.bfloat16, NS_BF16)


def q8_grad_weight(dys: Sequence, xs: Sequence, grads: Sequence, beta: float = 0.0, stream=None):
    """G <- beta G + dY^T X in place (ns_q8_grad_weight): `dys` holds bf16
    tensors of tokens x out, `xs` the layers' inputs as (q, scale) pairs of
    tokens x in, `grads` out x in tensors, all bf16 or all fp32, not read when
    beta == 0. Returns the list of `grads`, which `orthogonalize` takes as it
    is when they are contiguous."""
    import torch
    dys, xs, grads = list(dys), list(xs), list(grads)
    _same_length(dys, xs, grads)
    if not dys:
        return grads
    code = _code(grads[0].dtype)
    call = _Call(stream)
    layers = []
    for dy, x in zip(dys, xs):
        call.matrix(dy, "dy", torch.bfloat16)
        x = call.rows(x, "x")
        if dy.shape[0] != x[0].shape[0]:
            raise ValueError(f"dy has {dy.shape[0]} rows, x {x[0].shape[0]}")
        layers.append((dy.shape[0], dy.shape[1], x[0].shape[1], x, None, dy))
    outs = _outputs(call, grads, [(o, k) for _, o, k, *_ in layers], grads[0].dtype)
    return _product(call, Q8_GRAD_WEIGHT, layers, outs, grads[0].dtype, code, beta)
