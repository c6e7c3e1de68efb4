"""ctypes binding of the 8-bit linear-layer calls of libns.so (include/ns.h,
ns_q8_*): argument checks and marshalling only.

A quantised matrix is a pair (q, scale): int8 values, rows x cols, and one
fp32 scale per row; `Q8Rows` names the two. Every call takes lists, one entry
per layer.
"""
from __future__ import annotations

import contextlib
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
        # (lists of structs go as the address of an array of their 8-byte members)
        L.ns_q8_quantize.argtypes = [_vp, i32, i32, i32, _vp]
        L.ns_q8_dequantize.argtypes = [_vp, i32, i32, _vp]
        L.ns_q8_matmul.argtypes = [_vp, i32, i32, _vp, size, _vp]
        L.ns_q8_grad_input.argtypes = [_vp, i32, _vp, size, _vp]
        L.ns_q8_grad_weight.argtypes = [_vp, i32, ctypes.c_float, i32, _vp, size, _vp]
        L.ns_q8_workspace_bytes.argtypes = [i32, _vp, i32, i32, ctypes.POINTER(size)]
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
    """The tensors of one call: checked one by one, on one device. Matrices
    come back as (rows, cols, pitch, address), the address 0 when empty."""

    def __init__(self, device):
        if device.type != "cuda":
            raise ValueError("all tensors of a call must be on the same CUDA device")
        self.device, self.seen = device, []

    def matrix(self, t, name: str, dtype):
        shape, stride = t.shape, t.stride()
        if len(shape) != 2:
            raise ValueError(f"{name} must be 2-D")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
        if t.device != self.device:
            raise ValueError(f"{name}: all tensors of a call must be on the same CUDA device")
        self.seen.append(t)
        rows, cols = shape
        if rows == 0 or cols == 0:
            return rows, cols, max(1, cols), 0
        if cols > 1 and stride[1] != 1:
            raise ValueError(f"the rows of {name} must be contiguous")
        pitch = cols
        if rows > 1:
            pitch = stride[0]
            if pitch < cols:
                raise ValueError(f"the rows of {name} overlap")
        return rows, cols, pitch, t.data_ptr()

    def rows(self, pair, name: str):
        """Of a (q, scale) pair: q's (rows, cols, pitch, address), and the
        address of the scales."""
        import torch
        q, scale = pair
        m = self.matrix(q, name, torch.int8)
        shape = scale.shape
        if len(shape) != 1 or shape[0] != m[0] or scale.dtype != torch.float32:
            raise ValueError(f"{name} needs one float32 scale per row")
        if shape[0] > 1 and scale.stride(0) != 1:
            raise ValueError(f"the scales of {name} must be contiguous")
        if scale.device != self.device:
            raise ValueError(f"{name}: all tensors of a call must be on the same CUDA device")
        self.seen.append(scale)
        return m, scale.data_ptr()

    def enter(self, stream):
        """A context in which the device and the stream are current, so that
        what the call allocates belongs to them, and the stream's handle."""
        import torch
        stack = contextlib.nullcontext()
        index = self.device.index
        if stream is not None:
            if stream.device != self.device:
                raise ValueError("the stream is on another device than the tensors")
            if stream != torch.cuda.current_stream(self.device):
                # memory that the caller frees early stays theirs until the
                # stream has used it
                for t in self.seen:
                    t.record_stream(stream)
            return torch.cuda.stream(stream), stream.cuda_stream
        if torch.cuda.current_device() != index:
            stack = torch.cuda.device(self.device)
        return stack, torch.cuda.current_stream(self.device).cuda_stream


def _int64s(values):
    return (_i64 * len(values))(*values)


def quantize_rows(tensors: Sequence, pow2: bool = False, stream=None):
    """Rows to 8 bits (ns_q8_quantize): a list of 2-D bf16 or fp32 tensors (all
    of one dtype; rows contiguous, at any pitch) to a list of `Q8Rows`, whose q
    lies at a pitch of a multiple of 16 bytes. pow2: scales that are powers of
    two, with which products with bf16 values are exact. For a layer's input
    this is its checkpoint for q8_grad_weight; for its weights, the channels'
    form for q8_matmul and q8_grad_input."""
    import torch
    tensors = list(tensors)
    if not tensors:
        return []
    dt, device = tensors[0].dtype, tensors[0].device
    code = _code(dt)
    call = _Call(device)
    mats = [call.matrix(t, "every matrix", dt) for t in tensors]
    context, handle = call.enter(stream)
    with context:
        out, flat = [], []
        for rows, cols, pitch, at in mats:
            ld = (cols + 15) // 16 * 16
            q = torch.empty_strided((rows, cols), (ld, 1), dtype=torch.int8, device=device)
            scale = torch.empty(rows, dtype=torch.float32, device=device)
            if cols == 0:
                scale.fill_(2.0 ** -126)
            out.append(Q8Rows(q, scale))
            flat += (rows, cols, at, pitch, q.data_ptr(), ld or 1, scale.data_ptr())
        _check(lib().ns_q8_quantize(_int64s(flat), len(mats), Q8_POW2 if pow2 else Q8_ABSMAX, code, handle))
    return out


def dequantize_rows(matrices: Sequence, dtype=None, stream=None):
    """The values of 8-bit matrices ((q, scale) pairs) as a list of tensors of
    `dtype` (default bf16) (ns_q8_dequantize)."""
    import torch
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _code(dtype)
    matrices = list(matrices)
    if not matrices:
        return []
    device = matrices[0][0].device
    call = _Call(device)
    pairs = [call.rows(m, "every matrix") for m in matrices]
    context, handle = call.enter(stream)
    with context:
        out, flat = [], []
        for (rows, cols, pitch, at), scale in pairs:
            v = torch.empty((rows, cols), dtype=dtype, device=device)
            out.append(v)
            flat += (rows, cols, v.data_ptr(), cols or 1, at, pitch, scale)
        _check(lib().ns_q8_dequantize(_int64s(flat), len(pairs), code, handle))
    return out


def _product(call: _Call, op: int, layers, outs, shapes, dtype, code: int, stream, beta: float = 0.0):
    """Runs one product over `layers`, their ns_q8_layer members up to `out`;
    `outs` holds the outputs, or None for new ones of `shapes`."""
    import torch
    n = len(layers)
    if outs is not None:
        outs = list(outs)
        if len(outs) != n:
            raise ValueError("one output per layer is needed")
        for t, shape in zip(outs, shapes):
            if tuple(t.shape) != shape:
                raise ValueError(f"an output is {tuple(t.shape)}, its layer needs {shape}")
        spots = [call.matrix(t, "an output", dtype) for t in outs]
    context, handle = call.enter(stream)
    with context:
        if outs is None:
            outs = [torch.empty(shape, dtype=dtype, device=call.device) for shape in shapes]
            spots = [(0, 0, shape[1] or 1, t.data_ptr()) for t, shape in zip(outs, shapes)]
        flat = []
        for members, (_, _, pitch, at) in zip(layers, spots):
            flat += members
            flat += (at, pitch)
        arr = _int64s(flat)
        L = lib()
        need = ctypes.c_size_t(0)
        _check(L.ns_q8_workspace_bytes(op, arr, n, code, ctypes.byref(need)))
        size, ws = need.value, None
        if size:
            # a block of the caching allocator: the call's own until it has run
            # on this stream, also inside a captured graph
            block = torch.empty(size, dtype=torch.uint8, device=call.device)
            ws = block.data_ptr()
        if op == Q8_MATMUL:
            rc = L.ns_q8_matmul(arr, n, code, ws, size, handle)
        elif op == Q8_GRAD_INPUT:
            rc = L.ns_q8_grad_input(arr, n, ws, size, handle)
        else:
            rc = L.ns_q8_grad_weight(arr, n, beta, code, ws, size, handle)
        _check(rc)
    return outs


def _same_length(*lists):
    if len({len(v) for v in lists}) != 1:
        raise ValueError("one entry per layer is needed in every list")


_NONE = (0, 0, 0)


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
    call = _Call(xs[0][0].device)
    layers, shapes = [], []
    for x, w in zip(xs, ws):
        (t, k, ldx, xq), x_scale = call.rows(x, "x")
        (o, kw, ldw, wq), w_scale = call.rows(w, "w")
        if k != kw:
            raise ValueError(f"x has {k} columns, w {kw}")
        layers.append((t, o, k, xq, ldx, x_scale, wq, ldw, w_scale, 0, 0))
        shapes.append((t, o))
    return _product(call, Q8_MATMUL, layers, out, shapes, dtype, code, stream)


def q8_grad_input(dys: Sequence, ws: Sequence, out=None, stream=None):
    """dX = dY W of 8-bit layers (ns_q8_grad_input): `dys` holds bf16 tensors of
    tokens x out, `ws` (q, scale) pairs of out x in. Returns a list of
    tokens x in bf16 tensors, new ones or those of `out`."""
    import torch
    dys, ws = list(dys), list(ws)
    _same_length(dys, ws)
    if not dys:
        return []
    call = _Call(dys[0].device)
    layers, shapes = [], []
    for dy, w in zip(dys, ws):
        t, o, ldd, dyp = call.matrix(dy, "dy", torch.bfloat16)
        (ow, k, ldw, wq), w_scale = call.rows(w, "w")
        if o != ow:
            raise ValueError(f"dy has {o} columns, w {ow} rows")
        layers.append((t, o, k, *_NONE, wq, ldw, w_scale, dyp, ldd))
        shapes.append((t, k))
    return _product(call, Q8_GRAD_INPUT, layers, out, shapes, torch.bfloat16, NS_BF16, stream)


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
    dtype = grads[0].dtype
    code = _code(dtype)
    call = _Call(dys[0].device)
    layers, shapes = [], []
    for dy, x in zip(dys, xs):
        t, o, ldd, dyp = call.matrix(dy, "dy", torch.bfloat16)
        (tx, k, ldx, xq), x_scale = call.rows(x, "x")
        if t != tx:
            raise ValueError(f"dy has {t} rows, x {tx}")
        layers.append((t, o, k, xq, ldx, x_scale, *_NONE, dyp, ldd))
        shapes.append((o, k))
    return _product(call, Q8_GRAD_WEIGHT, layers, grads, shapes, dtype, code, stream, beta)
