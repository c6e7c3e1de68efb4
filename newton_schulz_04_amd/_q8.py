"""ctypes binding of the 8-bit linear-layer calls of libns.so (include/ns.h,
ns_q8_*): argument checks and marshalling only.

A quantised matrix is a pair (q, scale): int8 values, rows x cols, and one
fp32 scale per row; `Q8Rows` names the two. Every call takes lists, one entry
per layer.

The calls are the pieces that a layer's autograd.Function is written from; they
have no gradients of their own. In grad mode a tensor that requires grad is
refused, as its gradient would be lost without a word: under torch.no_grad() and
in an autograd.Function's methods all are taken. Tensors that a call writes to
(`out`, `grads`) count it as a change in place.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
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


_SAME_DEVICE = "all tensors of a call must be on the same CUDA device"


def _on_cuda(device):
    if device.type != "cuda":
        raise ValueError(_SAME_DEVICE)
    return device


def _refuse_grad(name: str):
    import torch
    if torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad, and this call has no gradient: call it under torch.no_grad() or in an "
                         "autograd.Function")


def _matrix(t, name: str, dtype, device):
    """Checks a matrix of a call; its (rows, cols, pitch, address), the
    address 0 when it is empty."""
    if t.requires_grad:
        _refuse_grad(name)
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != device.index:   # (-1 on the CPU)
        raise ValueError(f"{name}: {_SAME_DEVICE}")
    rows, cols = shape
    if rows == 0 or cols == 0:
        return rows, cols, cols or 1, 0
    pitch, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if rows == 1:
        pitch = cols
    elif pitch < cols:
        raise ValueError(f"the rows of {name} overlap")
    return rows, cols, pitch, t.data_ptr()


def _pair(pair, name: str, device, int8, float32):
    """Checks a (q, scale) pair; q's _matrix and the address of the scales."""
    q, scale = pair
    m = _matrix(q, name, int8, device)
    if scale.requires_grad:
        _refuse_grad(f"the scale of {name}")
    shape = scale.shape
    if len(shape) != 1 or shape[0] != m[0] or scale.dtype != float32:
        raise ValueError(f"{name} needs one float32 scale per row")
    if shape[0] > 1 and scale.stride(0) != 1:
        raise ValueError(f"the scales of {name} must be contiguous")
    if scale.get_device() != device.index:
        raise ValueError(f"{name}: {_SAME_DEVICE}")
    return m, scale.data_ptr()


_NO_CONTEXT = contextlib.nullcontext()


def _enter(device, stream, tensors):
    """A context that makes the tensors' device and the stream current, so
    that what a call allocates belongs to them, and the stream's handle.
    `tensors` gives all that the call reads or writes and the caller holds."""
    import torch
    if stream is None:
        here = torch.cuda.current_device() == device.index
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        handle = raw(device.index) if raw else torch.cuda.current_stream(device).cuda_stream
        return _NO_CONTEXT if here else torch.cuda.device(device), handle
    if stream.device != device:
        raise ValueError("the stream is on another device than the tensors")
    if stream != torch.cuda.current_stream(device):
        # memory that the caller frees early stays theirs until the stream
        # has used it
        for t in tensors():
            t.record_stream(stream)
    return torch.cuda.stream(stream), stream.cuda_stream


def _int64s(values):
    return (_i64 * len(values))(*values)


def _empty(shapes, dtype, device):
    """New contiguous tensors of `shapes`, aligned to 16 bytes; one block for
    several of one width, with rows between them where the alignment needs
    some. (unsafe_split: tensors of their own to autograd, not views of the
    block that could not be modified in place.)"""
    import torch
    n, width = len(shapes), shapes[0][1]
    if n > 1 and width > 0 and all(s[1] == width for s in shapes):
        unit = 16 // math.gcd(width * dtype.itemsize, 16)
        parts = [m for rows, _ in shapes for m in (rows, -rows % unit)]
        return torch.unsafe_split_with_sizes(torch.empty((sum(parts), width), dtype=dtype, device=device), parts)[::2]
    return [torch.empty(s, dtype=dtype, device=device) for s in shapes]


def quantize_rows(tensors: Sequence, pow2: bool = False, stream=None):
    """Rows to 8 bits (ns_q8_quantize): a list of 2-D bf16 or fp32 tensors (all
    of one dtype; rows contiguous, at any pitch) to a list of `Q8Rows`, whose q
    lies at a pitch of a multiple of 16 bytes. pow2: scales that are powers of
    two, up to one bit coarser, with which q8_grad_input and q8_grad_weight take
    about half of the time (fp32 gradients: a third). For a layer's input
    this is its checkpoint for q8_grad_weight; for its weights, the channels'
    form for q8_matmul and q8_grad_input. The results of a list of equal
    shapes share one block of memory, which lives as long as any of them."""
    import torch
    tensors = list(tensors)
    if not tensors:
        return []
    first = tensors[0]
    dt, n = first.dtype, len(tensors)
    code, device = _code(dt), _on_cuda(first.device)
    mats = [_matrix(t, "every matrix", dt, device) for t in tensors]
    context, handle = _enter(device, stream, lambda: tensors)
    with context:
        rows, cols = mats[0][:2]
        if n > 1 and rows > 0 and all(m[0] == rows and m[1] == cols for m in mats):
            ld = (cols + 15) // 16 * 16
            qs = torch.unsafe_split(
                torch.empty_strided((n * rows, cols), (ld, 1), dtype=torch.int8, device=device), rows)
            scales = torch.unsafe_split(torch.empty(n * rows, dtype=torch.float32, device=device), rows)
        else:
            lds = [(m[1] + 15) // 16 * 16 for m in mats]
            qs = [torch.empty_strided(m[:2], (ld, 1), dtype=torch.int8, device=device) for m, ld in zip(mats, lds)]
            scales = [torch.empty(m[0], dtype=torch.float32, device=device) for m in mats]
        flat = []
        for (rows, cols, pitch, at), q, scale in zip(mats, qs, scales):
            if cols == 0:
                scale.fill_(2.0 ** -126)
            flat += (rows, cols, at, pitch, q.data_ptr(), (cols + 15) // 16 * 16 or 1, scale.data_ptr())
        _check(lib().ns_q8_quantize(_int64s(flat), n, Q8_POW2 if pow2 else Q8_ABSMAX, code, handle))
    return [Q8Rows(q, scale) for q, scale in zip(qs, scales)]


def dequantize_rows(matrices: Sequence, dtype=None, stream=None):
    """The values of 8-bit matrices ((q, scale) pairs) as a list of tensors of
    `dtype` (default bf16) (ns_q8_dequantize). Here and in the products, the new
    tensors of a list of one width may share one block of memory."""
    import torch
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _code(dtype)
    matrices = list(matrices)
    if not matrices:
        return []
    device = _on_cuda(matrices[0][0].device)
    int8, float32 = torch.int8, torch.float32
    pairs = [_pair(m, "every matrix", device, int8, float32) for m in matrices]
    context, handle = _enter(device, stream, lambda: [t for m in matrices for t in m])
    with context:
        out = _empty([m[:2] for m, _ in pairs], dtype, device)
        flat = []
        for ((rows, cols, pitch, at), scale), v in zip(pairs, out):
            flat += (rows, cols, v.data_ptr(), cols or 1, at, pitch, scale)
        _check(lib().ns_q8_dequantize(_int64s(flat), len(pairs), code, handle))
    return out


def _product(op: int, layers, out, shapes, dtype, code: int, device, stream, tensors, beta: float = 0.0):
    """Runs one product over `layers`, their ns_q8_layer members up to `out`,
    into the tensors `out`, or new ones of `shapes`."""
    import torch
    n, given = len(layers), ()
    if out is not None:
        out = list(out)
        if len(out) != n:
            raise ValueError("one output per layer is needed")
        spots = [_matrix(t, "an output", dtype, device) for t in out]
        given = out
        for m, shape in zip(spots, shapes):
            if m[:2] != shape:
                raise ValueError(f"an output is {m[:2]}, its layer needs {shape}")
    context, handle = _enter(device, stream, lambda: [*tensors(), *(out or ())])
    with context:
        if out is None:
            out = _empty(shapes, dtype, device)
            spots = [(*s, s[1] or 1, t.data_ptr()) for t, s in zip(out, shapes)]
        flat = []
        for members, m in zip(layers, spots):
            flat += members
            flat += (m[3], m[2])
        arr, L = _int64s(flat), lib()

        def call(ws, size):
            if op == Q8_MATMUL:
                return L.ns_q8_matmul(arr, n, code, ws, size, handle)
            if op == Q8_GRAD_INPUT:
                return L.ns_q8_grad_input(arr, n, ws, size, handle)
            return L.ns_q8_grad_weight(arr, n, beta, code, ws, size, handle)

        # most calls need no workspace; one that does is refused without it,
        # with nothing enqueued
        rc = call(None, 0)
        if rc:
            need = ctypes.c_size_t(0)
            if rc == 1 and L.ns_q8_workspace_bytes(op, arr, n, code, ctypes.byref(need)) == 0 and need.value:
                # a block of the caching allocator: the call's own until it
                # has run on this stream, also inside a captured graph
                block = torch.empty(need.value, dtype=torch.uint8, device=device)
                rc = call(block.data_ptr(), need.value)
            _check(rc)
    if given:
        torch.autograd.graph.increment_version(given)
    return out


_LENGTHS = "one entry per layer is needed in every list"


def q8_matmul(xs: Sequence, ws: Sequence, dtype=None, out=None, stream=None):
    """Y = X W^T of 8-bit layers (ns_q8_matmul): `xs` holds (q, scale) pairs of
    tokens x in, `ws` of out x in. Returns a list of tokens x out tensors of
    `dtype` (default bf16), new ones or those of `out`."""
    import torch
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _code(dtype)
    xs, ws = list(xs), list(ws)
    if len(xs) != len(ws):
        raise ValueError(_LENGTHS)
    if not xs:
        return []
    device = _on_cuda(xs[0][0].device)
    int8, float32 = torch.int8, torch.float32
    layers, shapes = [], []
    for x, w in zip(xs, ws):
        (t, k, ldx, xq), x_scale = _pair(x, "x", device, int8, float32)
        (o, kw, ldw, wq), w_scale = _pair(w, "w", device, int8, float32)
        if k != kw:
            raise ValueError(f"x has {k} columns, w {kw}")
        layers.append((t, o, k, xq, ldx, x_scale, wq, ldw, w_scale, 0, 0))
        shapes.append((t, o))
    return _product(Q8_MATMUL, layers, out, shapes, dtype, code, device, stream,
                    lambda: [t for pair in (*xs, *ws) for t in pair])


def q8_grad_input(dys: Sequence, ws: Sequence, out=None, stream=None):
    """dX = dY W of 8-bit layers (ns_q8_grad_input): `dys` holds bf16 tensors of
    tokens x out, `ws` (q, scale) pairs of out x in. Returns a list of
    tokens x in bf16 tensors, new ones or those of `out`. W enters with 16 bits
    of q s at least, all of them where its scales are powers of two, which is
    also twice as fast."""
    import torch
    dys, ws = list(dys), list(ws)
    if len(dys) != len(ws):
        raise ValueError(_LENGTHS)
    if not dys:
        return []
    device = _on_cuda(dys[0].device)
    int8, float32, bfloat16 = torch.int8, torch.float32, torch.bfloat16
    layers, shapes = [], []
    for dy, w in zip(dys, ws):
        t, o, ldd, dyp = _matrix(dy, "dy", bfloat16, device)
        (ow, k, ldw, wq), w_scale = _pair(w, "w", device, int8, float32)
        if o != ow:
            raise ValueError(f"dy has {o} columns, w {ow} rows")
        layers.append((t, o, k, 0, 0, 0, wq, ldw, w_scale, dyp, ldd))
        shapes.append((t, k))
    return _product(Q8_GRAD_INPUT, layers, out, shapes, bfloat16, NS_BF16, device, stream,
                    lambda: [*dys, *(t for pair in ws for t in pair)])


def q8_grad_weight(dys: Sequence, xs: Sequence, grads: Sequence, beta: float = 0.0, stream=None):
    """G <- beta G + dY^T X in place (ns_q8_grad_weight): `dys` holds bf16
    tensors of tokens x out, `xs` the layers' inputs as (q, scale) pairs of
    tokens x in, `grads` out x in tensors, all bf16 or all fp32, not read when
    beta == 0. Returns the list of `grads`, which `orthogonalize` takes as it
    is when they are contiguous. X enters with all 24 bits of q s for fp32
    gradients, with 16 at least for bf16 ones; where its scales are powers of
    two, q s has no more than 8, and the product takes a third or half of the
    time."""
    import torch
    dys, xs, grads = list(dys), list(xs), list(grads)
    if not len(dys) == len(xs) == len(grads):
        raise ValueError(_LENGTHS)
    if not dys:
        return grads
    dtype = grads[0].dtype
    code = _code(dtype)
    device = _on_cuda(dys[0].device)
    int8, float32, bfloat16 = torch.int8, torch.float32, torch.bfloat16
    layers, shapes = [], []
    for dy, x in zip(dys, xs):
        t, o, ldd, dyp = _matrix(dy, "dy", bfloat16, device)
        (tx, k, ldx, xq), x_scale = _pair(x, "x", device, int8, float32)
        if t != tx:
            raise ValueError(f"dy has {t} rows, x {tx}")
        layers.append((t, o, k, xq, ldx, x_scale, 0, 0, 0, dyp, ldd))
        shapes.append((o, k))
    return _product(Q8_GRAD_WEIGHT, layers, grads, shapes, dtype, code, device, stream,
                    lambda: [*dys, *(t for pair in xs for t in pair)], beta)
