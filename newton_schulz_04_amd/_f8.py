"""ctypes binding of the 8-bit floating-point calls of libns.so (include/ns.h,
ns_f8_*): argument checks and marshalling only.

An 8-bit matrix is a pair (q, scale), `F8Blocks`: q of float8_e4m3fn or float8_e5m2,
rows x cols, and scales of float32, or of float8_e8m0fnu (powers of two, one byte), for
blocks of 128 columns: ceil(cols / 128) x rows, or ceil(cols / 128) x ceil(rows / 128)
for squares of 128 x 128. Every call takes lists.

The calls are the pieces that a layer's autograd.Function is written from; they have
no gradients of their own. In grad mode a tensor that requires grad is refused, as its
gradient would be lost without a word: under torch.no_grad() and in an
autograd.Function's methods all are taken. Tensors that a call writes to (`out`) count
it as a change in place.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Sequence

from . import _binding
from ._binding import _check
from ._q8 import _code, _empty, _enter, _int64s, _LENGTHS, _matrix, _on_cuda, _refuse_grad, _SAME_DEVICE

F8_E4M3, F8_E5M2 = 0, 1
F8_SCALE_FP32, F8_SCALE_POW2 = 0, 1
F8_BLOCK = 128
_FORMS = ("rows", "transposed", "both")

_vp = ctypes.c_void_p


class F8Blocks(NamedTuple):
    """An 8-bit matrix: value (r, c) stands for q[r, c] * scale[c // 128, r], or
    * scale[c // 128, r // 128] for squares. Ranges of rows and of whole blocks of columns
    may be sliced out of it: q at addresses and pitches of a multiple of 16, one-byte
    scales at those of a multiple of 4."""
    q: "torch.Tensor"       # float8, rows x cols  # noqa: F821
    scale: "torch.Tensor"   # float32 or float8_e8m0fnu  # noqa: F821


_declared: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    global _declared
    if _declared is None:
        L = _binding.lib()
        i32, size = ctypes.c_int32, ctypes.c_size_t
        # (lists of structs go as the address of an array of their 8-byte members)
        L.ns_f8_quantize.argtypes = [_vp, i32, i32, i32, i32, i32, _vp]
        L.ns_f8_dequantize.argtypes = [_vp, i32, i32, _vp]
        L.ns_f8_matmul.argtypes = [_vp, i32, ctypes.c_float, i32, _vp, size, _vp]
        L.ns_f8_workspace_bytes.argtypes = [_vp, i32, i32, ctypes.POINTER(size)]
        for name in ("quantize", "dequantize", "matmul", "workspace_bytes"):
            getattr(L, "ns_f8_" + name).restype = ctypes.c_int
        _declared = L
    return _declared


_types = None


def _kinds():
    """({format dtype: ns_f8_format}, {scale dtype: ns_f8_scale})"""
    global _types
    if _types is None:
        import torch
        _types = ({torch.float8_e4m3fn: F8_E4M3, torch.float8_e5m2: F8_E5M2},
                  {torch.float32: F8_SCALE_FP32, torch.float8_e8m0fnu: F8_SCALE_POW2})
    return _types


def _format(dtype) -> int:
    form = _kinds()[0].get(dtype)
    if form is None:
        raise TypeError(f"unsupported 8-bit format {dtype}; use float8_e4m3fn or float8_e5m2")
    return form


def _up16(n: int) -> int:
    return (n + 15) // 16 * 16


def _pitch(cols: int) -> int:
    """Bytes from row to row of a new matrix: whole cache lines for long rows, as the
    products load them (2043 x 6101 by 2048: 86 us at a pitch of 6112, 78 at 6144; 8000 x
    1027: 30 and 27; quantised in 4 to 8% less). Shorter rows, whose values would grow by
    more than an eighth, gain nothing by it (quantised 20000 x 520: 13.2 and 13.6, its
    product 44 and 43)."""
    return (cols + 127) // 128 * 128 if cols >= 1024 else _up16(cols) or 16


def _blocks(n: int) -> int:
    return (n + F8_BLOCK - 1) // F8_BLOCK


def _pair(pair, name: str, index: int):
    """Checks an 8-bit matrix of a call on device `index`; its rows, columns and the
    members of ns_f8_matrix. (Lists of experts pass here twice a layer: one look at
    each attribute.)"""
    q, scale = pair
    forms, kinds = _kinds()
    form, kind = forms.get(q.dtype), kinds.get(scale.dtype)
    if form is None:
        _format(q.dtype)
    if kind is None:
        raise TypeError(f"the scales of {name} must be float32 or float8_e8m0fnu, not {scale.dtype}")
    if q.requires_grad:
        _refuse_grad(name)
    if scale.requires_grad:
        _refuse_grad(f"the scale of {name}")
    shape, shape_s = q.shape, scale.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = shape
    nb, nr = (cols + 127) // 128, (rows + 127) // 128
    if len(shape_s) != 2 or shape_s[0] != nb or (shape_s[1] != rows and shape_s[1] != nr):
        raise ValueError(f"{name} of {rows} x {cols} needs scales of {nb} x {rows}, or {nb} x {nr} for squares, not "
                         f"{tuple(shape_s)}")
    if q.get_device() != index or scale.get_device() != index:   # (-1 on the CPU)
        raise ValueError(f"{name}: {_SAME_DEVICE}")
    if rows == 0 or cols == 0:
        return rows, cols, (rows, cols, 0, 16, 0, 16, form | kind << 32, 0)
    per = shape_s[1]
    pitch, step = q.stride()
    ld, step_s = scale.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if rows == 1:
        pitch = (cols + 15) // 16 * 16
    elif pitch < cols:
        raise ValueError(f"the rows of {name} overlap")
    if step_s != 1 and per > 1:
        raise ValueError(f"the scales of a block of {name} must be contiguous")
    if nb == 1:
        ld = (per + 15) // 16 * 16
    elif ld < per:
        raise ValueError(f"the scales of {name} overlap")
    return rows, cols, (rows, cols, q.data_ptr(), pitch, scale.data_ptr(), ld, form | kind << 32,
                        0 if per == rows else 1)


def _new(n: int, rows: int, cols: int, per: int, dtype, kind, device):
    """n 8-bit matrices of one shape, which share a block of memory each for values and
    scales; (q, scale) pairs and the pitches."""
    import torch
    ld, lds, nb = _pitch(cols), _up16(per) or 16, _blocks(cols)
    q = torch.empty_strided((n * rows, cols), (ld, 1), dtype=dtype, device=device)
    s = torch.empty_strided((n * nb, per), (lds, 1), dtype=kind, device=device)
    if n == 1:
        return [F8Blocks(q, s)], ld, lds
    # (unsafe_split: tensors of their own to autograd, as in the int8 calls)
    qs = torch.unsafe_split(q, rows) if rows else [q] * n
    ss = torch.unsafe_split(s, nb) if nb else [s] * n
    return [F8Blocks(a, b) for a, b in zip(qs, ss)], ld, lds


def f8_quantize(tensors: Sequence, form: str = "rows", square: bool = False, pow2: bool = True, dtype=None,
                stream=None):
    """2-D bf16 or fp32 tensors (all of one dtype; rows contiguous, at any pitch) to
    8-bit floats with a scale for each block of 128 (ns_f8_quantize), a list of
    `F8Blocks` in the format `dtype` (default float8_e4m3fn, or float8_e5m2).

    form: "rows" for the matrices, "transposed" for their transposes, "both" for
    pairs (matrix, transpose) from one pass over the values. square: a scale for each
    128 x 128 values, the same both ways (weights); otherwise for 1 x 128 along the
    output's rows. pow2: scales that are powers of two, of one byte, with which
    f8_matmul takes about half the time; otherwise float32 scales. The results of a
    list of equal shapes share blocks of memory, which live as long as any of them."""
    import torch
    if form not in _FORMS:
        raise ValueError(f"form must be one of {', '.join(_FORMS)}, not {form!r}")
    dtype = torch.float8_e4m3fn if dtype is None else dtype
    code8 = _format(dtype)
    tensors = list(tensors)
    if not tensors:
        return []
    first = tensors[0]
    dt, n = first.dtype, len(tensors)
    code, device = _code(dt), _on_cuda(first.device)
    mats = [_matrix(t, "every matrix", dt, device) for t in tensors]
    kind = torch.float8_e8m0fnu if pow2 else torch.float32
    context, handle = _enter(device, stream, lambda: tensors)
    with context:
        def new(turned):
            sizes = [(m[1], m[0]) if turned else m[:2] for m in mats]
            rows, cols = sizes[0]
            if all(s == (rows, cols) for s in sizes):
                made, ld, lds = _new(n, rows, cols, _blocks(rows) if square else rows, dtype, kind, device)
                return made, [(p.q.data_ptr(), ld, p.scale.data_ptr(), lds) for p in made]
            made, where = [], []
            for rows, cols in sizes:
                (p,), ld, lds = _new(1, rows, cols, _blocks(rows) if square else rows, dtype, kind, device)
                made.append(p)
                where.append((p.q.data_ptr(), ld, p.scale.data_ptr(), lds))
            return made, where
        none = (0, 0, 0, 0)
        direct, at = new(False) if form != "transposed" else (None, [none] * n)
        turned, at_t = new(True) if form != "rows" else (None, [none] * n)
        flat = []
        for (rows, cols, pitch, address), a, b in zip(mats, at, at_t):
            flat += (rows, cols, address, pitch)
            flat += a
            flat += b
        _check(lib().ns_f8_quantize(_int64s(flat), n, code8, F8_SCALE_POW2 if pow2 else F8_SCALE_FP32, int(square),
                                    code, handle))
    if form == "both":
        return list(zip(direct, turned))
    return direct if turned is None else turned


def f8_dequantize(matrices: Sequence, dtype=None, stream=None):
    """The values of 8-bit matrices as a list of tensors of `dtype` (default bf16)
    (ns_f8_dequantize). Here and in f8_matmul, the new tensors of a list of one width
    may share one block of memory."""
    import torch
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _code(dtype)
    matrices = list(matrices)
    if not matrices:
        return []
    device = _on_cuda(matrices[0][0].device)
    pairs = [_pair(m, "every matrix", device.index) for m in matrices]
    context, handle = _enter(device, stream, lambda: [t for m in matrices for t in m])
    with context:
        out = _empty([p[:2] for p in pairs], dtype, device)
        flat = []
        for (rows, cols, members), v in zip(pairs, out):
            flat += members
            flat += (v.data_ptr(), cols or 1)
        _check(lib().ns_f8_dequantize(_int64s(flat), len(pairs), code, handle))
    return out


def f8_matmul(xs: Sequence, ws: Sequence, dtype=None, out: Optional[Sequence] = None, beta: float = 0.0, stream=None):
    """C <- beta C + X W^T of 8-bit matrices (ns_f8_matmul), both with the sum's axis
    along their rows: a layer's output from its input and weights, its input's
    gradient from dY and the transposed weights, its weights' gradient from the
    transposes of dY and of the input. `xs` holds `F8Blocks` of m x k in either
    format, `ws` of n x k in float8_e4m3fn. Returns a list of m x n tensors of `dtype`
    (default that of `out`, else bf16), new ones or those of `out`, which are not read
    when beta == 0. fp32 results have the accuracy of fp32 sums, at half the rate of
    bf16 ones, which lose up to 7 2^-13 of the largest of each eight products."""
    import torch
    xs, ws = list(xs), list(ws)
    if len(xs) != len(ws):
        raise ValueError(_LENGTHS)
    given = ()
    if out is not None:
        given = out = list(out)
        if len(out) != len(xs):
            raise ValueError("one output per product is needed")
    elif beta != 0.0:
        raise ValueError("beta needs outputs to add to")
    if dtype is None:
        dtype = out[0].dtype if out else torch.bfloat16
    code = _code(dtype)
    if not xs:
        return []
    n = len(xs)
    device = _on_cuda(xs[0][0].device)
    index, layers, shapes = device.index, [], []
    for x, w in zip(xs, ws):
        m, k, a = _pair(x, "x", index)
        c, kw, b = _pair(w, "w", index)
        if k != kw:
            raise ValueError(f"x has {k} columns, w {kw}")
        layers.append(a + b)
        shapes.append((m, c))
    if out is not None:
        spots = [_matrix(t, "an output", dtype, device) for t in out]
        for m, shape in zip(spots, shapes):
            if m[:2] != shape:
                raise ValueError(f"an output is {m[:2]}, its product needs {shape}")
    context, handle = _enter(device, stream, lambda: [*(t for pair in (*xs, *ws) for t in pair), *given])
    with context:
        if out is None:
            out = _empty(shapes, dtype, device)
            spots = [(*s, s[1] or 1, t.data_ptr()) for t, s in zip(out, shapes)]
        flat = []
        for members, m in zip(layers, spots):
            flat += members
            flat += (m[3], m[2])
        arr, L = _int64s(flat), lib()
        # most calls need no workspace; one that does is refused without it, with
        # nothing enqueued
        rc = L.ns_f8_matmul(arr, n, beta, code, None, 0, handle)
        if rc:
            need = ctypes.c_size_t(0)
            if rc == 1 and L.ns_f8_workspace_bytes(arr, n, code, ctypes.byref(need)) == 0 and need.value:
                # a block of the caching allocator: the call's own until it has run on
                # this stream, also inside a captured graph
                block = torch.empty(need.value, dtype=torch.uint8, device=device)
                rc = L.ns_f8_matmul(arr, n, beta, code, block.data_ptr(), need.value, handle)
            _check(rc)
    if given:
        torch.autograd.graph.increment_version(given)
    return out
