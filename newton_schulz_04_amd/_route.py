"""ctypes binding of the experts' router of libns.so (include/ns.h, ns_route_*):
argument checks and marshalling only.

`route_experts` is the forward call, `route_experts_grad` its backward: the pieces that
a router's autograd.Function is written from; they have no gradients of their own. In
grad mode a tensor that requires grad is refused, as its gradient would be lost without
a word: under torch.no_grad() and in an autograd.Function's methods all are taken.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional

from . import _binding
from ._binding import _check
from ._q8 import _code, _enter, _matrix, _on_cuda, _refuse_grad, _SAME_DEVICE

ROUTE_MAX_EXPERTS, ROUTE_MAX_K = 1024, 16

_i64, _vp = ctypes.c_int64, ctypes.c_void_p


# ns_route and ns_route_grad
_ROUTE = struct.Struct("qqQqQiiQQQQQQ")
_ROUTE_GRAD = struct.Struct("qqQqiiQQQQQQq")
# tokens that one workgroup routes by itself, with no workspace, whatever the experts
_ALONE = 32


class Route(NamedTuple):
    """What `route_experts` returns for T tokens, E experts and top_k = k."""
    experts: "torch.Tensor"   # int32, T x k: the chosen, -1 for none  # noqa: F821
    weights: "torch.Tensor"   # float32, T x k  # noqa: F821
    counts: "torch.Tensor"    # int32, E: tokens of each expert  # noqa: F821
    probs: "torch.Tensor"     # float32, E: the sum of its p  # noqa: F821
    tokens: "torch.Tensor"    # int32, one number: tokens that count  # noqa: F821
    loss: "torch.Tensor"      # float32, one number: the balance loss  # noqa: F821


_declared: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    global _declared
    if _declared is None:
        L = _binding.lib()
        i32, size = ctypes.c_int32, ctypes.c_size_t
        L.ns_route_experts.argtypes = [_vp, i32, _vp, size, _vp]
        L.ns_route_workspace_bytes.argtypes = [_i64, _i64, ctypes.POINTER(size)]
        L.ns_route_experts_grad.argtypes = [_vp, i32, _vp]
        for name in ("experts", "workspace_bytes", "experts_grad"):
            getattr(L, "ns_route_" + name).restype = ctypes.c_int
        _declared = L
    return _declared


def _logits(logits, top_k):
    code, device = _code(logits.dtype), _on_cuda(logits.device)
    tokens, experts, pitch, at = _matrix(logits, "logits", logits.dtype, device)
    if not 1 <= experts <= ROUTE_MAX_EXPERTS:
        raise ValueError(f"1 to {ROUTE_MAX_EXPERTS} experts are taken, not {experts}")
    if not 1 <= top_k <= min(ROUTE_MAX_K, experts):
        raise ValueError(f"top_k must be 1 to {min(ROUTE_MAX_K, experts)}, not {top_k}")
    return code, device, tokens, experts, max(pitch, experts), at


def _given(t, name: str, shape, dtype, device):
    """Checks a contiguous tensor of a call; its address (0 when it is empty)."""
    if t.requires_grad:
        _refuse_grad(name)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {shape}, not {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != device.index:
        raise ValueError(f"{name}: {_SAME_DEVICE}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() if t.numel() else 0


def route_experts(logits, top_k: int, normalize: bool = True, mask=None, stream=None) -> Route:
    """The top_k experts of each token, their weights, the experts' counts and the
    balance loss (ns_route_experts), as a `Route` of new tensors.

    logits: tokens x experts, bf16 or fp32, rows contiguous at any pitch; an expert of
    logit -Inf is never chosen. normalize: weights that add up to 1 for a token, rather
    than the softmax's. mask: bool, tokens; those of False (padding) have experts -1,
    weights 0 and count for nothing. All stays on the device; `counts` are what the lists
    of the layers' calls are cut by, whose sizes are the host's: reading them waits for
    the device, which a captured graph cannot."""
    import torch
    code, device, tokens, experts, pitch, at = _logits(logits, top_k)
    mask_at = 0 if mask is None else _given(mask, "mask", (tokens,), torch.bool, device)
    context, handle = _enter(device, stream, lambda: [logits] if mask is None else [logits, mask])
    with context:
        i32, f32 = torch.int32, torch.float32
        r = Route(torch.empty((tokens, top_k), dtype=i32, device=device),
                  torch.empty((tokens, top_k), dtype=f32, device=device),
                  torch.empty(experts, dtype=i32, device=device), torch.empty(experts, dtype=f32, device=device),
                  torch.empty((), dtype=i32, device=device), torch.empty((), dtype=f32, device=device))
        L, block, size = lib(), None, 0
        if tokens > _ALONE:
            need = ctypes.c_size_t(0)
            _check(L.ns_route_workspace_bytes(tokens, experts, ctypes.byref(need)))
            size = need.value
            # a block of the caching allocator: the call's own until it has run on this
            # stream, also inside a captured graph
            block = torch.empty(size, dtype=torch.uint8, device=device) if size else None
        args = _ROUTE.pack(tokens, experts, at, pitch, mask_at, top_k, 1 if normalize else 0,
                           r.experts.data_ptr() if tokens else 0, r.weights.data_ptr() if tokens else 0,
                           r.counts.data_ptr(), r.probs.data_ptr(), r.tokens.data_ptr(), r.loss.data_ptr())
        _check(L.ns_route_experts(args, code, block.data_ptr() if size else None, size, handle))
    return r


def route_experts_grad(logits, experts, counts, tokens, dweights=None, dloss=None, normalize: bool = True, out=None,
                       stream=None):
    """The logits' gradient from those of a route's weights and of its balance loss,
    either of which may be None (ns_route_experts_grad). experts, counts, tokens: the
    `Route`'s; counts may be summed over data-parallel ranks. dweights: float32, as the
    route's weights; dloss: float32, one number on the device. Returns a tensor like
    logits, a new one or `out`, which may be the logits."""
    import torch
    top_k = experts.shape[1] if experts.dim() == 2 else 0
    code, device, rows, n, pitch, at = _logits(logits, top_k)
    i32, f32 = torch.int32, torch.float32
    chosen = _given(experts, "experts", (rows, top_k), i32, device)
    count_at = _given(counts, "counts", (n,), i32, device)
    tokens_at = _given(tokens, "tokens", (), i32, device)
    dw = 0 if dweights is None else _given(dweights, "dweights", (rows, top_k), f32, device)
    dl = 0 if dloss is None else _given(dloss, "dloss", (), f32, device)
    given = ()
    if out is not None:
        given = (out,)
        spot = _matrix(out, "out", logits.dtype, device)
        if spot[:2] != (rows, n):
            raise ValueError(f"out is {spot[:2]}, the logits {(rows, n)}")
    held = [t for t in (logits, experts, counts, tokens, dweights, dloss, out) if t is not None]
    context, handle = _enter(device, stream, lambda: held)
    with context:
        if out is None:
            out = torch.empty((rows, n), dtype=logits.dtype, device=device)
            spot = (rows, n, n, out.data_ptr())
        args = _ROUTE_GRAD.pack(rows, n, at, pitch, top_k, 1 if normalize else 0, chosen, count_at, tokens_at, dw, dl,
                                spot[3], max(spot[2], n))
        _check(lib().ns_route_experts_grad(args, code, handle))
    if given:
        torch.autograd.graph.increment_version(given)
    return out
