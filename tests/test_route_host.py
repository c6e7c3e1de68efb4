"""The router's calls on the CPU: what they refuse. No call here reaches the GPU."""
import ctypes

import pytest
import torch

import newton_schulz_04_amd as ns
from newton_schulz_04_amd import _route

OK, EINVAL, EDTYPE = 0, 1, 2


class Route(ctypes.Structure):
    """ns_route"""
    _fields_ = [("tokens", ctypes.c_int64), ("experts", ctypes.c_int64), ("logits", ctypes.c_void_p),
                ("ld", ctypes.c_int64), ("mask", ctypes.c_void_p), ("top_k", ctypes.c_int32),
                ("normalize", ctypes.c_int32), ("chosen", ctypes.c_void_p), ("weights", ctypes.c_void_p),
                ("counts", ctypes.c_void_p), ("probs", ctypes.c_void_p), ("routed", ctypes.c_void_p),
                ("loss", ctypes.c_void_p)]


class RouteGrad(ctypes.Structure):
    """ns_route_grad"""
    _fields_ = [("tokens", ctypes.c_int64), ("experts", ctypes.c_int64), ("logits", ctypes.c_void_p),
                ("ld", ctypes.c_int64), ("top_k", ctypes.c_int32), ("normalize", ctypes.c_int32),
                ("chosen", ctypes.c_void_p), ("counts", ctypes.c_void_p), ("routed", ctypes.c_void_p),
                ("dweights", ctypes.c_void_p), ("dloss", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("ld_out", ctypes.c_int64)]


def test_the_binding_lays_out_the_structs():
    assert ctypes.sizeof(Route) == _route._ROUTE.size and ctypes.sizeof(RouteGrad) == _route._ROUTE_GRAD.size
    assert bytes(Route(*range(1, 14))) == _route._ROUTE.pack(*range(1, 14))
    assert bytes(RouteGrad(*range(1, 14))) == _route._ROUTE_GRAD.pack(*range(1, 14))


def route(**kw):
    v = dict(tokens=100, experts=16, logits=0x1000, ld=16, mask=0x2000, top_k=2, normalize=1, chosen=0x3000,
             weights=0x4000, counts=0x5000, probs=0x6000, routed=0x7000, loss=0x8000)
    v.update(kw)
    return Route(**v)


def grad(**kw):
    v = dict(tokens=100, experts=16, logits=0x1000, ld=16, top_k=2, normalize=1, chosen=0x3000, counts=0x5000,
             routed=0x7000, dweights=0x8000, dloss=0x9000, out=0xA000, ld_out=16)
    v.update(kw)
    return RouteGrad(**v)


COMMON = [dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(experts=0), dict(experts=1025, ld=2000), dict(logits=None),
          dict(logits=0x1001), dict(ld=15), dict(ld=1 << 31), dict(top_k=0), dict(top_k=17, experts=64, ld=64),
          dict(top_k=3, experts=2), dict(normalize=2), dict(chosen=None), dict(chosen=0x3002), dict(counts=None),
          dict(counts=0x5001), dict(routed=None), dict(routed=0x7002)]


@pytest.mark.parametrize("kw", COMMON + [dict(weights=None), dict(weights=0x4001), dict(probs=None), dict(probs=0x6002),
                                         dict(loss=None), dict(loss=0x8001)])
def test_route_refusals(kw):
    ws = 0x100000, 1 << 24
    assert _route.lib().ns_route_experts(ctypes.byref(route(**kw)), 0, *ws, None) == EINVAL, kw
    assert ns.last_error()


@pytest.mark.parametrize("kw", COMMON + [dict(dweights=0x8001), dict(dloss=0x9002), dict(out=None), dict(out=0xA001),
                                         dict(ld_out=15), dict(ld_out=1 << 31)])
def test_gradient_refusals(kw):
    assert _route.lib().ns_route_experts_grad(ctypes.byref(grad(**kw)), 0, None) == EINVAL, kw
    assert ns.last_error()


def test_arguments():
    L = _route.lib()
    assert L.ns_route_experts(None, 0, None, 0, None) == EINVAL and L.ns_route_experts_grad(None, 0, None) == EINVAL
    assert L.ns_route_experts(ctypes.byref(route()), 3, None, 0, None) == EDTYPE
    assert L.ns_route_experts_grad(ctypes.byref(grad()), 3, None) == EDTYPE
    assert L.ns_route_experts(ctypes.byref(route(logits=0x1002)), 1, 0x100000, 1 << 24, None) == EINVAL
    # nothing to do, nothing read
    assert L.ns_route_experts_grad(ctypes.byref(grad(tokens=0, logits=None, chosen=None, out=None)), 0, None) == OK


def test_workspace():
    L, need = _route.lib(), ctypes.c_size_t(7)

    def ask(tokens, experts):
        return L.ns_route_workspace_bytes(tokens, experts, ctypes.byref(need)), need.value

    assert ask(0, 16) == (OK, 0) and ask(16, 256) == (OK, 0)
    # (as the binding takes for granted)
    assert all(ask(_route._ALONE, e) == (OK, 0) for e in (1, 16, 256, 257, 1024))
    rc, n = ask(100000, 256)
    assert rc == OK and n >= 2 * 4 * 256
    for bad in ((-1, 16), (5, 0), (5, 1025), ((1 << 24) + 1, 4)):
        assert ask(*bad)[0] == EINVAL
    assert L.ns_route_workspace_bytes(5, 5, None) == EINVAL
    r = route(tokens=100000, experts=256, ld=256)
    for ws in ((None, 0), (0x100000, n - 1), (0x100008, n)):
        assert L.ns_route_experts(ctypes.byref(r), 0, *ws, None) == EINVAL
        assert "workspace" in ns.last_error()


def test_binding_refusals():
    x = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ns.route_experts(x, 2)
    with pytest.raises(TypeError):
        ns.route_experts(x.half(), 2)
    with pytest.raises(ValueError, match="CUDA"):
        ns.route_experts_grad(x, torch.zeros((4, 2), dtype=torch.int32), torch.zeros(8, dtype=torch.int32),
                              torch.tensor(4, dtype=torch.int32))
    dev = type("D", (), {"index": -1, "type": "cpu"})()
    ok = torch.zeros((4, 2), dtype=torch.int32)
    assert _route._given(ok, "t", (4, 2), torch.int32, dev) == ok.data_ptr()
    for t, shape in ((ok, (4, 3)), (ok.T, (2, 4)), (ok[:, 0], (4,))):
        with pytest.raises(ValueError):
            _route._given(t, "t", shape, torch.int32, dev)
    with pytest.raises(TypeError):
        _route._given(ok.long(), "t", (4, 2), torch.int32, dev)
    with pytest.raises(ValueError, match="grad"):
        _route._given(torch.zeros(3, requires_grad=True), "t", (3,), torch.float32, dev)
