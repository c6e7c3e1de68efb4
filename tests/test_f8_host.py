"""The 8-bit floating-point calls on the CPU: what they refuse, what they accept
without touching a device, and the workspace they ask for. No call here reaches the
GPU: every one is either refused or has nothing to do."""
import ctypes

import pytest
import torch

import newton_schulz_04_amd as ns
from newton_schulz_04_amd import _f8

OK, EINVAL, EDTYPE = 0, 1, 2


class Rows(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "cols", "values", "ld_values", "q", "ld_q", "scale", "ld_scale",
                                              "qt", "ld_qt", "scale_t", "ld_scale_t")]


class Matrix(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "cols", "q", "ld_q", "scale", "ld_scale")] + \
               [(n, ctypes.c_int32) for n in ("format", "scale_type", "square", "reserved")]


class Values(ctypes.Structure):
    _fields_ = [("matrix", Matrix), ("values", ctypes.c_int64), ("ld_values", ctypes.c_int64)]


class Product(ctypes.Structure):
    _fields_ = [("a", Matrix), ("b", Matrix), ("out", ctypes.c_int64), ("ld_out", ctypes.c_int64)]


def test_the_binding_lays_out_the_structs():
    assert ctypes.sizeof(Rows) == 96 and ctypes.sizeof(Matrix) == 64
    assert ctypes.sizeof(Values) == 80 and ctypes.sizeof(Product) == 144


def rows(**kw):
    v = dict(rows=130, cols=200, values=0x100000, ld_values=200, q=0x200000, ld_q=208, scale=0x300000, ld_scale=132,
             qt=0x400000, ld_qt=144, scale_t=0x500000, ld_scale_t=200)
    v.update(kw)
    return Rows(**v)


def matrix(r, k, at, **kw):
    v = dict(rows=r, cols=k, q=at, ld_q=-(-k // 16) * 16, scale=at + 0x8000000, ld_scale=-(-r // 4) * 4, scale_type=1)
    v.update(kw)
    return Matrix(**v)


def product(m=40, n=50, k=200, a=None, b=None, **kw):
    v = dict(out=0x70000000, ld_out=n)
    v.update(kw)
    return Product(matrix(m, k, 0x10000000, **(a or {})), matrix(n, k, 0x30000000, **(b or {})), v["out"], v["ld_out"])


def quantize(items, count=None, fmt=0, kind=1, square=0, dtype=0):
    arr = (Rows * max(1, len(items)))(*items)
    return _f8.lib().ns_f8_quantize(arr if items else None, len(items) if count is None else count, fmt, kind, square,
                                    dtype, None)


def need(items, dtype=0, count=None):
    out = ctypes.c_size_t(77)
    arr = (Product * max(1, len(items)))(*items)
    rc = _f8.lib().ns_f8_workspace_bytes(arr if items else None, len(items) if count is None else count, dtype,
                                         ctypes.byref(out))
    return rc, out.value


def matmul(items, dtype=0, count=None, ws=None, nbytes=0, beta=0.0):
    arr = (Product * max(1, len(items)))(*items)
    return _f8.lib().ns_f8_matmul(arr if items else None, len(items) if count is None else count, beta, dtype, ws,
                                  nbytes, None)


NOTHING = dict(values=0, q=0, scale=0, qt=0, scale_t=0)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(cols=-1), EINVAL), (dict(rows=(1 << 24) + 1), EINVAL),
    (dict(cols=(1 << 24) + 1, ld_values=1 << 25, ld_q=1 << 25), EINVAL),
    (dict(values=0), EINVAL), (dict(values=0x100001), EINVAL), (dict(ld_values=199), EINVAL),
    (dict(ld_values=1 << 31), EINVAL), (dict(q=0), EINVAL), (dict(scale=0), EINVAL), (dict(qt=0), EINVAL),
    (dict(scale_t=0), EINVAL), (dict(q=0, scale=0, qt=0, scale_t=0), EINVAL),
    (dict(q=0x200008), EINVAL), (dict(ld_q=200), EINVAL), (dict(ld_q=192), EINVAL), (dict(ld_q=1 << 31), EINVAL),
    (dict(qt=0x400001), EINVAL), (dict(ld_qt=128), EINVAL), (dict(ld_qt=136), EINVAL),
    (dict(scale=0x300002), EINVAL), (dict(ld_scale=130), EINVAL), (dict(ld_scale=128), EINVAL),
    (dict(scale_t=0x500001), EINVAL), (dict(ld_scale_t=198), EINVAL), (dict(ld_scale_t=1 << 31), EINVAL),
    (dict(rows=0, **NOTHING), OK), (dict(cols=0, **NOTHING), OK),
])
def test_quantize_refusals(kw, status):
    assert quantize([rows(**kw)]) == status, ns.last_error()
    assert bool(ns.last_error()) == (status != OK)


def test_quantize_arguments():
    assert quantize([], count=-1) == EINVAL and quantize([], count=1) == EINVAL
    assert quantize([], count=0) == OK
    assert quantize([rows()], fmt=2) == EINVAL and quantize([rows()], kind=2) == EINVAL
    assert quantize([rows()], square=2) == EINVAL and quantize([rows()], dtype=5) == EDTYPE
    assert quantize([rows(values=0x100002)], dtype=1) == EINVAL
    # outputs that overlap: two matrices' q, a matrix's own two forms, scales within q
    apart = dict(scale=0x600000, qt=0x700000, scale_t=0x800000)
    assert quantize([rows(), rows(**apart)]) == EINVAL and "overlap" in ns.last_error()
    assert quantize([rows(qt=0x200010)]) == EINVAL
    assert quantize([rows(scale=0x200100)]) == EINVAL
    # fp32 scales are four bytes wide
    assert quantize([rows(scale_t=0x300000 + 500)], kind=0) == EINVAL and "overlap" in ns.last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(cols=(1 << 24) + 1), EINVAL), (dict(q=0), EINVAL), (dict(q=0x1008), EINVAL),
    (dict(ld_q=200), EINVAL), (dict(scale=0), EINVAL), (dict(scale=0x2001), EINVAL), (dict(ld_scale=8), EINVAL),
    (dict(format=2), EINVAL), (dict(scale_type=2), EINVAL), (dict(square=-1), EINVAL),
    (dict(rows=0, q=0, scale=0), OK), (dict(cols=0, q=0, scale=0), OK),
])
def test_dequantize_refusals(kw, status):
    v = (Values * 1)(Values(matrix(40, 200, 0x10000000, **kw), 0x100000, 200))
    assert _f8.lib().ns_f8_dequantize(v, 1, 0, None) == status, ns.last_error()


def test_dequantize_arguments():
    L = _f8.lib()
    v = (Values * 2)(Values(matrix(40, 200, 0x10000000), 0x100000, 200), Values(matrix(40, 200, 0x10000000), 0x100100, 200))
    assert L.ns_f8_dequantize(v, 2, 0, None) == EINVAL and "overlap" in ns.last_error()
    assert L.ns_f8_dequantize(v, -1, 0, None) == EINVAL and L.ns_f8_dequantize(None, 1, 0, None) == EINVAL
    assert L.ns_f8_dequantize(v, 1, 7, None) == EDTYPE and L.ns_f8_dequantize(None, 0, 0, None) == OK
    v[0].ld_values = 199
    assert L.ns_f8_dequantize(v, 1, 0, None) == EINVAL
    v[0].ld_values, v[0].values = 200, 0
    assert L.ns_f8_dequantize(v, 1, 0, None) == EINVAL


@pytest.mark.parametrize("side", ["a", "b"])
@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=(1 << 24) + 1), dict(cols=-1), dict(cols=201), dict(q=0), dict(q=0x10000008), dict(ld_q=200),
    dict(ld_q=192), dict(ld_q=(1 << 21) + 16), dict(scale=0), dict(scale=0x40000002), dict(ld_scale=50), dict(ld_scale=12),
    dict(ld_scale=1 << 31), dict(format=3), dict(scale_type=2), dict(square=2), dict(scale_type=0, scale=0x40000002),
])
def test_matmul_refuses_operands(side, kw):
    p = product(m=50, **{side: kw})
    assert need([p])[0] == EINVAL, kw
    assert matmul([p]) == EINVAL and ns.last_error()


def test_matmul_refusals():
    assert matmul([product(b=dict(format=1))]) == EINVAL and "e4m3" in ns.last_error()
    assert need([product(a=dict(format=1))])[0] == OK
    # fp32 scales need no more than their own alignment
    assert need([product(a=dict(scale_type=0, ld_scale=41, scale=0x40000004))])[0] == OK
    for kw in (dict(out=0), dict(out=0x70000001), dict(ld_out=49), dict(ld_out=(1 << 21) + 1)):
        assert matmul([product(**kw)]) == EINVAL, kw
    assert matmul([product(out=0x70000002)], dtype=1) == EINVAL
    assert matmul([], count=-1) == EINVAL and matmul([], count=1) == EINVAL and matmul([], count=0) == OK
    assert need([product()], dtype=4)[0] == EDTYPE and matmul([product()], dtype=4) == EDTYPE
    assert matmul([product(), product()]) == EINVAL and "overlap" in ns.last_error()
    assert _f8.lib().ns_f8_workspace_bytes((Product * 1)(product()), 1, 0, None) == EINVAL
    long = dict(cols=1 << 22, ld_q=1 << 22)
    assert matmul([product(k=1 << 22, a=long, b=long)]) == EINVAL
    # (one row of A: its pitch is not the limit, the sum's length is)
    assert matmul([product(m=1 << 24, n=1 << 21, k=16, ld_out=1 << 21)]) == EINVAL and "tiles" in ns.last_error()


def test_matmul_without_outputs_or_sums():
    empty = dict(q=0, scale=0)
    assert matmul([product(m=0, a=empty, out=0), product(n=0, b=empty, out=0, ld_out=1)]) == OK, ns.last_error()
    # a sum over nothing reads no operands, but has outputs
    assert need([product(k=0, a=empty, b=empty)]) == (OK, 0)
    assert need([product(k=0, a=empty, b=empty, out=0)])[0] == EINVAL


def test_workspace():
    # few outputs and a long sum: pieces that meet in a workspace
    long = product(m=128, n=256, k=1 << 16)
    rc, n = need([long])
    assert rc == OK and n >= 2 * 128 * 256 * 4
    other = product(m=128, n=256, k=1 << 16, out=0x78000000)
    assert need([long, other]) == (OK, 2 * n)
    assert matmul([long]) == EINVAL and "workspace" in ns.last_error()
    assert matmul([long], ws=0x100000, nbytes=n - 1) == EINVAL
    assert matmul([long], ws=0x100008, nbytes=n) == EINVAL
    assert need([product(m=4096, n=8192, k=6144, ld_out=8192)]) == (OK, 0)
    assert need([product(m=32, n=256, k=1 << 16)]) == (OK, 0)


def test_binding_refusals():
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    q, s = torch.zeros((4, 16)).to(e4), torch.ones((1, 4))
    for call in (lambda: ns.f8_quantize([torch.zeros(4, 8)]), lambda: ns.f8_dequantize([(q, s)]),
                 lambda: ns.f8_matmul([(q, s)], [(q, s)])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        ns.f8_quantize([torch.zeros((4, 8))], dtype=torch.int8)
    with pytest.raises(ValueError, match="form"):
        ns.f8_quantize([torch.zeros((4, 8))], form="columns")
    with pytest.raises(TypeError):
        ns.f8_quantize([torch.zeros((4, 8), dtype=torch.float16)])
    with pytest.raises(TypeError):
        ns.f8_matmul([(q, s)], [(q, s)], dtype=torch.float16)
    with pytest.raises(ValueError):
        ns.f8_matmul([(q, s)], [])
    with pytest.raises(ValueError, match="beta"):
        ns.f8_matmul([(q, s)], [(q, s)], beta=1.0)
    with pytest.raises(ValueError):
        ns.f8_matmul([(q, s)], [(q, s)], out=[])
    assert ns.f8_quantize([]) == [] and ns.f8_dequantize([]) == [] and ns.f8_matmul([], []) == []
    # pairs: on the CPU's device index, so that the device is not what is refused
    def pair(q, s):
        return _f8._pair((q, s), "x", -1)

    assert pair(q, s)[2][6:] == (0, 0)
    assert pair(q, s.to(e8))[2][6:] == (1 << 32, 0)
    assert pair(torch.zeros((200, 16)).to(e4), torch.ones((1, 2)))[2][7] == 1
    for bad in ((q, torch.ones((2, 4))), (q, torch.ones((1, 3))), (q, torch.ones(4)), (q[0], s),
                (torch.zeros((2, 300)).to(e4), torch.ones((4, 3)).T), (q.T, s)):
        with pytest.raises(ValueError):
            pair(*bad)
    for bad in ((q.float(), s), (q, s.double()), (q, s.to(torch.bfloat16))):
        with pytest.raises(TypeError):
            pair(*bad)
    with pytest.raises(ValueError, match="grad"):
        pair(q, s.requires_grad_())


@pytest.mark.parametrize("cols,pitch", [(1, 16), (100, 112), (1000, 1008), (1023, 1024), (1024, 1024), (1027, 1152),
                                        (6101, 6144)])
def test_new_matrices_hold_long_rows_in_whole_lines(cols, pitch):
    for n in (1, 3):
        made, ld, lds = _f8._new(n, 5, cols, 5, torch.float8_e4m3fn, torch.float8_e8m0fnu, "cpu")
        assert (ld, lds) == (pitch, 16)
        for q, s in made:
            assert q.shape == (5, cols) and q.stride() == (pitch, 1) and q.storage_offset() % 16 == 0
            assert s.shape == (-(-cols // 128), 5) and s.stride() == (16, 1)
