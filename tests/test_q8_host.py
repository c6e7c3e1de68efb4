"""The 8-bit linear-layer calls on the CPU: what they refuse, what they accept
without touching a device (empty layers), and the workspace they ask for. No
call here reaches the GPU: every one is either refused or has nothing to do."""
import ctypes

import pytest
import torch

import newton_schulz_04_amd as ns
from newton_schulz_04_amd import _q8

OK, EINVAL, EDTYPE = 0, 1, 2


def rows(**kw):
    v = dict(rows=4, cols=8, values=0x1000, ld_values=8, q=0x2000, ld_q=8, scale=0x3000)
    v.update(kw)
    return _q8.RowsStruct(**v)


def layer(**kw):
    v = dict(tokens=4, out_features=6, in_features=8, xq=0x10000, ld_xq=8, x_scale=0x20000, wq=0x30000, ld_wq=8,
             w_scale=0x40000, dy=0x50000, ld_dy=6, out=0x60000, ld_out=8)
    v.update(kw)
    return _q8.LayerStruct(**v)


def arr(items):
    return ((type(items[0])) * len(items))(*items) if items else None


def run_rows(items, mode=0, dtype=0, count=None, back=False):
    L, n = _q8.lib(), len(items) if count is None else count
    if back:
        return L.ns_q8_dequantize(arr(items), n, dtype, None)
    return L.ns_q8_quantize(arr(items), n, mode, dtype, None)


def run_op(op, items, dtype=0, count=None, ws=None, nbytes=0, beta=0.0):
    L, n = _q8.lib(), len(items) if count is None else count
    if op == 0:
        return L.ns_q8_matmul(arr(items), n, dtype, ws, nbytes, None)
    if op == 1:
        return L.ns_q8_grad_input(arr(items), n, ws, nbytes, None)
    return L.ns_q8_grad_weight(arr(items), n, beta, dtype, ws, nbytes, None)


def need(op, items, dtype=0):
    out = ctypes.c_size_t(77)
    rc = _q8.lib().ns_q8_workspace_bytes(op, arr(items), len(items), dtype, ctypes.byref(out))
    return rc, out.value


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(cols=-1), EINVAL), (dict(rows=(1 << 24) + 1), EINVAL),
    (dict(cols=(1 << 24) + 1, ld_values=1 << 25, ld_q=1 << 25), EINVAL),
    (dict(values=None), EINVAL), (dict(q=None), EINVAL), (dict(scale=None), EINVAL),
    (dict(values=0x1001), EINVAL), (dict(scale=0x3002), EINVAL),
    (dict(ld_values=7), EINVAL), (dict(ld_q=7), EINVAL), (dict(ld_q=1 << 31), EINVAL),
    (dict(rows=0, values=None, q=None, scale=None), OK), (dict(cols=0, values=None, q=None, scale=None), OK),
])
def test_rows_refusals(kw, status, back):
    assert run_rows([rows(**kw)], back=back) == status, ns.last_error()
    assert bool(ns.last_error()) == (status != OK)


def test_rows_arguments():
    assert run_rows([], count=-1) == EINVAL
    assert run_rows([], count=0) == OK
    assert run_rows([], count=1) == EINVAL          # NULL list
    assert run_rows([rows()], mode=2) == EINVAL
    assert run_rows([rows()], dtype=5) == EDTYPE
    assert run_rows([rows(values=0x1002)], dtype=1) == EINVAL   # aligned for bf16, not for fp32
    # outputs that overlap: the same q twice, scales in q, the same values twice
    assert run_rows([rows(), rows(scale=0x4000)]) == EINVAL and "overlap" in ns.last_error()
    assert run_rows([rows(scale=0x2010)]) == EINVAL
    assert run_rows([rows(), rows(q=0x9000, scale=0xA000)], back=True) == EINVAL


@pytest.mark.parametrize("op", [0, 1, 2])
@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), EINVAL), (dict(out_features=-1), EINVAL), (dict(in_features=-1), EINVAL),
    (dict(tokens=(1 << 24) + 1), EINVAL), (dict(out_features=(1 << 24) + 1, ld_dy=1 << 25), EINVAL),
    (dict(out=None), EINVAL), (dict(out=0x60001), EINVAL),
    (dict(xq=None, wq=None), EINVAL), (dict(x_scale=None, w_scale=None), EINVAL),
    (dict(x_scale=0x20001, w_scale=0x40002), EINVAL),
    (dict(ld_xq=7, ld_wq=7), EINVAL), (dict(ld_xq=(1 << 21) + 1, ld_wq=(1 << 21) + 1), EINVAL),
    (dict(ld_out=5), EINVAL), (dict(ld_out=(1 << 21) + 1), EINVAL),
])
def test_product_refusals(op, kw, status):
    assert need(op, [layer(**kw)])[0] == status, ns.last_error()
    assert run_op(op, [layer(**kw)]) == status
    assert ns.last_error()


@pytest.mark.parametrize("op", [1, 2])
def test_gradient_refusals(op):
    for kw in (dict(dy=None), dict(dy=0x50001), dict(ld_dy=5), dict(ld_dy=(1 << 21) + 1)):
        assert run_op(op, [layer(**kw)]) == EINVAL, kw
    # what a call does not read it does not check
    unread = dict(wq=None, w_scale=None, ld_wq=0) if op == 2 else dict(xq=None, x_scale=None, ld_xq=0)
    assert need(op, [layer(**unread)])[0] == OK


def test_matmul_refusals():
    big = dict(in_features=131072, ld_xq=131072, ld_wq=131072)
    assert run_op(0, [layer(**big)]) == EINVAL and "NS_Q8_MAX_K" in ns.last_error()
    assert need(0, [layer(dy=None, ld_dy=0)])[0] == OK
    # an fp32 input gradient is not offered, and no other dtype exists
    assert need(1, [layer()], dtype=1)[0] == EDTYPE
    for op in (0, 2):
        assert run_op(op, [layer()], dtype=9) == EDTYPE
    assert need(7, [layer()])[0] == EINVAL
    assert _q8.lib().ns_q8_workspace_bytes(0, arr([layer()]), 1, 0, None) == EINVAL


@pytest.mark.parametrize("op", [0, 1, 2])
def test_counts_and_empty_layers(op):
    assert run_op(op, [], count=-1) == EINVAL
    assert run_op(op, [], count=0) == OK
    assert run_op(op, [], count=2) == EINVAL
    empty = dict(xq=None, wq=None, dy=None, x_scale=None, w_scale=None, out=None)
    # no outputs: nothing is read, checked or written
    shapes = {0: [dict(tokens=0), dict(out_features=0)], 1: [dict(tokens=0), dict(in_features=0)],
              2: [dict(out_features=0), dict(in_features=0)]}[op]
    assert run_op(op, [layer(**empty, **s) for s in shapes]) == OK, ns.last_error()


def test_outputs_must_not_overlap():
    for op in (0, 1, 2):
        assert run_op(op, [layer(), layer()]) == EINVAL and "overlap" in ns.last_error()
    # rows interleaved at one pitch are apart; a column further they are not
    side = dict(out_features=6, ld_out=24)
    assert need(0, [layer(**side), layer(out=0x60000 + 12, **side), layer(out=0x60000 + 24, **side)])[0] == OK
    assert need(0, [layer(**side), layer(out=0x60000 + 10, **side)])[0] == EINVAL
    assert need(0, [layer(**side), layer(out=0x60000 + 44, **side)])[0] == EINVAL   # into the next row
    assert need(0, [layer(**side), layer(out=0x60000 + 48 * 4, **side)])[0] == OK
    # a single row inside the gap of another output's rows
    assert need(0, [layer(**side), layer(tokens=1, out=0x60000 + 16, out_features=6)])[0] == OK
    assert need(0, [layer(**side), layer(tokens=1, out=0x60000 + 50, out_features=6)])[0] == EINVAL


def test_workspace():
    # few outputs and a long sum: pieces that meet in a workspace
    long = layer(tokens=8192, out_features=18, in_features=2304, ld_xq=2304, ld_dy=18, ld_out=2304)
    rc, n = need(2, [long])
    assert rc == OK and n >= 2 * 18 * 2304 * 4
    # per layer, whatever else is in the list
    other = layer(tokens=8192, out_features=18, in_features=2304, ld_xq=2304, ld_dy=18, ld_out=2304, out=0x9000000)
    assert need(2, [long, other]) == (OK, 2 * n)
    assert run_op(2, [long]) == EINVAL and "workspace" in ns.last_error()
    assert run_op(2, [long], ws=0x100000, nbytes=n - 1) == EINVAL
    assert run_op(2, [long], ws=0x100008, nbytes=n) == EINVAL
    # enough tiles: no pieces
    assert need(2, [layer(tokens=512, out_features=8192, in_features=6144, ld_xq=6144, ld_dy=8192,
                          ld_out=6144)]) == (OK, 0)
    # operands at other alignments are copied to rows of 16 bytes first
    odd = layer(tokens=512, out_features=8192, in_features=6144, ld_xq=6145, ld_dy=8192, ld_out=6144)
    assert need(2, [odd]) == (OK, 512 * 6144)
    odd.xq, odd.ld_xq = 0x10001, 6144
    assert need(2, [odd]) == (OK, 512 * 6144)


def test_too_large_an_output_is_refused():
    huge = layer(tokens=1 << 24, out_features=1 << 21, in_features=8, ld_out=1 << 21)
    assert need(0, [huge])[0] == EINVAL


def test_binding_refusals():
    q, s = torch.zeros((4, 8), dtype=torch.int8), torch.ones(4)
    w, ws = torch.zeros((6, 8), dtype=torch.int8), torch.ones(6)
    dy, g = torch.zeros((4, 6), dtype=torch.bfloat16), torch.zeros((6, 8))
    for call in (lambda: ns.quantize_rows([torch.zeros(4, 8)]), lambda: ns.dequantize_rows([(q, s)]),
                 lambda: ns.q8_matmul([(q, s)], [(w, ws)]), lambda: ns.q8_grad_input([dy], [(w, ws)]),
                 lambda: ns.q8_grad_weight([dy], [(q, s)], [g])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        ns.quantize_rows([torch.zeros((4, 8), dtype=torch.float16)])
    with pytest.raises(TypeError):
        ns.q8_matmul([(q, s)], [(w, ws)], dtype=torch.float16)
    with pytest.raises(ValueError):
        ns.q8_matmul([(q, s)], [])
    assert ns.quantize_rows([]) == [] and ns.dequantize_rows([]) == [] and ns.q8_matmul([], []) == []
    assert ns.q8_grad_input([], []) == [] and ns.q8_grad_weight([], [], []) == []


def test_new_tensors_of_one_block_are_their_own_to_autograd():
    """Each can be modified in place, by itself, within a graph."""
    a, b, c = _q8._empty([(2, 16), (0, 16), (3, 16)], torch.float32, "cpu")
    assert [t.shape for t in (a, b, c)] == [(2, 16), (0, 16), (3, 16)]
    a.zero_(), c.fill_(2.0)
    bias = torch.ones(16, requires_grad=True)
    a.add_(bias)
    square = (a * a).sum()
    c.mul_(3.0)   # not a version of `a`
    square.backward()
    assert not c.requires_grad and torch.equal(bias.grad, torch.full((16,), 4.0)) and bool((c == 6).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", [1, 3, 8, 12, 1027])
def test_new_tensors_are_aligned(width, dtype):
    shapes = [(5, width), (0, width), (1, width), (16, width), (7, width)]
    new = _q8._empty(shapes, dtype, "cpu")
    assert [tuple(t.shape) for t in new] == shapes
    assert all(t.is_contiguous() and t.data_ptr() % 16 == 0 for t in new)
    for i, t in enumerate(new):
        t.fill_(i)
    assert all(bool((t == i).all()) for i, t in enumerate(new))
