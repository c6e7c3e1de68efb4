"""The 8-bit linear-layer calls on the GPU against the formulas in 64 bits.

Bounds, derived (u = half a step: bf16 2^-8, fp32 2^-24):
  quantise, dequantise   the definition is exact: equality
  matmul     the integer sum is exact; its rounding to fp32 and two products in
             fp32, then the output: |ref| ((1 + 2^-24)^3 (1 + u_out) - 1)
  gradients  a term dy q s is off by the rounding of q s, (1 + 2^-24)(1 + 2^-8)
             - 1 of it, nothing when s is a power of two and q s a normal
             number; the product of two bf16 values is exact in fp32; K sums in
             fp32 are off by at most K 2^-23 of the sum of magnitudes in any
             order (a whole step each, should an adder truncate), the join of
             pieces and beta G included (K + 40 sums); then the output
"""
import math

import pytest
import torch

import newton_schulz_04_amd as ns
from nsutil import TOL, oracle_run, rel_err

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
U = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ns.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def pitched(rows, cols, pitch, offset, dtype, fill):
    """A rows x cols view at a pitch, `offset` elements into a buffer that
    holds `fill` all around it; and the buffer."""
    buf = torch.full((offset + rows * pitch + pitch,), fill, dtype=dtype, device="cuda")
    return buf[offset:offset + rows * pitch].view(rows, pitch)[:, :cols], buf


def outside_is(buf, view, value):
    """Every element of buf outside the view still holds `value`."""
    keep = buf.clone()
    offset = (view.data_ptr() - buf.data_ptr()) // buf.element_size()
    rows, cols = view.shape
    pitch = view.stride(0) if rows > 1 else cols
    if view.numel():
        torch.as_strided(keep, (rows, cols), (pitch, 1), offset).fill_(value)
    return bool((keep == value).all()) or (value != value and bool(torch.isnan(keep.float()).all()))


def definition(x, pow2):
    """(q, s) in 64 bits on the CPU, row by row from the definition."""
    v = x.detach().cpu().double()
    top = v.abs().amax(1)
    if pow2:
        s = torch.tensor([2.0 ** -126 if t == 0 else 2.0 ** max(-126, next(
            e for e in range(-160, 130) if 127 * 2.0 ** e >= t)) for t in top.tolist()], dtype=torch.float64)
    else:
        s = (top / 127).float().double().clamp_min(2.0 ** -126)
    q = torch.round(v / s[:, None])
    return q.to(torch.int8), s.float()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows,cols,pitch,offset", [
    (1, 1, 1, 0), (3, 7, 7, 0), (5, 64, 64, 0), (130, 257, 260, 3), (17, 2048, 2048, 0), (9, 2049, 2056, 0),
    (6, 6144, 6144, 0), (3, 8193, 8200, 1), (2, 20000, 20000, 0), (1, 100001, 100001, 0),
])
def test_quantize_is_the_definition(rows, cols, pitch, offset, pow2, dtype):
    g = gen(rows * 1000 + cols)
    x, _ = pitched(rows, cols, pitch, offset, dtype, float("nan"))
    v = torch.randn((rows, cols), generator=g, device="cuda") * torch.exp(3 * torch.randn((rows, 1), generator=g, device="cuda"))
    x.copy_(v.to(dtype))
    (q, s), = ns.quantize_rows([x], pow2=pow2)
    want_q, want_s = definition(x, pow2)
    assert torch.equal(s.cpu(), want_s)
    assert torch.equal(q.cpu(), want_q)
    for out in (BF16, FP32):
        back, = ns.dequantize_rows([(q, s)], dtype=out)
        assert torch.equal(back.cpu(), (want_q.double() * want_s.double()[:, None]).float().to(out))


@pytest.mark.parametrize("pow2", [False, True])
def test_quantize_ties_and_extremes(pow2):
    """Rows whose quotients are exact halves, subnormal rows, zero rows, rows of
    one value, rows up to the largest float."""
    half = torch.arange(-127, 127, device="cuda").float() + 0.5
    rows = []
    for top, scale in ((127.0, 1.0), (127.0, 2.0 ** -20), (127.0, 2.0 ** 100), (127.0, 3.0), (127.0, 1.7)):
        rows.append(torch.cat([half, torch.tensor([top, -top], device="cuda")]) * scale)
    n = rows[0].numel()
    rows.append(torch.zeros(n, device="cuda"))
    rows.append(torch.full((n,), 5.5, device="cuda"))
    rows.append(torch.linspace(-1, 1, n, device="cuda") * 1e-42)
    rows.append(torch.linspace(-1, 1, n, device="cuda") * 3.1e-36)
    rows.append(torch.linspace(-1, 1, n, device="cuda") * 2.0 ** -119)
    rows.append(torch.linspace(-1, 1, n, device="cuda") * 3.4028234e38)
    rows.append(torch.linspace(-1, 1, n, device="cuda") * 127 / 64)     # 127 2^e exactly on top
    x = torch.stack(rows)
    (q, s), = ns.quantize_rows([x], pow2=pow2)
    want_q, want_s = definition(x, pow2)
    assert torch.equal(s.cpu(), want_s)
    assert torch.equal(q.cpu(), want_q)


def test_quantize_nan_and_inf_rows():
    x = torch.randn((6, 300), generator=gen(1), device="cuda")
    x[1, 7], x[3, 299], x[4, 0] = float("nan"), float("inf"), -float("inf")
    (q, s), = ns.quantize_rows([x])
    bad = torch.tensor([False, True, False, True, True, False], device="cuda")
    assert torch.equal(torch.isnan(s), bad)
    assert not bool(q[bad].any())
    back, = ns.dequantize_rows([(q, s)], dtype=FP32)
    assert torch.equal(torch.isnan(back), bad[:, None].expand_as(back))
    want_q, want_s = definition(x[~bad], False)
    assert torch.equal(q[~bad].cpu(), want_q) and torch.equal(s[~bad].cpu(), want_s)


def test_rows_write_nothing_else():
    """Row gaps and the bytes around outputs stay as they were, at odd pitches."""
    from newton_schulz_04_amd import _q8
    for rows, cols, pq, offset in [(5, 37, 41, 3), (4, 2051, 2053, 1), (3, 16, 16, 0)]:
        x = torch.randn((rows, cols), generator=gen(cols), device="cuda")
        q, buf = pitched(rows, cols, pq, offset, torch.int8, 99)
        scale = torch.full((rows + 2,), 7.0, device="cuda")
        arr = (_q8.RowsStruct * 1)(_q8.RowsStruct(rows, cols, x.data_ptr(), cols, q.data_ptr(), pq, scale[1:].data_ptr()))
        st = torch.cuda.current_stream().cuda_stream
        assert _q8.lib().ns_q8_quantize(arr, 1, 0, 1, st) == 0, ns.last_error()
        want_q, want_s = definition(x, False)
        assert torch.equal(q.cpu(), want_q) and torch.equal(scale[1:-1].cpu(), want_s)
        assert scale[0] == 7 and scale[-1] == 7 and outside_is(buf, q, 99)
        back, bb = pitched(rows, cols, pq, offset, FP32, 5.0)
        arr[0].values, arr[0].ld_values = back.data_ptr(), pq
        assert _q8.lib().ns_q8_dequantize(arr, 1, 1, st) == 0, ns.last_error()
        assert torch.equal(back, q.float() * scale[1:-1, None]) and outside_is(bb, back, 5.0)


# --- products ------------------------------------------------------------------
def q8_matrix(rows, cols, g, pow2=False, pitch=None, offset=0, full=False):
    """A random 8-bit matrix at a pitch; the bytes between its rows are -77."""
    q, _ = pitched(rows, cols, cols if pitch is None else pitch, offset, torch.int8, -77)
    lo = -128 if full else -127
    q.copy_(torch.randint(lo, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8))
    s = torch.exp2(torch.randint(-9, -3, (rows,), generator=g, device="cuda").float())
    if not pow2:
        s = s * (1 + torch.rand(rows, generator=g, device="cuda"))
    return q, s


def grads_in(rows, cols, g, pitch=None, offset=0):
    dy, _ = pitched(rows, cols, cols if pitch is None else pitch, offset, BF16, float("nan"))
    dy.copy_((torch.randn((rows, cols), generator=g, device="cuda") * torch.exp(torch.randn((rows, 1), generator=g, device="cuda"))).to(BF16))
    if rows > 3:
        dy[rows // 2] = 0
    return dy


def wide(pair):
    return pair[0].double() * pair[1].double()[:, None]


def product_of(x, w):
    """Xq Wq^T: the integer sums are exact in 64 bits, then the scales."""
    sums = x[0].double() @ w[0].double().T.contiguous()
    return sums * x[1].double()[:, None] * w[1].double()


def check(got, ref, tol):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} off, first at "
                                 f"{bad.nonzero()[0].tolist()}: {got[bad][0].item()} for {ref[bad][0].item()}")


def matmul_bound(ref, dtype):
    return ref.abs() * ((1 + 2.0 ** -24) ** 3 * (1 + U[dtype]) - 1 + 1e-12)


def grad_bound(ref, mags, terms, dtype, pow2):
    ux = 0.0 if pow2 else (1 + 2.0 ** -24) * (1 + 2.0 ** -8) - 1
    inner = mags * (ux + (terms + 40) * 2.0 ** -23)
    return inner + (ref.abs() + inner) * U[dtype] + 1e-35


SIZES = [(1, 1, 1), (1, 18, 2304), (2, 64, 32), (3, 5, 7), (7, 33, 65), (16, 128, 256), (17, 130, 200),
         (33, 257, 520), (64, 64, 64), (100, 300, 1000), (129, 511, 96), (255, 256, 257), (256, 512, 768),
         (300, 770, 1536), (513, 1030, 640), (1000, 18, 2304), (2500, 24, 100), (70, 2048, 6144), (8, 8192, 320),
         (640, 512, 544)]
# many 128 x 128 tiles, and enough outputs for the 256 x 256 ones: sums that end
# inside a slot, at its end and within the first, outputs that end inside a
# tile; the last leaves a part round of large tiles, which runs as halves
LARGE = [(2100, 2064, 2208), (2101, 2058, 2201), (2100, 2064, 24), (2100, 5, 2201), (3, 2058, 2201),
         (4000, 1040, 1056), (1025, 4097, 64), (2048, 2048, 2048), (3330, 3333, 3341), (3500, 3400, 801),
         (4300, 4112, 4112)]
# pitches: contiguous; padded to 16 bytes; odd, at an odd offset
LAYOUTS = ["contiguous", "padded", "odd"]


def layout(cols, kind, elt):
    if kind == "contiguous":
        return cols, 0
    if kind == "padded":
        unit = 16 // elt
        return -(-cols // unit) * unit + unit, unit
    return cols + 3, 1


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("kind", LAYOUTS)
@pytest.mark.parametrize("t,o,k", SIZES + LARGE)
def test_matmul(t, o, k, kind, dtype):
    g = gen(t + 31 * o + 77 * k)
    pq, off = layout(k, kind, 1)
    x, w = q8_matrix(t, k, g, pitch=pq, offset=off, full=True), q8_matrix(o, k, g, pitch=pq, offset=off, full=True)
    po, oo = layout(o, kind, 2 if dtype == BF16 else 4)
    y, buf = pitched(t, o, po, oo, dtype, 3.0)
    got, = ns.q8_matmul([x], [w], dtype=dtype, out=[y])
    assert got is y
    ref = product_of(x, w)
    check(got, ref, matmul_bound(ref, dtype))
    assert outside_is(buf, y, 3.0)


@pytest.mark.parametrize("kind", LAYOUTS)
@pytest.mark.parametrize("t,o,k", SIZES + LARGE)
def test_grad_input(t, o, k, kind):
    g = gen(t + 31 * o + 79 * k)
    pw, ow = layout(k, kind, 1)
    pd, od = layout(o, kind, 2)
    w, dy = q8_matrix(o, k, g, pitch=pw, offset=ow), grads_in(t, o, g, pitch=pd, offset=od)
    dx, buf = pitched(t, k, *layout(k, kind, 2), BF16, 3.0)
    ns.q8_grad_input([dy], [w], out=[dx])
    ref, mags = dy.double() @ wide(w), dy.double().abs() @ wide(w).abs()
    check(dx, ref, grad_bound(ref, mags, o, BF16, False))
    assert outside_is(buf, dx, 3.0)


@pytest.mark.parametrize("dtype,beta,pow2", [(BF16, 0.0, False), (BF16, 0.9375, True), (FP32, 1.0, True),
                                             (FP32, 0.5, False)])
@pytest.mark.parametrize("kind", LAYOUTS)
@pytest.mark.parametrize("t,o,k", SIZES + LARGE)
def test_grad_weight(t, o, k, kind, dtype, beta, pow2):
    g = gen(t + 31 * o + 83 * k)
    px, ox = layout(k, kind, 1)
    pd, od = layout(o, kind, 2)
    x, dy = q8_matrix(t, k, g, pow2=pow2, pitch=px, offset=ox), grads_in(t, o, g, pitch=pd, offset=od)
    out, buf = pitched(o, k, *layout(k, kind, 2 if dtype == BF16 else 4), dtype, 3.0)
    out.copy_(torch.randn((o, k), generator=g, device="cuda").to(dtype))
    before = out.double()
    if beta == 0.0:
        out.fill_(float("nan"))
    ns.q8_grad_weight([dy], [x], [out], beta=beta)
    dt = dy.double().T.contiguous()
    ref, mags = beta * before + dt @ wide(x), beta * before.abs() + dt.abs() @ wide(x).abs()
    check(out, ref, grad_bound(ref, mags, t, dtype, pow2))
    assert outside_is(buf, out, 3.0)


@pytest.mark.parametrize("t", [31, 32, 33, 64, 65, 127, 1025, 4096])
@pytest.mark.parametrize("o,k", [(1, 15), (7, 300), (8, 16), (9, 17), (64, 129), (65, 130)])
def test_grad_weight_of_few_rows(t, o, k):
    """Around the sizes at which few rows take a kernel of their own: the last
    rows of contiguous operands end where their memory's contents change."""
    g = gen(t + 31 * o + 89 * k)
    dy = torch.full((t * o + 64,), float("nan"), dtype=BF16, device="cuda")[32:-32].view(t, o)
    dy.copy_(grads_in(t, o, g))
    x = q8_matrix(t, k, g, offset=1)
    out = torch.full((o, k), float("nan"), device="cuda")
    ns.q8_grad_weight([dy], [x], [out])
    dt = dy.double().T.contiguous()
    check(out, dt @ wide(x), grad_bound(dt @ wide(x), dt.abs() @ wide(x).abs(), t, FP32, False))


@pytest.mark.parametrize("beta", [0.0, 0.5])
def test_layers_without_tokens_or_width(beta):
    g = gen(5)
    x0, x1 = q8_matrix(0, 48, g), q8_matrix(9, 48, g)
    w = q8_matrix(20, 48, g)
    y0, y1 = ns.q8_matmul([x0, x1], [w, w])
    assert y0.shape == (0, 20) and y1.shape == (9, 20)
    dy0, dy1 = grads_in(0, 20, g), grads_in(9, 20, g)
    dx0, dx1 = ns.q8_grad_input([dy0, dy1], [w, w])
    assert dx0.shape == (0, 48) and bool(dx1.any())
    gr = [torch.full((20, 48), 2.0, device="cuda") for _ in range(2)]
    ns.q8_grad_weight([dy0, dy1], [x0, x1], gr, beta=beta)
    assert bool((gr[0] == 2 * beta).all()) and not bool((gr[1] == 2 * beta).all())
    # sums over nothing are zero
    e = (torch.empty((3, 0), dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda"))
    f = (torch.empty((5, 0), dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda"))
    y, = ns.q8_matmul([e], [f], out=[torch.full((3, 5), 9.0, dtype=BF16, device="cuda")])
    assert not bool(y.any())
    dx, = ns.q8_grad_input([torch.empty((3, 0), dtype=BF16, device="cuda")],
                           [(torch.empty((0, 6), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))])
    assert dx.shape == (3, 6) and not bool(dx.any())


def ragged(seed, n, o, k, pow2=False):
    g = gen(seed)
    ts = [(37 * i * i + 11 * i) % 190 if i % 5 != 3 else 0 for i in range(n)]
    xs = [q8_matrix(t, k + i % 3, g, pow2=pow2, pitch=-(-(k + i % 3) // 16) * 16) for i, t in enumerate(ts)]
    ws = [q8_matrix(o + i % 2, k + i % 3, g, pitch=-(-(k + i % 3) // 16) * 16) for i in range(n)]
    dys = [grads_in(t, o + i % 2, g) for i, t in enumerate(ts)]
    return xs, ws, dys


def test_lists_give_the_bits_of_single_calls():
    """More layers than one launch takes, ragged and some without tokens."""
    xs, ws, dys = ragged(7, 90, 72, 144)
    ys, dxs = ns.q8_matmul(xs, ws), ns.q8_grad_input(dys, ws)
    gs = ns.q8_grad_weight(dys, xs, [torch.ones((dy.shape[1], x[0].shape[1]), device="cuda") for dy, x in zip(dys, xs)], beta=0.5)
    for i in reversed(range(90)):
        assert torch.equal(ys[i], ns.q8_matmul([xs[i]], [ws[i]])[0])
        assert torch.equal(dxs[i], ns.q8_grad_input([dys[i]], [ws[i]])[0])
        one = torch.ones((dys[i].shape[1], xs[i][0].shape[1]), device="cuda")
        assert torch.equal(gs[i], ns.q8_grad_weight([dys[i]], [xs[i]], [one], beta=0.5)[0])
        ref = product_of(xs[i], ws[i])
        check(ys[i], ref, matmul_bound(ref, BF16))
    many = [torch.randn((3, 20 + i), generator=gen(i), device="cuda") for i in range(150)]
    for (q, s), x in zip(ns.quantize_rows(many), many):
        wq, wsc = definition(x, False)
        assert torch.equal(q.cpu(), wq) and torch.equal(s.cpu(), wsc)


@pytest.mark.parametrize("t,o,k", [(40, 70, 96), (300, 513, 520), (1, 256, 512)])
def test_nan_and_inf_stay_in_their_rows(t, o, k):
    """A NaN or Inf reaches exactly the sums that hold it; NaN between the rows
    of dY (a slice of a wider gradient) reaches nothing."""
    g = gen(t + o)
    x, w = q8_matrix(t, k, g), q8_matrix(o, k, g)
    dy = grads_in(t, o, g, pitch=2 * o + 16, offset=8)
    x[1][t - 1] = float("nan")
    y, = ns.q8_matmul([x], [w])
    bad = torch.zeros((t, o), dtype=torch.bool, device="cuda")
    bad[t - 1] = True
    assert torch.equal(torch.isnan(y), bad)
    dy[t - 1, o // 2] = float("nan")
    dy[0, o - 1] = float("inf")
    dx, = ns.q8_grad_input([dy], [w])
    bad = torch.zeros((t, k), dtype=torch.bool, device="cuda")
    bad[t - 1] = bad[0] = True
    assert torch.equal(~torch.isfinite(dx), bad)
    x[1][t - 1] = 0.5
    gw, = ns.q8_grad_weight([dy], [x], [torch.zeros((o, k), device="cuda")])
    bad = torch.zeros((o, k), dtype=torch.bool, device="cuda")
    bad[o // 2] = bad[o - 1] = True
    assert torch.equal(~torch.isfinite(gw), bad)


def test_gradients_against_differences():
    """One integer step of a weight or an input changes sum(dY Y) by its
    gradient times the scale. Small integers and power-of-two scales make Y
    exact in fp32, so the differences are exact and only the fp32 sums of the
    gradients differ from them."""
    g = gen(11)
    t, o, k = 21, 14, 40
    x, w = q8_matrix(t, k, g, pow2=True), q8_matrix(o, k, g, pow2=True)
    for q, s in (x, w):
        q.clamp_(-100, 100)
        s.fill_(2.0 ** -5)
    dy = grads_in(t, o, g)
    gw, = ns.q8_grad_weight([dy], [x], [torch.empty((o, k), device="cuda")])
    dx, = ns.q8_grad_input([dy], [w])
    base = ns.q8_matmul([x], [w], dtype=FP32)[0].double()
    for i in range(0, k, 7):
        for r in range(o):
            w2 = (w[0].clone(), w[1])
            w2[0][r, i] += 1
            d = (dy.double() * (ns.q8_matmul([x], [w2], dtype=FP32)[0].double() - base)).sum() / w[1][r].double()
            mag = (dy[:, r].double().abs() * wide(x)[:, i].abs()).sum()
            assert abs(gw[r, i].double() - d) <= mag * (t + 40) * 2.0 ** -23
        for r in range(t):
            x2 = (x[0].clone(), x[1])
            x2[0][r, i] += 1
            d = (dy.double() * (ns.q8_matmul([x2], [w], dtype=FP32)[0].double() - base)).sum() / x[1][r].double()
            mag = (dy[r].double().abs() * wide(w)[:, i].abs()).sum()
            assert abs(dx[r, i].double() - d) <= mag * (o + 40) * 2.0 ** -23 + (d.abs() + 1e-9) * 2.0 ** -8


def test_a_layers_step_into_the_orthogonalization():
    """As they are used: a layer's input is kept in 8 bits, the forward product
    takes it and the 8-bit weights, the backward pass reads it back through the
    weight gradient, which accumulates into momentum; the momentum is
    orthogonalised."""
    g = gen(21)
    shapes = [(300, 96, 136), (0, 96, 136), (77, 18, 520)]
    x = [torch.randn((t, k), generator=g, device="cuda").to(BF16) for t, _, k in shapes]
    w = [torch.randn((o, k), generator=g, device="cuda") / k ** 0.5 for _, o, k in shapes]
    dy = [torch.randn((t, o), generator=g, device="cuda").to(BF16) for t, o, _ in shapes]
    mom = [torch.randn((o, k), generator=g, device="cuda").to(BF16) for _, o, k in shapes]
    start = [m.double() for m in mom]
    xq, wq = ns.quantize_rows(x, pow2=True), ns.quantize_rows(w)
    y, dx = ns.q8_matmul(xq, wq), ns.q8_grad_input(dy, wq)
    ns.q8_grad_weight(dy, xq, mom, beta=0.9375)
    for i, (t, o, k) in enumerate(shapes):
        # a row's quantisation is off by half a scale per value
        assert bool(((wide(xq[i]) - x[i].double()).abs() <= 0.5 * xq[i].scale.double()[:, None]).all())
        ref = product_of(xq[i], wq[i])
        check(y[i], ref, matmul_bound(ref, BF16))
        ref, mags = dy[i].double() @ wide(wq[i]), dy[i].double().abs() @ wide(wq[i]).abs()
        check(dx[i], ref, grad_bound(ref, mags, o, BF16, False))
        dt = dy[i].double().T.contiguous()
        ref, mags = 0.9375 * start[i] + dt @ wide(xq[i]), 0.9375 * start[i].abs() + dt.abs() @ wide(xq[i]).abs()
        check(mom[i], ref, grad_bound(ref, mags, t, BF16, True))
    held = [m.cpu() for m in mom]
    ns.orthogonalize(mom)
    for m, h in zip(mom, held):
        assert rel_err(m.cpu(), oracle_run(h)) <= TOL[BF16]


def test_side_stream_and_early_frees():
    """On a stream of its own, with inputs dropped right after the calls."""
    side = torch.cuda.Stream()
    g = gen(31)
    x, w, dy = q8_matrix(700, 640, g), q8_matrix(48, 640, g), grads_in(700, 48, g)
    want = (ns.q8_matmul([x], [w])[0], ns.q8_grad_input([dy], [w])[0],
            ns.q8_grad_weight([dy], [x], [torch.empty((48, 640), device="cuda")])[0])
    torch.cuda.synchronize()
    gw = torch.empty((48, 640), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    y, = ns.q8_matmul([x], [w], stream=side)
    dx, = ns.q8_grad_input([dy], [w], stream=side)
    ns.q8_grad_weight([dy], [x], [gw], stream=side)
    del x, w, dy
    junk = [torch.full((700, 640), 55, dtype=torch.int8, device="cuda") for _ in range(8)]
    side.synchronize()
    del junk
    for a, b in zip((y, dx, gw), want):
        assert torch.equal(a, b)


def test_captured_graphs_replay():
    """Two graphs captured from the calls, replayed in turn several times with
    eager work and synchronizations between, against the eager results."""
    def make(seed, t, o, k):
        g = gen(seed)
        return dict(x=torch.randn((t, k), generator=g, device="cuda").to(BF16), dy=grads_in(t, o, g),
                    w=ns.quantize_rows([torch.randn((o, k), generator=g, device="cuda")])[0],
                    g=torch.zeros((o, k), device="cuda"))

    def step(s):
        xq = ns.quantize_rows([s["x"]])
        s["y"], = ns.q8_matmul(xq, [s["w"]])
        s["dx"], = ns.q8_grad_input([s["dy"]], [s["w"]])
        ns.q8_grad_weight([s["dy"]], xq, [s["g"]], beta=0.5)

    sets = [make(41, 900, 24, 300), make(42, 33, 260, 512)]
    graphs = []
    for s in sets:
        warm = torch.cuda.Stream()
        warm.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(warm):
            step(s)
        torch.cuda.current_stream().wait_stream(warm)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(s)
        graphs.append(graph)
        s["g"].zero_()
    eager = [dict(s, g=s["g"].clone()) for s in sets]
    for replay in range(3):
        for s, e, graph in zip(sets, eager, graphs):
            fresh = torch.randn(s["x"].shape, generator=gen(100 + replay), device="cuda").to(BF16)
            s["x"].copy_(fresh)
            graph.replay()
            step(e)     # reads the same x; its own g
            torch.cuda.synchronize()
            for name in ("y", "dx", "g"):
                assert torch.equal(s[name], e[name]), (replay, name)


def test_long_rows_pass_32_bit_offsets():
    """Row offsets beyond 2^31 bytes: a tall checkpoint, its last tokens used."""
    rows, k = (1 << 31) // 2048 + 300, 2048
    q = torch.zeros((rows, k), dtype=torch.int8, device="cuda")
    s = torch.zeros(rows, device="cuda")
    g = gen(51)
    q[-200:] = torch.randint(-127, 128, (200, k), generator=g, device="cuda", dtype=torch.int8)
    s[-200:] = 0.25
    dy = torch.zeros((rows, 16), dtype=BF16, device="cuda")
    dy[-200:] = torch.randn((200, 16), generator=g, device="cuda").to(BF16)
    gw, = ns.q8_grad_weight([dy], [(q, s)], [torch.empty((16, k), device="cuda")])
    d, x = dy[-200:].double().T.contiguous(), q[-200:].double() * 0.25
    check(gw, d @ x, grad_bound(d @ x, d.abs() @ x.abs(), 240, FP32, True))
    w = q8_matrix(24, k, g)
    y, = ns.q8_matmul([(q, s)], [w])
    ref = product_of((q[-200:], s[-200:]), w)
    check(y[-200:], ref, matmul_bound(ref, BF16))
    assert not bool(y[:-200].any())
    back, = ns.dequantize_rows([(q[-70000:], s[-70000:])])
    assert torch.equal(back[-200:], (x).to(BF16))


@pytest.mark.parametrize("seed", range(6))
def test_drawn_lists(seed):
    """Lists of random layers of every kind and layout in one call."""
    import random
    r, g = random.Random(seed), gen(1000 + seed)
    xs, ws, dys, gs = [], [], [], []
    for _ in range(r.randint(1, 9)):
        t, o, k = (int(math.exp(r.uniform(0, math.log(m)))) for m in (700, 900, 900))
        if r.random() < 0.15:
            t = 0
        kind = r.choice(LAYOUTS)
        p, off = layout(k, kind, 1)
        xs.append(q8_matrix(t, k, g, pitch=p, offset=off))
        ws.append(q8_matrix(o, k, g, pitch=p, offset=off))
        dys.append(grads_in(t, o, g, *layout(o, kind, 2)))
        gs.append(torch.randn((o, k), generator=g, device="cuda"))
    before = [v.double() for v in gs]
    ys, dxs = ns.q8_matmul(xs, ws, dtype=FP32), ns.q8_grad_input(dys, ws)
    ns.q8_grad_weight(dys, xs, gs, beta=0.75)
    for x, w, dy, y, dx, gw, b in zip(xs, ws, dys, ys, dxs, gs, before):
        ref = product_of(x, w)
        check(y, ref, matmul_bound(ref, FP32))
        ref = dy.double() @ wide(w)
        check(dx, ref, grad_bound(ref, dy.double().abs() @ wide(w).abs(), dy.shape[1], BF16, False))
        d = dy.double().T.contiguous()
        ref = 0.75 * b + d @ wide(x)
        check(gw, ref, grad_bound(ref, 0.75 * b.abs() + d.abs() @ wide(x).abs(), dy.shape[0], FP32, False))


@pytest.mark.parametrize("slots", [3, 4, 5, 13, 14, 15, 64, 65, 66, 67])
def test_same_bits_from_slow_memory(slots):
    """Operands that come late, from memory that a copy on another stream keeps
    busy, give the bits of operands at hand: for sums of each length modulo the
    kernels' rings."""
    g = gen(slots)
    m, n = 1100, 1232
    busy, side = torch.empty(1 << 29, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    k8, k16 = 64 * slots - 7, 32 * slots - 7
    p8, p16 = -(-k8 // 16) * 16, -(-k16 // 8) * 8
    x, w = q8_matrix(m, k8, g, pitch=p8), q8_matrix(n, k8, g, pitch=p8)
    dy, wi = grads_in(m, k16, g, pitch=p16), q8_matrix(k16, n, g)
    dt, xw = grads_in(k16, 1112, g), q8_matrix(k16, n, g)

    def run():
        gw = torch.ones((1112, n), device="cuda")
        return (*ns.q8_matmul([x], [w]), *ns.q8_grad_input([dy], [wi]), *ns.q8_grad_weight([dt], [xw], [gw], beta=0.5))

    first = run()
    torch.cuda.synchronize()
    check(first[0], product_of(x, w), matmul_bound(product_of(x, w), BF16))
    for _ in range(4):
        with torch.cuda.stream(side):
            for _ in range(3):
                busy.add_(1)
        again = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
