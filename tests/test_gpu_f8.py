"""The 8-bit floating-point calls on the GPU against the formulas in 64 bits.

Bounds, derived (u = half a step: bf16 2^-8, fp32 2^-24):
  quantise, dequantise   the definition is exact: equality
  matmul, whole numbers  products of small whole numbers, scales of small powers of two:
             every product and sum is exact in any order (groups of eight products lie
             within 13 bits, sums below 2^24), so only the output rounds: equality
  matmul, bf16   the 8-bit MFMA cuts the products of a group of eight k at 2^-13 of the
             largest one's power of two, so a group is off by at most 8 2^-13 max |p|;
             fp32 sums: K 2^-23 of the sum of magnitudes in any order; fp32 scales: three
             roundings of a block's sum (2^-24 each, of its magnitude); then the output
  matmul, fp32   products of widened values are exact: the sums, the scales, the output
"""
import pytest
import torch

import newton_schulz_04_amd as ns

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
E4, E5, E8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
U = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ns.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(seed, *shape):
    return torch.randn(shape, generator=gen(seed), device="cuda")


def blocks(n):
    return -(-n // 128)


# --- the definition, on the CPU in 64 bits -------------------------------------
SHAPE = {E4: (3, -6, 448.0), E5: (2, -14, 57344.0)}   # mantissa bits, least exponent, largest


def to_grid(y, fmt):
    """y (float64) to the nearest number of the format, ties to even."""
    mant, least, top = SHAPE[fmt]
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** least)))
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64), e - mant)
    return (torch.round(y / step) * step).clamp(-top, top)


def definition(x, fmt, pow2, square):
    """(values of q, scales of ceil(cols/128) x rows or x ceil(rows/128)) in float64."""
    v = x.detach().cpu().double()
    rows, cols = v.shape
    tall = 128 if square else 1
    q = torch.zeros_like(v)
    scale = torch.zeros((blocks(cols), -(-rows // tall)), dtype=torch.float64)
    top = SHAPE[fmt][2]
    for b in range(blocks(cols)):
        for r in range(-(-rows // tall)):
            part = v[r * tall:(r + 1) * tall, 128 * b:128 * b + 128]
            m = float(part.abs().max())
            if pow2:
                e = -126
                while top * 2.0 ** e < m:
                    e += 1
                s = 2.0 ** e
            else:
                s = max(float(torch.tensor(m / top, dtype=torch.float64).float()), 2.0 ** -126)
            scale[b, r] = s
            q[r * tall:(r + 1) * tall, 128 * b:128 * b + 128] = to_grid(part / s, fmt)
    return q, scale


def spread(scale, rows, cols):
    """Each value's scale."""
    s = scale.double().repeat_interleave(128, 0)[:cols].T
    return s if s.shape[0] == rows else s.repeat_interleave(128, 0)[:rows]


def values(pair):
    q, s = pair
    # (one-byte scales by way of the bits of 2^(b - 127) in 64 bits: the device's pow is
    # not exact)
    if s.dtype == E8:
        b = s.contiguous().view(torch.uint8).long()
        s = torch.where(b == 255, NAN, ((b + 1023 - 127) << 52).view(torch.float64))
    return q.float().double() * spread(s.double(), *q.shape)


def pitched(rows, cols, pitch, offset, dtype, fill):
    buf = torch.full((offset + rows * pitch + pitch,), fill, dtype=dtype, device="cuda")
    return buf[offset:offset + rows * pitch].view(rows, pitch)[:, :cols], buf


# --- quantise ------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("rows,cols,pitch,offset", [
    (1, 1, 1, 0), (1, 128, 128, 0), (3, 7, 9, 1), (130, 257, 264, 0), (128, 128, 128, 0), (129, 100, 101, 3),
    (300, 16, 16, 0), (5, 1030, 1031, 1),
])
def test_quantize_is_the_definition(rows, cols, pitch, offset, square, pow2, fmt, dtype):
    x, _ = pitched(rows, cols, pitch, offset, dtype, NAN)
    x.copy_((randn(rows + cols, rows, cols) * torch.exp(3 * randn(7, rows, 1))).to(dtype))
    pair, = ns.f8_quantize([x], form="both", square=square, pow2=pow2, dtype=fmt)
    for (q, s), v in zip(pair, (x, x.T)):
        want_q, want_s = definition(v, fmt, pow2, square)
        assert q.dtype == fmt and s.dtype == (E8 if pow2 else FP32)
        assert torch.equal(s.float().double().cpu(), want_s)
        assert torch.equal(q.float().double().cpu(), want_q)
        for out in (BF16, FP32):
            back, = ns.f8_dequantize([(q, s)], dtype=out)
            assert torch.equal(back.cpu(), (want_q * spread(want_s, *v.shape)).float().to(out))
    for form, want in (("rows", pair[0]), ("transposed", pair[1])):
        got, = ns.f8_quantize([x], form=form, square=square, pow2=pow2, dtype=fmt)
        assert torch.equal(got.q.view(torch.uint8), want.q.view(torch.uint8))
        assert torch.equal(got.scale.float(), want.scale.float())


@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("pow2", [True, False])
def test_quantize_ties_and_extremes(pow2, fmt):
    """Quotients on and beside the borders between 8-bit floats, subnormal ones, blocks
    of zeros, of the least and the largest floats."""
    mant, least, top = SHAPE[fmt]
    grid = [m * 2.0 ** e for e in range(least - mant, 17) for m in range(2 ** mant, 2 ** (mant + 1)) if m * 2.0 ** e <= top]
    grid = sorted({g for g in grid} | {0.0} | {i * 2.0 ** (least - mant) for i in range(2 ** mant)})
    edge = torch.tensor([(a + b) / 2 for a, b in zip(grid, grid[1:])], dtype=torch.float64)
    near = torch.cat([edge, edge * (1 + 2.0 ** -23), edge * (1 - 2.0 ** -23), -edge])
    near = near[: near.numel() // 127 * 127].view(-1, 127)
    rows = []
    for scale in (1.0, 2.0 ** -40, 2.0 ** 100 / top * 448, 3.0, 1.7, 1.1e-37 / top, 7.3e35 / top):
        for part in near:
            rows.append(torch.cat([part, torch.tensor([top], dtype=torch.float64)]) * scale)
    line = torch.linspace(-1, 1, 128, dtype=torch.float64)
    rows += [torch.zeros(128, dtype=torch.float64), torch.full((128,), 5.5, dtype=torch.float64), line * 1e-42,
             line * 3.1e-36, line * 2.0 ** -119, line * 3.4028234e38, line * top, line * top / 64]
    x = torch.stack(rows).float().cuda()
    (q, s), = ns.f8_quantize([x], pow2=pow2, dtype=fmt)
    want_q, want_s = definition(x, fmt, pow2, False)
    assert torch.equal(s.float().double().cpu(), want_s)
    assert torch.equal(q.float().double().cpu(), want_q)


@pytest.mark.parametrize("pow2", [True, False])
def test_quantize_nan_and_inf_blocks(pow2):
    x = randn(1, 200, 300)
    x[1, 7], x[3, 299], x[140, 130] = NAN, float("inf"), -float("inf")
    pair, = ns.f8_quantize([x], form="both", pow2=pow2)
    for (q, s), v in zip(pair, (x, x.T)):
        wrong = ~torch.isfinite(v)
        r, c = wrong.nonzero(as_tuple=True)
        bad = torch.zeros((blocks(v.shape[1]), v.shape[0]), dtype=torch.bool, device="cuda")
        bad[c // 128, r] = True
        assert torch.equal(torch.isnan(s.float()), bad)
        back, = ns.f8_dequantize([(q, s)], dtype=FP32)
        each = bad.repeat_interleave(128, 0)[:v.shape[1]].T
        assert torch.equal(torch.isnan(back), each) and not bool(q.float()[each].any())
        want_q, want_s = definition(torch.where(each, torch.zeros_like(v), v), E4, pow2, False)
        assert torch.equal(back[~each].cpu(), (want_q * spread(want_s, *v.shape)).float()[~each.cpu()])


def test_quantize_writes_nothing_else():
    """Row gaps and the bytes around outputs stay as they were."""
    from newton_schulz_04_amd import _f8
    rows, cols = 130, 200
    x = randn(3, rows, cols)
    for pow2, kind in ((1, torch.uint8), (0, torch.int32)):
        q = torch.full((rows + 2, 240), 99, dtype=torch.uint8, device="cuda")
        qt = torch.full((cols + 2, 144), 99, dtype=torch.uint8, device="cuda")
        s = torch.full((2 + 2, 136), 77, dtype=kind, device="cuda")
        st = torch.full((2 + 2, 208), 77, dtype=kind, device="cuda")
        arr = _f8._int64s([rows, cols, x.data_ptr(), cols, q[1].data_ptr(), 240, s[1].data_ptr(), 136,
                           qt[1].data_ptr(), 144, st[1].data_ptr(), 208])
        rc = _f8.lib().ns_f8_quantize(arr, 1, 0, pow2, 0, 1, torch.cuda.current_stream().cuda_stream)
        assert rc == 0, ns.last_error()
        assert bool((q[[0, -1]] == 99).all()) and bool((q[:, cols:] == 99).all())
        assert bool((qt[[0, -1]] == 99).all()) and bool((qt[:, rows:] == 99).all())
        assert bool((s[[0, -1]] == 77).all()) and bool((s[:, rows:] == 77).all())
        assert bool((st[[0, -1]] == 77).all()) and bool((st[:, cols:] == 77).all())
        pair, = ns.f8_quantize([x], form="both", pow2=bool(pow2))
        assert torch.equal(q[1:-1, :cols], pair[0].q.view(torch.uint8))
        assert torch.equal(qt[1:-1, :rows], pair[1].q.view(torch.uint8))
        assert torch.equal(s[1:-1, :rows], pair[0].scale.view(kind)) and torch.equal(st[1:-1, :cols], pair[1].scale.view(kind))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cols", [*range(1, 18), *range(120, 138), 255, 259])
def test_row_ends(cols, dtype):
    """Rows of every length modulo the pieces they are read in, between NaNs, and matrices
    whose row gaps hold NaNs back to values."""
    rows = 9
    x, _ = pitched(rows, cols, cols + 3, 1, dtype, NAN)
    x.copy_(randn(cols, rows, cols).to(dtype))
    for square in (False, True):
        want_q, want_s = definition(x, E4, True, square)
        (q, s), t = ns.f8_quantize([x], form="both", square=square)[0]
        assert torch.equal(q.float().double().cpu(), want_q) and torch.equal(s.float().double().cpu(), want_s)
        turned_q, turned_s = definition(x.T, E4, True, square)
        assert torch.equal(t.q.float().double().cpu(), turned_q) and torch.equal(t.scale.float().double().cpu(), turned_s)
        gaps = torch.full((rows, -(-cols // 16) * 16), 0x7F, dtype=torch.uint8, device="cuda")
        gaps[:, :cols] = q.view(torch.uint8)
        for out in (BF16, FP32):
            back, = ns.f8_dequantize([(gaps.view(E4)[:, :cols], s)], dtype=out)
            assert torch.equal(back.cpu(), (want_q * spread(want_s, rows, cols)).float().to(out))


@pytest.mark.parametrize("form", ["rows", "transposed", "both"])
def test_lists_give_what_single_calls_give(form):
    """More matrices than a launch takes, of equal and of mixed shapes, some empty."""
    for shapes in ([(37, 50)] * 45, [(i % 7 * 30, i % 5 * 70) for i in range(90)]):
        xs = [randn(i, *s).bfloat16() for i, s in enumerate(shapes)]
        got = ns.f8_quantize(xs, form=form)
        assert len(got) == len(xs)
        for x, g in zip(xs, got):
            one, = ns.f8_quantize([x], form=form)
            for a, b in zip(g if form == "both" else [g], one if form == "both" else [one]):
                assert a.q.shape == b.q.shape and torch.equal(a.q.view(torch.uint8), b.q.view(torch.uint8))
                assert torch.equal(a.scale.float(), b.scale.float())
        flat = [p for g in got for p in (g if form == "both" else [g])]
        back = ns.f8_dequantize(flat, dtype=FP32)
        for p, b in zip(flat, back):
            assert torch.equal(b.double(), values(p))


# --- products ------------------------------------------------------------------
def operand(rows, cols, seed, fmt=E4, pow2=True, square=False, whole=False, gap=0):
    """An 8-bit matrix whose row gaps hold NaNs: random values of the format, or small
    whole numbers with scales of 1, 2 or 4."""
    g = gen(seed)
    pitch = -(-cols // 16) * 16 + gap or 16
    q = torch.full((rows, pitch), NAN, device="cuda").to(fmt)[:, :cols]
    nb, per = blocks(cols), blocks(rows) if square else rows
    lds = -(-per // 4) * 4 + 4
    if whole:
        v = torch.randint(-7, 8, (rows, cols), generator=g, device="cuda").float()
        if fmt == E5:   # (7 and 5 are not numbers of two mantissa bits... 5 and 7 are; 9 is not)
            v = v.clamp(-4, 4)
        e = torch.randint(0, 3, (nb, per), generator=g, device="cuda").float()
        sv = torch.exp2(e)
    else:
        v = (torch.randn((rows, cols), generator=g, device="cuda") * 100).clamp(-440, 440)
        sv = torch.exp2(torch.randint(-12, 12, (nb, per), generator=g, device="cuda").float())
        if not pow2:
            sv = sv * (1 + torch.rand((nb, per), generator=g, device="cuda"))
    q.copy_(v.to(fmt))
    s = torch.full((nb, lds), NAN, device="cuda").to(E8 if pow2 else FP32)[:, :per]
    s.copy_(sv.to(s.dtype))
    return ns.F8Blocks(q, s)


SIZES = [
    # m, n, k: the least, odd ones, tiles and their edges, several slots, split sums
    (1, 1, 1), (1, 5, 17), (2, 16, 128), (7, 33, 130), (16, 100, 257), (17, 40, 700), (32, 31, 1000),
    (33, 1, 5), (33, 130, 128), (100, 257, 129), (128, 256, 384), (129, 255, 385), (200, 300, 512), (130, 513, 640),
    (64, 70, 5000), (256, 512, 1024),
]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("out", [BF16, FP32])
def test_matmul_of_whole_numbers_is_exact(m, n, k, out):
    for i, (fmt, pow2, sqa, sqb) in enumerate([(E4, True, False, True), (E4, True, False, False), (E5, True, True, False),
                                               (E4, False, False, True), (E5, False, False, False), (E4, False, True, True)]):
        a = operand(m, k, 10 * i + 1, fmt, pow2, sqa, whole=True, gap=16 * (i % 2))
        b = operand(n, k, 10 * i + 2, E4, pow2 or i == 4, sqb, whole=True)   # (mixed scale types once)
        want = values(a) @ values(b).T
        assert float(want.abs().max()) < 2 ** 24
        got, = ns.f8_matmul([a], [b], dtype=out)
        assert torch.equal(got.double(), want.to(out).double()), (fmt, pow2, sqa, sqb)


def bound(a, b, ref, out, pow2):
    """Largest error of each output, from the header of this file."""
    va, vb = values(a).abs(), values(b).abs()
    (m, k), n = va.shape, vb.shape[0]
    mag = va @ vb.T
    err = (k + 40) * 2.0 ** -23 * mag
    if not pow2:
        err = err + 4 * 2.0 ** -24 * mag
    if out == BF16:
        pad = -k % 8
        va, vb = (torch.nn.functional.pad(v, (0, pad)) for v in (va, vb))
        top = torch.zeros_like(mag)
        for c in range(0, k + pad, 8):
            top += (va[:, None, c:c + 8] * vb[None, :, c:c + 8]).amax(2)
        err = err + 8 * 2.0 ** -13 * top
    return err + U[out] * (ref.abs() + err)


@pytest.mark.parametrize("m,n,k", [(1, 48, 300), (20, 33, 1029), (65, 70, 900), (129, 130, 385)])
@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("sqa,sqb", [(False, True), (False, False), (True, False)])
def test_matmul_against_64_bits(m, n, k, fmt, pow2, sqa, sqb):
    a, b = operand(m, k, 5, fmt, pow2, sqa), operand(n, k, 6, E4, pow2, sqb)
    ref = values(a) @ values(b).T
    for out in (BF16, FP32):
        got, = ns.f8_matmul([a], [b], dtype=out)
        assert got.dtype == out
        assert bool(((got.double() - ref).abs() <= bound(a, b, ref, out, pow2)).all()), out


@pytest.mark.parametrize("m,n,k", [(3, 20, 140), (40, 260, 300), (129, 515, 3000), (130, 300, 0), (5, 9, 0)])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_matmul_adds_to_its_output(m, n, k, out):
    """beta C, into a slice of a wider buffer, aligned or not, whose rest stays; with
    beta 0 nothing of C is read."""
    a, b = operand(m, k, 7, whole=True), operand(n, k, 8, square=True, whole=True)
    prod = values(a) @ values(b).T if k else torch.zeros((m, n), dtype=torch.float64, device="cuda")
    for off, width in ((0, n), (8, n + 24), (1, n + 3)):
        wide = torch.full((m, width), 3.0, dtype=out, device="cuda")
        c = wide[:, off:off + n]
        c.copy_(torch.randint(-64, 65, (m, n), generator=gen(9), device="cuda").to(out))
        want = (0.5 * c.double() + prod).to(out)
        version = c._version
        back, = ns.f8_matmul([a], [b], out=[c], beta=0.5)
        assert back is c and c._version > version
        assert torch.equal(c, want)
        c.fill_(NAN)
        ns.f8_matmul([a], [b], out=[c], beta=0.0)
        assert torch.equal(c.double(), prod.to(out).double())
        rest = torch.ones(width, dtype=torch.bool)
        rest[off:off + n] = False
        assert bool((wide[:, rest] == 3).all())


def test_matmul_of_lists():
    """Ragged counts, some without tokens, of both formats and scale types, more than a
    launch takes; any order. Whole numbers, whose sums are the same however they are cut."""
    sizes = [(0, 64, 300)] + [(1 + 17 * i % 190, 16 + 24 * (i % 5), 128 + 50 * (i % 9)) for i in range(60)] + [(9, 40, 0)]
    xs, wts = [], []
    for i, (m, n, k) in enumerate(sizes):
        xs.append(operand(m, k, i, E5 if i % 3 == 0 else E4, i % 4 != 1, whole=True))
        wts.append(operand(n, k, 1000 + i, E4, i % 4 != 2, square=i % 2 == 0, whole=True))
    for out in (BF16, FP32):
        every = ns.f8_matmul(xs, wts, dtype=out)
        back = ns.f8_matmul(xs[::-1], wts[::-1], dtype=out)[::-1]
        for i, (x, w) in enumerate(zip(xs, wts)):
            want = (values(x) @ values(w).T).to(out)
            assert torch.equal(every[i], want) and torch.equal(back[i], want), sizes[i]


@pytest.mark.parametrize("sizes", [
    [(4096, 2560, 300)], [(4100, 2564, 143)], [(2048, 2560, 64), (1000, 2560, 65), (1024, 2304, 200), (300, 300, 400)],
    [(4096, 2560, k) for k in (1, 16, 128, 256)], [(4096, 2570, 130)],
])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_matmul_of_large_tiles(sizes, out):
    """Enough tiles of 256 x 256 for the chip, whole and ragged, beside small products;
    sums of every length modulo the ring; added to an output."""
    for fmt, square, beta in ((E4, True, 0.0), (E5, False, 0.5)):
        xs = [operand(m, k, 3 * i, fmt, whole=True) for i, (m, n, k) in enumerate(sizes)]
        wts = [operand(n, k, 3 * i + 1, square=square, whole=True) for i, (m, n, k) in enumerate(sizes)]
        cs = [torch.randint(-64, 65, (m, n), generator=gen(i), device="cuda").to(out) for i, (m, n, k) in enumerate(sizes)]
        want = [(beta * c.double() + values(x) @ values(w).T).to(out) for c, x, w in zip(cs, xs, wts)]
        if beta == 0.0:
            for c in cs:
                c.fill_(NAN)
        ns.f8_matmul(xs, wts, out=cs, beta=beta)
        for c, w, size in zip(cs, want, sizes):
            assert torch.equal(c, w), (size, fmt)


def test_large_tiles_against_64_bits():
    a, b = operand(4096, 900, 5), operand(2560, 900, 6, square=True)
    for out in (BF16, FP32):
        got, = ns.f8_matmul([a], [b], dtype=out)
        some = torch.randint(0, 4096, (64,), generator=gen(2), device="cuda")
        part = ns.F8Blocks(a.q[some], a.scale[:, some])
        for c in range(0, 2560, 256):
            w = ns.F8Blocks(b.q[c:c + 256], b.scale[:, c // 128:c // 128 + 2])
            ref = values(part) @ values(w).T
            assert bool(((got[some, c:c + 256].double() - ref).abs() <= bound(part, w, ref, out, True)).all())


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("m", [5, 70])
def test_matmul_scales_at_the_ends_of_their_range(m, out):
    """Products whose scales alone would pass fp32's range, with results within it; NaN
    scales and NaN values make NaN of their row or column and of nothing else."""
    n, k = 40, 256
    for pow2 in (True, False):
        a, b = operand(m, k, 3, pow2=pow2, whole=True), operand(n, k, 4, pow2=pow2, whole=True)
        f = 1.0 if pow2 else 1.5
        a.scale.copy_(torch.full_like(a.scale.float(), f * 2.0 ** 100).to(a.scale.dtype))
        b.scale.copy_(torch.full_like(b.scale.float(), f * 2.0 ** -96).to(b.scale.dtype))
        got, = ns.f8_matmul([a], [b], dtype=out)
        assert torch.equal(got.double(), (values(a) @ values(b).T).to(out).double())
        a.scale[1, 2] = NAN
        b.q[3, 200] = NAN
        got, = ns.f8_matmul([a], [b], dtype=out)
        bad = torch.zeros_like(got, dtype=torch.bool)
        bad[2], bad[:, 3] = True, True
        assert torch.equal(torch.isnan(got), bad)


def test_matmul_on_another_stream_and_in_a_graph():
    a, b = operand(200, 3000, 1), operand(70, 3000, 2, square=True)
    few = operand(3, 3000, 5)
    x = randn(11, 200, 300).bfloat16()
    want = ns.f8_matmul([a, few], [b, b])
    want_q, = ns.f8_quantize([x], form="both")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ns.f8_matmul([a, few], [b, b], stream=side)
    side.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        out = ns.f8_matmul([a, few], [b, b])
    side.synchronize()
    with torch.cuda.graph(graph):
        out = ns.f8_matmul([a, few], [b, b])
        kept, = ns.f8_quantize([x], form="both")
    for step in range(3):
        for o in out:
            o.fill_(NAN)
        x.copy_(randn(11 + step, 200, 300).bfloat16())
        want_q, = ns.f8_quantize([x], form="both")
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(out, want))
        for k, w in zip(kept, want_q):
            assert torch.equal(k.q.view(torch.uint8), w.q.view(torch.uint8)) and torch.equal(k.scale.float(), w.scale.float())


def test_a_layer_of_the_calls():
    """Forward, the input's gradient and the weights' gradient of a layer from its
    quantised tensors, against the same products in 64 bits."""
    tokens, n, k = 300, 520, 400
    x, w, dy = randn(1, tokens, k).bfloat16(), randn(2, n, k) / 20, randn(3, tokens, n).bfloat16()
    (xq, xt), = ns.f8_quantize([x], form="both")
    (wq, wt), = ns.f8_quantize([w], form="both", square=True)
    (dq, dt), = ns.f8_quantize([dy], form="both", dtype=E5)
    assert torch.equal(values(wq), values(wt).T)
    g = torch.zeros((n, k), device="cuda")
    for got, a, b in ((ns.f8_matmul([xq], [wq])[0], xq, wq), (ns.f8_matmul([dq], [wt])[0], dq, wt),
                      (ns.f8_matmul([dt], [xt], out=[g], beta=1.0)[0], dt, xt)):
        ref = values(a) @ values(b).T
        assert bool(((got.double() - ref).abs() <= bound(a, b, ref, got.dtype, True)).all())
    ns.orthogonalize([g])
    assert bool(torch.isfinite(g).all())
