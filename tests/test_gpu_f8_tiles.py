"""Every kind of tile of the 8-bit floating-point products on the GPU, at the shapes of
f8_tile_cases.py, which test_f8_kinds.py follows to their kernels.

Bounds, derived (u = half a step: bf16 2^-8, fp32 2^-24):
  whole numbers  products of whole numbers below 8, scales 1, 2 or 4: every product and sum
             is a whole number below 2^24 (asserted), and those of a group of eight k lie
             within 13 bits of one another's magnitude (7 * 7 * 16 < 2^10), so that only the
             output rounds: equality
  others     as in test_gpu_f8.py: bf16 outputs 8 2^-13 max |p| for each group of eight k,
             sums K 2^-23 of the sum of magnitudes, fp32 scales 4 2^-24 of it more, and the
             output's rounding
"""
import pytest
import torch

import newton_schulz_04_amd as ns
from f8_tile_cases import CASES, PLACED, name_of

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
E4, E5, E8 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
U = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}
DTYPES = {"bf16": BF16, "fp32": FP32}
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ns.lib()


def blocks(n):
    return -(-n // 128)


def operand(rows, cols, seed, fmt, fp32_scales, square, whole):
    """An 8-bit matrix between NaNs: whole numbers with scales of 1, 2 or 4, or values of
    the whole range with scales of 2^-12 .. 2^12, fp32 ones no powers of two."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.full((rows, -(-cols // 16) * 16), NAN, device="cuda").to(fmt)[:, :cols]
    nb, per = blocks(cols), blocks(rows) if square else rows
    if whole:
        v = torch.randint(-4 if fmt == E5 else -7, 5 if fmt == E5 else 8, (rows, cols), generator=g, device="cuda").float()
        sv = torch.exp2(torch.randint(0, 3, (nb, per), generator=g, device="cuda").float())
    else:
        v = (torch.randn((rows, cols), generator=g, device="cuda") * 100).clamp(-440, 440)
        sv = torch.exp2(torch.randint(-12, 13, (nb, per), generator=g, device="cuda").float())
        if fp32_scales:
            sv = sv * (1 + torch.rand((nb, per), generator=g, device="cuda"))
    q.copy_(v.to(fmt))
    s = torch.full((nb, -(-per // 4) * 4 + 4), NAN, device="cuda").to(FP32 if fp32_scales else E8)[:, :per]
    s.copy_(sv.to(s.dtype))
    return ns.F8Blocks(q, s)


def values(pair):
    """In 64 bits. (One-byte scales from their bits: the device's pow is not exact.)"""
    q, s = pair
    if s.dtype == E8:
        b = s.contiguous().view(torch.uint8).long()
        s = torch.where(b == 255, NAN, ((b + 1023 - 127) << 52).view(torch.float64))
    s = s.double().repeat_interleave(128, 0)[:q.shape[1]].T
    return q.float().double() * (s if s.shape[0] == q.shape[0] else s.repeat_interleave(128, 0)[:q.shape[0]])


def operands(products, fmt, whole, seed):
    a = [operand(m, k, seed + 2 * i, fmt, any_, False, whole) for i, (m, n, k, any_, sq, _) in enumerate(products)]
    b = [operand(n, k, seed + 2 * i + 1, E4, any_, sq, whole) for i, (m, n, k, any_, sq, _) in enumerate(products)]
    return a, b


@pytest.mark.parametrize("case", CASES, ids=name_of)
@pytest.mark.parametrize("fmt", [E4, E5], ids=["e4m3", "e5m2"])
def test_whole_numbers_are_exact(case, fmt):
    """Without an addend, whose NaNs are not read, and with half of one."""
    _, dtype, products = case
    out = DTYPES[dtype]
    a, b = operands(products, fmt, True, 10)
    exact = [values(x) @ values(w).T.contiguous() for x, w in zip(a, b)]
    assert all(float(e.abs().max()) < 2 ** 24 for e in exact)
    got = [torch.full(e.shape, NAN, dtype=out, device="cuda") for e in exact]
    ns.f8_matmul(a, b, out=got)
    for p, g, e in zip(products, got, exact):
        assert torch.equal(g, e.to(out)), p
    g = torch.Generator(device="cuda").manual_seed(3)
    got = [torch.randint(-64, 65, e.shape, generator=g, device="cuda").to(out) for e in exact]
    want = [(0.5 * c.double() + e).to(out) for c, e in zip(got, exact)]
    ns.f8_matmul(a, b, out=got, beta=0.5)
    for p, g, w in zip(products, got, want):
        assert torch.equal(g, w), p


@pytest.mark.parametrize("case", CASES, ids=name_of)
@pytest.mark.parametrize("fmt", [E4, E5], ids=["e4m3", "e5m2"])
def test_against_64_bits(case, fmt):
    """Some of the rows, the first and the last ones among them, by all columns."""
    _, dtype, products = case
    out = DTYPES[dtype]
    a, b = operands(products, fmt, False, 20)
    got = ns.f8_matmul(a, b, dtype=out)
    g = torch.Generator(device="cuda").manual_seed(4)
    for (m, n, k, any_, _, _), x, w, y in zip(products, a, b, got):
        rows = torch.unique(torch.cat([torch.randint(0, m, (12,), generator=g, device="cuda"),
                                       torch.tensor([0, m - 1], device="cuda")]))
        va = values(x)[rows]
        vb = values(w)
        ref = va @ vb.T.contiguous()
        va, vb = va.abs(), vb.abs()
        mag = va @ vb.T.contiguous()
        err = (k + 40 + (2 if any_ else 0)) * 2.0 ** -23 * mag
        if out == BF16:
            for c in range(0, k, 8):
                err += 8 * 2.0 ** -13 * (va[:, None, c:c + 8] * vb[None, :, c:c + 8]).amax(2)
        assert bool(((y[rows].double() - ref).abs() <= err + U[out] * (ref.abs() + err)).all()), (m, n, k)


@pytest.mark.parametrize("case", CASES, ids=name_of)
def test_nan_stays_in_its_row_or_column(case):
    """NaN scales of A's last row and B's first, a NaN in the last value of a row of each."""
    _, dtype, products = case
    a, b = operands(products, E4, True, 30)
    for x, w in zip(a, b):
        x.scale[-1, -1] = NAN
        x.q[1, -1] = NAN
        w.scale[0, 0] = NAN
        w.q[-1, -1] = NAN
    for (m, n, k, any_, square, _), y in zip(products, ns.f8_matmul(a, b, dtype=DTYPES[dtype])):
        bad = torch.zeros((m, n), dtype=torch.bool, device="cuda")
        bad[[1, m - 1]] = True
        bad[:, :128 if square else 1] = True
        bad[:, -1] = True
        assert torch.equal(torch.isnan(y), bad), (m, n, k)


@pytest.mark.parametrize("case", CASES, ids=name_of)
def test_the_same_call_gives_the_same_bits_around_its_output(case):
    """Into slices of wider buffers, whose rest stays, again and again."""
    _, dtype, products = case
    a, b = operands(products, E4, False, 40)
    wide = [torch.full((m + 2, n + 12), 3.0, dtype=DTYPES[dtype], device="cuda") for m, n, *_ in products]
    out = [w[1:-1, 8:-4] for w in wide]
    first = None
    for _ in range(3):
        for o in out:
            o.fill_(NAN)
        ns.f8_matmul(a, b, out=out)
        if first is None:
            first = [o.clone() for o in out]
        for w, o, f in zip(wide, out, first):
            assert torch.equal(o, f)
            assert all(bool((v == 3).all()) for v in (w[0], w[-1], w[:, :8], w[:, -4:]))


@pytest.mark.parametrize("m,n,k,dtype", PLACED)
def test_the_bits_do_not_depend_on_where_the_output_lies(m, n, k, dtype):
    (a,), (b,) = operands([(m, n, k, False, True, "big")], E4, False, 50)
    want, = ns.f8_matmul([a], [b], dtype=DTYPES[dtype])
    for offset, pitch in ((1, n), (0, n + 1), (2, n + 2)):
        room = torch.full((m * pitch + 8,), 3.0, dtype=DTYPES[dtype], device="cuda")
        out = room[offset:offset + m * pitch].view(m, pitch)[:, :n]
        ns.f8_matmul([a], [b], out=[out])
        assert torch.equal(out, want)
        assert bool((room[:offset] == 3).all()) and bool((room[offset + m * pitch:] == 3).all())
        assert bool((room[offset:offset + m * pitch].view(m, pitch)[:, n:] == 3).all())
