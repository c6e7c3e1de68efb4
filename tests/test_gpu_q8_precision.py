"""The gradients' precision with scales that are no powers of two: the 8-bit
operand enters the products with (almost) all bits of q s, so that the results
are as exact as their type lets them be.

Bounds, derived (half a step: bf16 2^-8, fp32 2^-24): a term dy q s is off by
  - the rounding of q s to fp32, 2^-24 of it, and
  - what its parts leave out. bf16 outputs: q s = t0 + t1, t0 its leading 8
    bits, so that the rest is below 2^-7 of it, t1 the rest rounded to bf16:
    2^-7 2^-8. fp32 outputs: three parts of 8 bits hold all 24.
  - 2^-46, twice what the parts carry so that none is zero beside a q s that
    is not: 2^-48 of q s in each.
Products of bf16 values are exact in fp32. Parts have the sign of q s, so their
magnitudes add up to its own: a sum of K terms in P parts is off by at most
(P K + 40) 2^-23 of the sum of magnitudes (a whole step for each addition; the
join of pieces and beta G are among the 40). Then the output's rounding.
Tokens (channels) of dY that are zero add exact zeros: with eight of them left
in a long sum the bound stays far below the rounding of q s to bf16.
"""
import pytest
import torch

import newton_schulz_04_amd as ns
from test_gpu_q8 import BF16, FP32, U, check, gen, grads_in, layout, pitched, q8_matrix, wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ns.lib()


def bound(ref, mags, terms, dtype):
    parts = 2 if dtype == BF16 else 3
    ux = 2.0 ** -24 + 2.0 ** -46 + (2.0 ** -15 if dtype == BF16 else 0.0)
    inner = mags * (ux + (parts * terms + 40) * 2.0 ** -23)
    return inner + (ref.abs() + inner) * U[dtype] + 1e-35


def few_along(dy, axis, g):
    """Leaves eight tokens (axis 0) or channels (axis 1) of dy, the last one
    among them; the number left."""
    n = dy.shape[axis]
    keep = torch.randperm(n, generator=g, device="cuda")[:8]
    keep[0] = n - 1
    mask = torch.zeros(n, dtype=torch.bool, device="cuda")
    mask[keep] = True
    dy.mul_(mask[:, None] if axis == 0 else mask)
    return int(mask.sum())


# few rows; few tiles, whole and in pieces; many tiles; large tiles, the last
# of them in halves
SIZES = [(1, 1, 1), (5, 3, 7), (33, 257, 520), (300, 770, 1536), (1000, 18, 2304), (2500, 24, 100), (4096, 64, 640),
         (70, 2048, 6144), (640, 512, 544), (2048, 200, 260), (2100, 2064, 2208), (3330, 3333, 3341)]


@pytest.mark.parametrize("dtype,beta", [(BF16, 0.0), (BF16, 0.9375), (FP32, 0.0), (FP32, 1.0)])
@pytest.mark.parametrize("kind", ["contiguous", "odd"])
@pytest.mark.parametrize("t,o,k", SIZES)
def test_grad_weight_keeps_the_operands_bits(t, o, k, kind, dtype, beta):
    g = gen(t + 31 * o + 97 * k)
    px, ox = layout(k, kind, 1)
    x, dy = q8_matrix(t, k, g, pitch=px, offset=ox), grads_in(t, o, g, *layout(o, kind, 2))
    terms = few_along(dy, 0, g)
    out = torch.randn((o, k), generator=g, device="cuda").to(dtype)
    before = out.double()
    ns.q8_grad_weight([dy], [x], [out], beta=beta)
    dt = dy.double().T.contiguous()
    ref, mags = beta * before + dt @ wide(x), beta * before.abs() + dt.abs() @ wide(x).abs()
    check(out, ref, bound(ref, mags, terms, dtype))


@pytest.mark.parametrize("kind", ["contiguous", "odd"])
@pytest.mark.parametrize("t,o,k", SIZES)
def test_grad_input_keeps_the_operands_bits(t, o, k, kind):
    g = gen(t + 31 * o + 101 * k)
    pw, ow = layout(k, kind, 1)
    w, dy = q8_matrix(o, k, g, pitch=pw, offset=ow), grads_in(t, o, g, *layout(o, kind, 2))
    terms = few_along(dy, 1, g)
    dx, = ns.q8_grad_input([dy], [w])
    ref, mags = dy.double() @ wide(w), dy.double().abs() @ wide(w).abs()
    check(dx, ref, bound(ref, mags, terms, BF16))


@pytest.mark.parametrize("t,o,k", [(2048, 200, 260), (1000, 18, 2304), (640, 512, 544), (2100, 2064, 2208)])
def test_one_scale_among_powers_of_two(t, o, k):
    """The last token's scale alone is no power of two, or the first's."""
    for at in (t - 1, 0):
        g = gen(t + at)
        x, dy = q8_matrix(t, k, g, pow2=True), grads_in(t, o, g)
        terms = few_along(dy, 0, g)
        dy[at] = torch.randn(o, generator=g, device="cuda").to(BF16)
        x[1][at] = 0.7371
        out = torch.empty((o, k), device="cuda")
        ns.q8_grad_weight([dy], [x], [out])
        dt = dy.double().T.contiguous()
        ref, mags = dt @ wide(x), dt.abs() @ wide(x).abs()
        check(out, ref, bound(ref, mags, terms + 1, FP32))


def test_norms_of_the_errors():
    """Dense operands: an output's error against 64 bits is its own rounding.
    Half a step at most is 2^-8 of a bf16 value; over values spread through a
    binade, steps of 2^-7 to 2^-8 of them, the root mean square is at most
    2^-8 / sqrt(3) = 2.26e-3 where all lie at its lower end, and the operand
    adds less than 2^-15: 2.4e-3 holds it in any case, 1.9e-3 where values lie
    evenly within their binades (at most 2^-8 / 2 / sqrt(3) (1 / ln 2)^(1/2) *
    1.41 = 1.92e-3). fp32: 4096 terms whose partial sums round at random, three
    parts: sqrt(3 4096) 2^-24 = 6.6e-6 of the magnitudes at most."""
    g = gen(3)
    t, o, k = 4096, 512, 768
    x, dy = q8_matrix(t, k, g), grads_in(t, o, g)
    dt = dy.double().T.contiguous()
    ref = dt @ wide(x)
    for dtype, most in ((BF16, 1.92e-3), (FP32, 6.6e-6)):
        out = torch.empty((o, k), dtype=dtype, device="cuda")
        ns.q8_grad_weight([dy], [x], [out])
        err = float((out.double() - ref).norm() / ref.norm())
        assert err <= most, err
    w = q8_matrix(o, k, g)
    dx, = ns.q8_grad_input([dy], [w])
    ref = dy.double() @ wide(w)
    assert float((dx.double() - ref).norm() / ref.norm()) <= 1.92e-3


@pytest.mark.parametrize("t,o,k", [(40, 70, 96), (300, 513, 520), (1000, 18, 2304), (2100, 2064, 2208)])
def test_infinities_stay_infinities(t, o, k):
    """An Inf of dY gives Inf of q's sign wherever q is not zero, NaN where it
    is (Inf 0), whatever bits of q s the parts of the operand hold: scales with
    few bits and with many in one sum."""
    g = gen(t + o + k)
    x, w = q8_matrix(t, k, g), q8_matrix(o, k, g)
    for q, s in (x, w):
        s[::2] = torch.exp2(torch.randint(-9, -3, (s[::2].numel(),), generator=g, device="cuda").float())
    for at in (0, 1, t - 1):
        dy = grads_in(t, o, g)
        dy[at, o // 2] = float("inf")
        gw, = ns.q8_grad_weight([dy], [x], [torch.zeros((o, k), device="cuda")])
        want = x[0][at].float() * float("inf")
        assert torch.equal(gw[o // 2].isnan(), want.isnan()) and torch.equal(gw[o // 2].nan_to_num(0, 1, -1),
                                                                             want.nan_to_num(0, 1, -1))
        dx, = ns.q8_grad_input([dy], [w])
        want = w[0][o // 2].float() * float("inf")
        got = dx[at].float()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0, 1, -1),
                                                                      want.nan_to_num(0, 1, -1))


@pytest.mark.parametrize("t,o,k", [(33, 257, 520), (640, 512, 544), (1000, 18, 2304), (2100, 2064, 2208)])
def test_the_smallest_scales(t, o, k):
    """Scales down to 2^-126, the quantiser's least: parts below bf16's normal
    numbers are rounded to its smallest one, 2^-133, half of it at most away
    from q s each, or cut there (twice that): 2^-132 in all three."""
    g = gen(t + o + k + 1)
    x, dy = q8_matrix(t, k, g), grads_in(t, o, g)
    x[1].copy_(torch.exp2(-126 + 20 * torch.rand(t, generator=g, device="cuda")))
    dy.mul_(2.0 ** 100)
    terms = few_along(dy, 0, g)
    dt = dy.double().T.contiguous()
    ref, mags = dt @ wide(x), dt.abs() @ wide(x).abs()
    lost = dt.abs().sum(1, keepdim=True) * 2.0 ** -132
    for dtype in (BF16, FP32):
        out = torch.empty((o, k), dtype=dtype, device="cuda")
        ns.q8_grad_weight([dy], [x], [out])
        check(out, ref, bound(ref, mags, terms, dtype) + lost * (1 + U[dtype]))
