"""Lists of several large layers, which share launches of 256 x 256 tiles, the
last round of them in halves, against single calls and the formulas; and large
tiles whose operands come late."""
import pytest
import torch

import newton_schulz_04_amd as ns
from test_gpu_q8 import BF16, FP32, check, gen, grad_bound, grads_in, layout, matmul_bound, product_of, q8_matrix, wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ns.lib()


# rows and columns of the outputs, and their sums' length: 100 + 80 + 64 + 50 + 40
# large tiles, of which each layer alone has too few to take them; the fourth
# layer's first 12 are whole tiles, its others and the fifth's run as halves
# (tests/sanitize/q8_limits.cpp holds the planner to that)
LAYERS = [(2560, 2560, 1600), (2040, 2550, 2101), (2048, 2048, 1537), (1270, 2555, 3000), (2048, 1280, 1555)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("kind", ["contiguous", "padded"])
def test_matmul_list(kind, dtype):
    g = gen(61)
    xs = [q8_matrix(m, k, g, pitch=layout(k, kind, 1)[0], full=True) for m, _, k in LAYERS]
    ws = [q8_matrix(n, k, g, pitch=layout(k, kind, 1)[0], full=True) for _, n, k in LAYERS]
    ys = ns.q8_matmul(xs, ws, dtype=dtype)
    for x, w, y in zip(xs, ws, ys):
        assert torch.equal(y, ns.q8_matmul([x], [w], dtype=dtype)[0])
        ref = product_of(x, w)
        check(y, ref, matmul_bound(ref, dtype))


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("kind", ["contiguous", "padded"])
def test_grad_input_list(kind, pow2):
    g = gen(62)
    dys = [grads_in(m, o, g, pitch=layout(o, kind, 2)[0]) for m, _, o in LAYERS]
    ws = [q8_matrix(o, n, g, pow2=pow2, pitch=layout(n, kind, 1)[0]) for _, n, o in LAYERS]
    dxs = ns.q8_grad_input(dys, ws)
    for dy, w, dx in zip(dys, ws, dxs):
        assert torch.equal(dx, ns.q8_grad_input([dy], [w])[0])
        ref, mags = dy.double() @ wide(w), dy.double().abs() @ wide(w).abs()
        check(dx, ref, grad_bound(ref, mags, dy.shape[1], BF16, pow2))


@pytest.mark.parametrize("dtype,beta", [(BF16, 0.0), (BF16, 0.9375), (FP32, 1.0)])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("kind", ["contiguous", "padded"])
def test_grad_weight_list(kind, pow2, dtype, beta):
    g = gen(63)
    dys = [grads_in(t, m, g, pitch=layout(m, kind, 2)[0]) for m, _, t in LAYERS]
    xs = [q8_matrix(t, n, g, pow2=pow2, pitch=layout(n, kind, 1)[0]) for _, n, t in LAYERS]
    start = [torch.randn((m, n), generator=g, device="cuda").to(dtype) for m, n, _ in LAYERS]
    grads = ns.q8_grad_weight(dys, xs, [s.clone() for s in start], beta=beta)
    for dy, x, s, gw in zip(dys, xs, start, grads):
        assert torch.equal(gw, ns.q8_grad_weight([dy], [x], [s.clone()], beta=beta)[0])
        dt = dy.double().T.contiguous()
        ref, mags = beta * s.double() + dt @ wide(x), beta * s.double().abs() + dt.abs() @ wide(x).abs()
        check(gw, ref, grad_bound(ref, mags, dy.shape[0], dtype, pow2))


@pytest.mark.parametrize("slots", [24, 25, 26, 27, 48, 49, 50, 51])
@pytest.mark.parametrize("pow2", [False, True])
def test_large_tiles_give_the_same_bits_from_slow_memory(slots, pow2):
    """300 large tiles, 44 of them as halves, and 516 small ones of matmul,
    while a copy on another stream keeps the memory busy: for sums of each
    length modulo the rings."""
    g = gen(slots)
    busy, side = torch.empty(1 << 29, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    m, n, k8, k16 = 5120, 3840, 64 * slots - 7, 32 * slots - 7
    p8, p16 = -(-k8 // 16) * 16, -(-k16 // 8) * 8
    x, w = q8_matrix(m, k8, g, pitch=p8), q8_matrix(n, k8, g, pitch=p8)
    xs, wn = q8_matrix(33000, k8, g, pitch=p8), q8_matrix(129, k8, g, pitch=p8)
    dy, wi = grads_in(m, k16, g, pitch=p16), q8_matrix(k16, n, g, pow2=pow2)
    dt, xw = grads_in(k16, m, g), q8_matrix(k16, n, g, pow2=pow2)

    def run():
        outs = [*ns.q8_matmul([x], [w]), *ns.q8_matmul([xs], [wn]), *ns.q8_grad_input([dy], [wi])]
        for dtype, beta in ((BF16, 0.0), (FP32, 0.0), (FP32, 0.5)):
            outs += ns.q8_grad_weight([dt], [xw], [torch.ones((m, n), dtype=dtype, device="cuda")], beta=beta)
        return outs

    first = run()
    torch.cuda.synchronize()
    for a, b, y in ((x, w, first[0]), (xs, wn, first[1])):
        check(y, product_of(a, b), matmul_bound(product_of(a, b), BF16))
    d, v = dt.double().T.contiguous(), wide(xw)
    check(first[4], d @ v, grad_bound(d @ v, d.abs() @ v.abs(), k16, FP32, pow2))
    for _ in range(3):
        with torch.cuda.stream(side):
            for _ in range(4):
                busy.add_(1)
        again = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
