"""The 8-bit floating-point calls and the router as programs use them: on two streams
at once, in several captured graphs, on views, in place, past 32 bits of offset, and
with infinities. What is compared is equal to the bit, but for the differences:

A central difference of step h of a sum S of weights and loss is off from the derivative
by at most h^2 / 6 max |S'''| and by the error of the two values of S over 2 h. In one
logit each softmax is a logistic function, whose third derivative is at most 1 / 8, so
|S'''| <= (largest - smallest coefficient) / 8; a value of S is off by (4 R + 160) 2^-24
of the sum of magnitudes of its terms, R the row's range of logits.
"""
import pytest
import torch

import newton_schulz_04_amd as ns

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ns.lib()


def randn(seed, *shape, dtype=FP32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def whole(seed, *shape):
    """Whole numbers, which 8-bit floats hold with any power-of-two scale near them, and
    whose products and sums are exact."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-7, 8, shape, generator=g, device="cuda", dtype=torch.int8).to(BF16)


def bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


def same(a, b):
    if isinstance(a, torch.Tensor):
        return a.shape == b.shape and a.dtype == b.dtype and torch.equal(bits(a), bits(b))
    return len(a) == len(b) and all(same(x, y) for x, y in zip(a, b))


class Work:
    """A router's and a layer's calls, with split sums, few tokens and a workspace for
    the router."""

    def __init__(self, seed):
        self.x, self.few = randn(seed, 200, 2500, dtype=BF16), randn(seed + 1, 5, 2500, dtype=BF16)
        self.w, self.logits = randn(seed + 2, 140, 2500), randn(seed + 3, 5000, 60)

    def run(self, stream=None):
        kw = dict(stream=stream)
        q = ns.f8_quantize([self.x, self.few], form="both", **kw)
        w, = ns.f8_quantize([self.w], square=True, **kw)
        y = ns.f8_matmul([q[0][0], q[1][0]], [w, w], **kw)
        back = ns.f8_dequantize([q[0][1]], **kw)
        r = ns.route_experts(self.logits, 4, **kw)
        g = ns.route_experts_grad(self.logits, r.experts, r.counts, r.tokens, dweights=r.weights, dloss=r.loss, **kw)
        return q, w, y, back, r, g


def test_two_streams_at_once():
    work = [Work(10), Work(20)]
    want = [w.run() for w in work]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[w.run(s) for w, s in zip(work, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for round_ in got:
        assert all(same(a, b) for a, b in zip(round_, want))


@pytest.mark.parametrize("shared", [False, True])
def test_two_graphs(shared):
    """Two captured graphs: of memory pools of their own, replayed at once on two streams;
    of one pool, replayed in turn."""
    work = [Work(30), Work(40)]
    for w in work:
        w.run()
    graphs, out = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for i, (w, g) in enumerate(zip(work, graphs)):
        with torch.cuda.graph(g, pool=graphs[0].pool() if shared and i else None):
            out.append(w.run())
    side = torch.cuda.current_stream() if shared else torch.cuda.Stream()
    for step in range(3):
        for i, w in enumerate(work):
            w.x.copy_(randn(50 + 2 * step + i, 200, 2500))
            w.logits.copy_(randn(60 + 2 * step + i, 5000, 60))
        want = [w.run() for w in work]
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(out, want)), step


@pytest.mark.parametrize("pow2", [True, False])
def test_views_of_matrices(pow2):
    """Rows and blocks of columns of a larger 8-bit matrix, as tensors of their own."""
    x, w = whole(1, 300, 700), whole(2, 280, 700)
    (q, t), = ns.f8_quantize([x], form="both", pow2=pow2, dtype=E5 if pow2 else E4)
    for square in (False, True):
        (wq,) = ns.f8_quantize([w], square=square, pow2=pow2)
        full, = ns.f8_matmul([q], [wq], dtype=FP32)
        for a, b in ((0, 300), (16, 17), (100, 140), (128, 300)):
            for c, d in ((0, 700), (128, 256), (256, 700), (384, 500)):
                part = ns.F8Blocks(q.q[a:b, c:d], q.scale[c // 128:-(-d // 128), a:b])
                other = ns.F8Blocks(wq.q[128:, c:d], wq.scale[c // 128:-(-d // 128), 1 if square else 128:])
                if square and pow2:
                    # one-byte scales begin at a multiple of 4, as their pitch is one
                    with pytest.raises(ns.NSError, match="not aligned to 4 bytes"):
                        ns.f8_matmul([part], [other], dtype=FP32)
                    s = torch.empty((other.scale.shape[0], 4), dtype=other.scale.dtype, device="cuda")[:, :2]
                    s.copy_(other.scale)
                    other = other._replace(scale=s)
                got, = ns.f8_matmul([part], [other], dtype=FP32)
                va, = ns.f8_dequantize([part], dtype=FP32)
                assert torch.equal(va, ns.f8_dequantize([q], dtype=FP32)[0][a:b, c:d])
                vb, = ns.f8_dequantize([other], dtype=FP32)
                ref = va.double() @ vb.double().T
                if pow2:
                    assert torch.equal(got.double(), ref)
                    if (c, d) == (0, 700):
                        assert torch.equal(got, full[a:b, 128:])
                else:
                    # (scales of m / 448: a block's whole-number sum times two factors, and
                    # 6 sums of blocks: at most 12 roundings of 2^-24 of the magnitudes)
                    mag = va.double().abs() @ vb.double().abs().T
                    assert bool(((got.double() - ref).abs() <= (d - c + 40) * 2.0 ** -23 * mag).all())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("experts", [8, 200, 700])
def test_gradient_in_place_of_the_logits(dtype, experts):
    for pitch in (experts, experts + 5):
        x = randn(3, 3000, pitch, dtype=dtype)[:, :experts]
        r = ns.route_experts(x, 3)
        kw = dict(dweights=randn(4, 3000, 3), dloss=torch.tensor(2.0, device="cuda"))
        want = ns.route_experts_grad(x, r.experts, r.counts, r.tokens, **kw)
        got = ns.route_experts_grad(x, r.experts, r.counts, r.tokens, out=x, **kw)
        assert got is x and torch.equal(got, want)


@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(normalize):
    """Logits a good step apart, so that no difference changes the choice."""
    tokens, experts, k, h, u = 6, 20, 3, 2.0 ** -6, 2.0 ** -24
    g = torch.Generator().manual_seed(5)
    x = torch.stack([torch.randperm(experts, generator=g) for _ in range(tokens)]).float() / 4
    dw, dl = torch.randn((tokens, k), generator=g), 3.0

    def total(v):
        r = ns.route_experts(v.cuda(), k, normalize=normalize)
        terms = torch.cat([(r.weights.double().cpu() * dw.double()).flatten(), dl * r.loss.double().cpu().reshape(1)])
        return float(terms.sum()), float(terms.abs().sum()), r

    _, _, r = total(x)
    got = ns.route_experts_grad(x.cuda(), r.experts, r.counts, r.tokens, dweights=dw.cuda(),
                                dloss=torch.tensor(dl).cuda(), normalize=normalize).double().cpu()
    share = dl * experts / tokens * float((r.counts / r.counts.sum()).max())
    third = (2 * float(dw.abs().max()) + share) / 8
    for t in range(tokens):
        for e in range(experts):
            up, down = x.clone(), x.clone()
            up[t, e] += h
            down[t, e] -= h
            (a, mag, _), (b, _, _) = total(up), total(down)
            err = (4 * experts / 4 + 160) * u * 1.1 * mag
            assert abs((a - b) / (2 * h) - float(got[t, e])) <= err / h + h * h / 6 * third, (t, e)


@pytest.mark.parametrize("m", [3, 60, 600])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_infinite_values_and_scales(m, out):
    """Infinities among A's values (which only e5m2 has) give what the formula gives; a
    scale of Inf gives NaN, as one of NaN does, in its own row alone."""
    k, n = 300, 300
    (a,), (b,) = ns.f8_quantize([whole(1, m, k)], dtype=E5), ns.f8_quantize([whole(2, n, k)])
    a.q[1, 7], a.q[2, 290] = INF, -INF
    va, vb = (ns.f8_dequantize([v], dtype=FP32)[0].double().cpu() for v in (a, b))
    assert bool(torch.isinf(va[1, 7]))
    want = (va @ vb.T).to(out).cuda()
    got, = ns.f8_matmul([a], [b], dtype=out)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, 5.0, 1e9, -1e9), torch.nan_to_num(want, 5.0, 1e9, -1e9))
    (a,), (b,) = (ns.f8_quantize([whole(i, r, k)], pow2=False) for i, r in ((1, m), (2, n)))
    a.scale[1, 2] = INF
    got, = ns.f8_matmul([a], [b], dtype=out)
    rows = torch.isnan(got)
    assert bool(rows[2].all()) and not bool(rows[:2].any()) and not bool(rows[3:].any())


def test_offsets_past_32_bits():
    rows, cols, n = 1_100_000, 2048, 128
    x = whole(1, rows, cols)
    at = rows // 128 * 128 - 256
    (q, t), = ns.f8_quantize([x], form="both")
    assert q.q.numel() > 2 ** 31
    (tail, tail_t), = ns.f8_quantize([x[at:]], form="both")
    assert same(q.q[at:], tail.q) and same(q.scale[:, at:].contiguous(), tail.scale.contiguous())
    assert same(t.q[:, at:], tail_t.q) and same(t.scale[at // 128:].contiguous(), tail_t.scale.contiguous())
    back, = ns.f8_dequantize([q])
    assert torch.equal(back[at:], x[at:]) and torch.equal(back[:at], x[:at])
    del back
    back, = ns.f8_dequantize([t])
    assert torch.equal(back[-3:], x[:, -3:].T)
    del back
    w, = ns.f8_quantize([whole(2, n, cols)], square=True)
    wide = torch.full((rows, cols), 3.0, dtype=BF16, device="cuda")
    ns.f8_matmul([q], [w], out=[wide[:, 100:100 + n]])
    part, = ns.f8_matmul([tail], [w])
    assert torch.equal(wide[at:, 100:100 + n], part) and bool((wide[at:, 100 + n:] == 3).all())
    del wide
    # a sum over all of them, the weights' gradient: whole numbers below 2^24
    dy = whole(3, rows, n)
    (dt,) = ns.f8_quantize([dy], form="transposed")
    got, = ns.f8_matmul([dt], [t], dtype=FP32)
    want = sum(dy[i:i + 100000].double().T @ x[i:i + 100000].double() for i in range(0, rows, 100000))
    assert torch.equal(got.double(), want)


def test_most_tokens():
    tokens, experts, k = 2 ** 24, 130, 4
    x = torch.empty((tokens, 136), dtype=BF16, device="cuda").normal_()[:, :experts]
    assert tokens * 136 > 2 ** 31
    r = ns.route_experts(x, k)
    at = tokens - 1000
    tail = ns.route_experts(x[at:], k)
    assert same(r.experts[at:], tail.experts) and same(r.weights[at:], tail.weights)
    assert int(r.tokens) == tokens and int(r.counts.sum()) == tokens * k
    assert torch.equal(r.counts.long(), torch.bincount(r.experts.flatten(), minlength=experts))
    kw = dict(dloss=torch.tensor(1e6, device="cuda"))
    g = ns.route_experts_grad(x, r.experts, r.counts, r.tokens, dweights=r.weights, **kw)
    part = ns.route_experts_grad(x[at:], r.experts[at:], r.counts, r.tokens, dweights=r.weights[at:], **kw)
    assert torch.equal(g[at:], part)
    assert bool((part != 0).any())
