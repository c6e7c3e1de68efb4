"""The experts' router on the GPU against its formulas in 64 bits.

Bounds, derived (u = 2^-24): a logit less the row's largest is off by u times their
distance, its exponential by as much of itself and a few u of its own; the sum of E of
them by 32 u more (16 of a lane one after the other, then lanes in pairs). So p is off by
less than (2 R + 60) u of itself, R the row's range of logits. Weights: two or three
roundings and a sum of up to 16 more, (4 R + 160) u. Sums over T tokens: T u more. A
gradient p (g - sum g p) is off by (4 R + 200) u p (|g| + sum |g| p), g itself by (4 R +
200) u of the sum of magnitudes it is made of; then the output rounds. Choices and counts
are equal: they compare logits, which no rounding touches.
"""
import numpy
import pytest
import torch

import newton_schulz_04_amd as ns

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
EPS = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ns.lib()


def logits_of(tokens, experts, dtype, seed=0, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn((tokens, experts), generator=g)).to(dtype)


def definition(logits, top_k, normalize, mask=None):
    """All outputs in 64 bits, token by token."""
    x = logits.double().numpy()
    tokens, experts = x.shape
    chosen = numpy.full((tokens, top_k), -1)
    weights, probs = numpy.zeros((tokens, top_k)), numpy.zeros(experts)
    counts, n = numpy.zeros(experts, dtype=int), 0
    p = numpy.zeros((tokens, experts))
    for t in range(tokens):
        order = sorted((e for e in range(experts) if x[t, e] != -INF),
                       key=lambda e: (0 if numpy.isnan(x[t, e]) else 1, -x[t, e] if not numpy.isnan(x[t, e]) else 0, e))
        if not order or (mask is not None and not mask[t]):
            continue
        n += 1
        with numpy.errstate(invalid="ignore"):
            v = numpy.exp(x[t] - (NAN if numpy.isnan(x[t]).any() else x[t].max()))
            p[t] = v / v.sum()
        pick = order[:top_k]
        chosen[t, :len(pick)] = pick
        w = p[t, pick]
        weights[t, :len(pick)] = w / w.sum() if normalize else w
        counts[pick] += 1
        probs += p[t]
    loss = experts * float((counts / max(1, counts.sum()) * probs).sum()) / n if n else 0.0
    return dict(experts=chosen, weights=weights, counts=counts, probs=probs, tokens=n, loss=loss, p=p)


def span(logits):
    x = logits.double()
    live = torch.isfinite(x)
    if not bool(live.any()):
        return 0.0
    return float((torch.where(live, x, -INF).amax(1) - torch.where(live, x, INF).amin(1)).clamp_min(0).max())


def near(got, want, rel, what):
    got = got.double().cpu().numpy() if torch.is_tensor(got) else got
    bad = numpy.isnan(want)
    assert numpy.array_equal(numpy.isnan(got), bad), what
    off = numpy.abs(got - want)
    assert (off[~bad] <= rel * numpy.abs(want[~bad]) + 2.0 ** -120).all(), (what, off[~bad].max())


def check(logits, top_k, normalize, mask=None, **kw):
    want = definition(logits, top_k, normalize, mask)
    r = ns.route_experts(logits.cuda() if not logits.is_cuda else logits, top_k, normalize=normalize,
                         mask=None if mask is None else mask.cuda(), **kw)
    assert numpy.array_equal(r.experts.cpu().numpy(), want["experts"])
    assert numpy.array_equal(r.counts.cpu().numpy(), want["counts"]) and int(r.tokens) == want["tokens"]
    R, T = span(logits.cpu()), logits.shape[0]
    near(r.weights, want["weights"], (4 * R + 160) * EPS, "weights")
    near(r.probs, want["probs"], (2 * R + 60 + T) * EPS, "probs")
    near(r.loss.reshape(1), numpy.array([want["loss"]]), (2 * R + 100 + T + logits.shape[1]) * EPS, "loss")
    return r, want


SIZES = [(1, 1, 1), (1, 2, 1), (3, 16, 16), (8, 16, 2), (5, 17, 3), (65, 31, 4), (64, 64, 8), (257, 47, 3), (33, 100, 6),
         (130, 128, 8), (19, 200, 5), (500, 256, 8), (7, 257, 2), (40, 512, 8), (30, 700, 16), (9, 1024, 4)]


@pytest.mark.parametrize("tokens,experts,top_k", SIZES)
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_is_the_definition(tokens, experts, top_k, normalize, dtype):
    """bf16 logits tie often; also at odd pitches, and with padding."""
    x = logits_of(tokens, experts, dtype, seed=experts)
    check(x, top_k, normalize)
    wide = torch.full((tokens, experts + 3), 99.0, dtype=dtype).cuda()
    wide[:, 1:experts + 1] = x.cuda()
    view = wide[:, 1:experts + 1]
    mask = torch.arange(tokens) % 3 != 1
    r, want = check(x, top_k, normalize, mask)
    again = ns.route_experts(view, top_k, normalize=normalize, mask=mask.cuda())
    assert all(torch.equal(a, b) for a, b in zip(r, again))


def test_route_without_tokens():
    for tokens in (0, 5):
        r, _ = check(logits_of(tokens, 12, FP32), 2, True, torch.zeros(tokens, dtype=torch.bool))
        assert float(r.loss) == 0 and not bool(r.counts.any()) and not bool(r.probs.any())


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_route_ties_signs_and_masked_experts(dtype):
    low = torch.finfo(dtype).min
    rows = [
        [0.0] * 20,                                             # all alike
        [-0.0, 0.0] * 10,                                       # the zeros are
        [low] * 20,                                             # the type's lowest number is a number
        [low] * 10 + [1.0] + [low] * 9,
        [-INF] * 20,                                            # nothing to choose
        [-INF] * 19 + [3.0],                                    # less than top_k
        [-INF] * 7 + [2.0, 2.0] + [-INF] * 11,
        [1.0, 2.0] * 10,
        [torch.finfo(dtype).max] + [0.0] * 19,
        [80.0] + [-80.0] * 19,
    ]
    x = torch.tensor(rows).to(dtype)
    for normalize in (True, False):
        for top_k in (1, 3, 16):
            r, want = check(x, top_k, normalize)
            assert want["tokens"] == 9 and r.experts[4].tolist() == [-1] * top_k
            assert r.experts[0].tolist() == list(range(top_k)) == r.experts[1].tolist() == r.experts[2].tolist()


def test_route_nan_and_inf():
    x = logits_of(4, 24, FP32, seed=3)
    x[1, 5], x[2, 7] = NAN, INF
    r, want = check(x, 3, True)
    assert int(r.experts[1, 0]) == 5 and int(r.experts[2, 0]) == 7
    assert bool(torch.isnan(r.weights[1:3]).all()) and not bool(torch.isnan(r.weights[[0, 3]]).any())
    assert bool(torch.isnan(r.probs).all()) and bool(torch.isnan(r.loss))


@pytest.mark.parametrize("tokens,experts", [(20000, 8), (9000, 256), (3000, 600)])
def test_route_of_many_tokens_gives_the_same_bits_each_time(tokens, experts):
    x = logits_of(tokens, experts, FP32, seed=1).cuda()
    first = ns.route_experts(x, 4)
    want = torch.topk(x.cpu(), 4).indices.int()
    assert torch.equal(first.experts.cpu(), want)
    assert torch.equal(first.counts.cpu().long(), torch.bincount(want.flatten().long(), minlength=experts))
    p = torch.softmax(x.double(), 1).sum(0)
    assert bool(((first.probs.double() - p).abs() <= (2 * span(x.cpu()) + 60 + tokens) * EPS * p).all())
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, ns.route_experts(x, 4)))


# --- gradient --------------------------------------------------------------------
def objective(x, want, normalize, dw, dl):
    """What the gradient differentiates, in 64 bits: the choice and the counts held."""
    total, n = 0.0, want["tokens"]
    probs = numpy.zeros(x.shape[1])
    for t in range(x.shape[0]):
        if want["experts"][t, 0] < 0:
            continue
        v = numpy.exp(x[t] - x[t].max())
        p = v / v.sum()
        probs += p
        ok = want["experts"][t] >= 0
        w = p[want["experts"][t][ok]]
        w = w / w.sum() if normalize else w
        total += float((w * dw[t][ok]).sum())
    c = want["counts"]
    return total + dl * x.shape[1] * float((c / max(1, c.sum()) * probs).sum()) / max(1, n)


def formula(want, normalize, dw, dl):
    """(gradient, the magnitudes that it is made of) in 64 bits."""
    p, c, n = want["p"], want["counts"], max(1, want["tokens"])
    tokens, experts = p.shape
    out, mag = numpy.zeros_like(p), numpy.zeros_like(p)
    for t in range(tokens):
        if want["experts"][t, 0] < 0:
            continue
        g = dl * experts / n * c / max(1, c.sum())
        a = numpy.abs(g)
        ok = want["experts"][t] >= 0
        pick, h, ha = want["experts"][t][ok], dw[t][ok], numpy.abs(dw[t][ok])
        if normalize:
            s = p[t, pick].sum()
            w = p[t, pick] / s
            h, ha = (h - (h * w).sum()) / s, (ha + (ha * w).sum()) / s
        g, a = g.copy(), a.copy()
        g[pick] += h
        a[pick] += ha
        out[t] = p[t] * (g - (g * p[t]).sum())
        mag[t] = p[t] * (a + (a * p[t]).sum())
    return out, mag


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (2, 3, 1), (5, 16, 2), (17, 30, 3), (33, 64, 8), (9, 100, 5),
                                                  (40, 256, 8), (6, 300, 3), (3, 1024, 16)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("parts", ["both", "weights", "loss"])
def test_gradient(tokens, experts, top_k, normalize, dtype, parts):
    x = logits_of(tokens, experts, dtype, seed=experts + tokens)
    if experts > 4:
        x[0, 1] = -INF
    mask = torch.arange(tokens) % 4 != 2
    want = definition(x, top_k, normalize, mask)
    g = torch.Generator().manual_seed(5)
    dw = torch.randn((tokens, top_k), generator=g) if parts != "loss" else None
    dl = torch.tensor(7.5) if parts != "weights" else None
    dwn, dln = (torch.zeros((tokens, top_k)) if dw is None else dw).double().numpy(), 0.0 if dl is None else 7.5
    ref, mag = formula(want, normalize, dwn, dln)
    r = ns.route_experts(x.cuda(), top_k, normalize=normalize, mask=mask.cuda())
    got = ns.route_experts_grad(x.cuda(), r.experts, r.counts, r.tokens, dweights=None if dw is None else dw.cuda(),
                                dloss=None if dl is None else dl.cuda(), normalize=normalize)
    assert got.dtype == dtype
    err = (4 * span(x) + 200) * 2 * EPS * mag
    off = numpy.abs(got.double().cpu().numpy() - ref)
    assert (off <= err + HALF[dtype] * (numpy.abs(ref) + err) + 2.0 ** -120).all()
    # against differences of the 64-bit objective, along random directions
    xd = x.double().numpy()
    rng = numpy.random.default_rng(1)
    for _ in range(3):
        d = numpy.where(numpy.isfinite(xd), rng.standard_normal(xd.shape), 0.0)
        h = 1e-5
        num = (objective(xd + h * d, want, normalize, dwn, dln) - objective(xd - h * d, want, normalize, dwn, dln)) / (2 * h)
        # (central differences: h^2 times third derivatives, and rounding 2^-52 / h)
        assert abs(num - float((ref * d).sum())) <= 1e-8 * (1 + float((mag * numpy.abs(d)).sum()))


def test_gradient_into_a_slice_and_of_odd_choices():
    """out at a pitch, its surroundings as they were; the same expert twice adds up; indexes
    outside the experts have no weight; a token whose first is -1 has no gradient."""
    x = logits_of(6, 20, FP32, seed=2).cuda()
    r = ns.route_experts(x, 3, normalize=False)
    chosen = r.experts.clone()
    chosen[1] = torch.tensor([4, 4, 7])
    chosen[2] = torch.tensor([3, 20, 5000])
    chosen[3, 0] = -1
    dw = torch.randn((6, 3), generator=torch.Generator().manual_seed(1)).cuda()
    wide = torch.full((6, 27), 5.0, device="cuda")
    out = wide[:, 3:23]
    back = ns.route_experts_grad(x, chosen, r.counts, r.tokens, dweights=dw, normalize=False, out=out)
    assert back is out and bool((wide[:, :3] == 5).all()) and bool((wide[:, 23:] == 5).all())
    p = torch.softmax(x.double(), 1)
    for t in range(6):
        g = torch.zeros(20, dtype=torch.float64, device="cuda")
        for i in range(3):
            if 0 <= int(chosen[t, i]) < 20 and t != 3:
                g[int(chosen[t, i])] += dw[t, i].double()
        want = p[t] * (g - (g * p[t]).sum())
        assert bool(((out[t].double() - want).abs() <= 400 * EPS * (p[t] * (g.abs() + (g.abs() * p[t]).sum())) + 1e-30).all())


def test_gradient_of_summed_counts():
    """Counts of several ranks: shares of all of them."""
    x = logits_of(30, 12, FP32, seed=4)
    r = ns.route_experts(x.cuda(), 2)
    more = r.counts + torch.arange(12, dtype=torch.int32, device="cuda")
    got = ns.route_experts_grad(x.cuda(), r.experts, more, r.tokens, dloss=torch.tensor(1.0).cuda())
    want = dict(definition(x, 2, True), counts=more.cpu().numpy())
    ref, mag = formula(want, True, numpy.zeros((30, 2)), 1.0)
    assert (numpy.abs(got.double().cpu().numpy() - ref) <= (4 * span(x) + 200) * 2 * EPS * mag + EPS * numpy.abs(ref)).all()


def test_on_another_stream_and_in_a_graph():
    x = logits_of(3000, 96, BF16, seed=6).cuda()
    dl = torch.tensor(0.5).cuda()
    want = ns.route_experts(x, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ns.route_experts(x, 4, stream=side)
    grad = ns.route_experts_grad(x, got.experts, got.counts, got.tokens, dloss=dl, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = ns.route_experts(x, 4)
        g = ns.route_experts_grad(x, r.experts, r.counts, r.tokens, dloss=dl)
    for step in range(3):
        for t in (*r, g):
            t.fill_(77)
        x.copy_(logits_of(3000, 96, BF16, seed=6 + step).cuda())
        want = ns.route_experts(x, 4)
        grad = ns.route_experts_grad(x, want.experts, want.counts, want.tokens, dloss=dl)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, r)) and torch.equal(g, grad)


def test_a_run_of_the_experts():
    """A layer of experts: route, quantise, the experts' products by their counts, and the
    way back, against autograd in 64 bits on the dequantised operands."""
    tokens, dim, hidden, experts, top_k = 150, 256, 144, 6, 2
    gen = torch.Generator().manual_seed(0)
    x = torch.randn((tokens, dim), generator=gen).bfloat16().cuda()
    w = [torch.randn((hidden, dim), generator=gen).cuda() / 16 for _ in range(experts)]
    logits = (2 * torch.randn((tokens, experts), generator=gen)).cuda()
    dy = torch.randn((tokens, hidden), generator=gen).bfloat16().cuda()
    r = ns.route_experts(logits, top_k)
    slots = torch.argsort(r.experts.flatten(), stable=True)
    cut = r.counts.tolist()
    rows = [i // top_k for i in slots.split(cut)]
    xs = [x[i] for i in rows]
    xq = ns.f8_quantize(xs, form="both")
    wq = ns.f8_quantize(w, form="both", square=True)
    ys = ns.f8_matmul([a for a, _ in xq], [a for a, _ in wq], dtype=FP32)
    flat = r.weights.flatten()[slots].split(cut)
    y = torch.zeros((tokens, hidden), device="cuda")
    for i, f, part in zip(rows, flat, ys):
        y.index_add_(0, i, part * f[:, None])
    # back: the weights' gradient, the products', the router's
    dyw = [dy[i].float() for i in rows]
    dweights = torch.zeros(tokens * top_k, device="cuda")
    dweights[slots] = torch.cat([(a * b).sum(1) for a, b in zip(dyw, ys)])
    dlogits = ns.route_experts_grad(logits, r.experts, r.counts, r.tokens, dweights=dweights.view(tokens, top_k),
                                    dloss=torch.tensor(0.1).cuda())
    dq = ns.f8_quantize([a * f[:, None] for a, f in zip(dyw, flat)], form="both")
    dx = ns.f8_matmul([a for a, _ in dq], [b for _, b in wq], dtype=FP32)
    dw = ns.f8_matmul([b for _, b in dq], [b for _, b in xq], dtype=FP32)
    # the same in 64 bits
    val = lambda q: ns.f8_dequantize([q], dtype=FP32)[0].double()   # noqa: E731
    l64 = logits.double().requires_grad_()
    p = torch.softmax(l64, 1)
    g = p.gather(1, r.experts.long())
    g = (g / g.sum(1, keepdim=True)).flatten()[slots].split(cut)
    total = 0.0
    for i, gi, (a, _), (b, _) in zip(rows, g, xq, wq):
        total = total + ((val(a) @ val(b).T) * gi[:, None] * dy[i].double()).sum()
    c = r.counts.double()
    total = total + 0.1 * experts * (c / c.sum() * p.sum(0)).sum() / tokens
    total.backward()
    assert float((dlogits.double() - l64.grad).norm() / l64.grad.norm()) < 1e-4
    for a, (q, _), (_, t) in zip(dx, dq, wq):
        want = val(q) @ val(t).T
        assert float((a.double() - want).norm()) <= 1e-5 * float(want.norm())
    for a, (_, q), (_, t) in zip(dw, dq, xq):
        want = val(q) @ val(t).T
        assert float((a.double() - want).norm()) <= 1e-5 * float(want.norm())
    ns.orthogonalize(dw)
    assert all(bool(torch.isfinite(v).all()) for v in dw)
