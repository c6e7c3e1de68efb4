"""A token's outputs and its gradient are its own: equal to the bit whatever stands beside
it, and what the documentation says for every index of a route."""
import pytest
import torch

import newton_schulz_04_amd as ns

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
EPS = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ns.lib()


def logits_of(tokens, experts, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (2 * torch.randn((tokens, experts), generator=g)).to(dtype).cuda()


NEIGHBOURS = {
    "nan": lambda x: x.index_fill_(1, torch.tensor([3], device="cuda"), NAN),
    "ties": lambda x: x.fill_(1.0),
    "none": lambda x: x.fill_(-INF),
    "one": lambda x: x.fill_(-INF).index_fill_(1, torch.tensor([1], device="cuda"), 2.0),
    "others": lambda x: x.copy_(x.flip(1)),
}


@pytest.mark.parametrize("kind", list(NEIGHBOURS))
@pytest.mark.parametrize("experts,top_k", [(16, 2), (40, 5), (64, 8), (100, 6), (256, 8), (256, 16), (700, 8)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_token_does_not_depend_on_its_neighbours(experts, top_k, dtype, kind):
    """One token of each four stays as it is while the others turn into what an order of
    its own, or none, is found for; the same token by itself; masked neighbours."""
    x = logits_of(400, experts, dtype, seed=experts)
    want = ns.route_experts(x, top_k)
    mine = torch.arange(0, 400, 4, device="cuda") + torch.arange(100, device="cuda") % 4
    rest = torch.ones(400, dtype=torch.bool, device="cuda")
    rest[mine] = False
    y = x.clone()
    y[rest] = NEIGHBOURS[kind](x[rest].clone())
    for got in (ns.route_experts(y, top_k), ns.route_experts(y, top_k, mask=~rest)):
        assert torch.equal(got.experts[mine], want.experts[mine])
        assert torch.equal(got.weights[mine], want.weights[mine])
    for t in mine[:6].tolist():
        one = ns.route_experts(x[t:t + 1], top_k)
        assert torch.equal(one.experts[0], want.experts[t]) and torch.equal(one.weights[0], want.weights[t])
    dw = torch.randn((400, top_k), generator=torch.Generator().manual_seed(1)).cuda()
    kw = dict(counts=want.counts, tokens=want.tokens, dloss=torch.tensor(3.0, device="cuda"), dweights=dw)
    grad = ns.route_experts_grad(x, want.experts, **kw)
    other = ns.route_experts_grad(y, want.experts, **kw)
    assert torch.equal(other[mine], grad[mine])


@pytest.mark.parametrize("experts", [20, 300])
@pytest.mark.parametrize("normalize", [True, False])
def test_a_first_index_outside_the_experts_has_no_weight_but_the_loss(experts, normalize):
    """Of the chosen indexes only a first one of -1 takes a token out: others outside the
    experts have no weight of their own, wherever they stand, and if all are."""
    x = logits_of(6, experts, FP32, seed=2)
    r = ns.route_experts(x, 3, normalize=normalize)
    chosen = r.experts.clone()
    chosen[1, 0], chosen[2, 0], chosen[3, 0] = experts, 2 ** 31 - 1, -1
    chosen[4], chosen[5, 0] = torch.tensor([-7, experts, -1]), -2
    dw = torch.randn((6, 3), generator=torch.Generator().manual_seed(1)).cuda()
    got = ns.route_experts_grad(x, chosen, r.counts, r.tokens, dweights=dw, dloss=torch.tensor(7.0, device="cuda"),
                                normalize=normalize)
    p = torch.softmax(x.double(), 1)
    c = r.counts.double()
    for t in range(6):
        g = 7.0 * experts / 6 * c / c.sum()
        a = g.clone()
        ok = [i for i in range(3) if 0 <= int(chosen[t, i]) < experts]
        e = chosen[t, ok].long()
        h, size = dw[t, ok].double(), dw[t, ok].double().abs()
        if normalize:
            w = p[t, e] / p[t, e].sum()
            h, size = (h - (h * w).sum()) / p[t, e].sum(), (size + (size * w).sum()) / p[t, e].sum()
        g[e] += h
        a[e] += size
        want = p[t] * (g - (g * p[t]).sum()) * (t != 3)
        # ((4 R + 200) roundings of p and of g, R at most 20, and the output's)
        assert bool(((got[t].double() - want).abs() <= (2 * 280 + 1) * EPS * p[t] * (a + (a * p[t]).sum())).all()), t


@pytest.mark.parametrize("tokens,experts,top_k", [(2 ** 20 + 3, 1024, 16), (70001, 600, 7), (100, 300, 4), (5, 1024, 16)])
def test_the_loss_of_its_sums(tokens, experts, top_k):
    """The loss from the call's own counts and sums of p, in 64 bits, more than 2^24 choices
    among them. Bound: the counts' sum is exact until it becomes a float (1 rounding); the
    sum of c P has at most 4 terms a thread, 6 exchanges and 7 wavefronts' parts to add (17);
    two divisions and a product (3): 21 of 2^-24."""
    g = torch.Generator(device="cuda").manual_seed(experts)
    # (experts of unlike popularity)
    x = torch.randn((tokens, experts), generator=g, device="cuda", dtype=BF16)
    x += 2 * torch.randn(experts, generator=g, device="cuda", dtype=BF16)
    r = ns.route_experts(x, top_k)
    c, p = r.counts.double(), r.probs.double()
    assert int(r.tokens) == tokens and float(c.sum()) == tokens * top_k
    want = experts * float((c / c.sum() * p).sum()) / tokens
    assert abs(float(r.loss) - want) <= 21 * EPS * want
