"""A token's outputs and its gradient are its own: equal to the bit whatever stands beside
it."""
import pytest
import torch

import newton_schulz_04_amd as ns

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


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
