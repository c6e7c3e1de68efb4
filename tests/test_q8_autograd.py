"""The 8-bit calls among autograd's: tensors that require grad are refused in
grad mode, and what a call writes to counts as changed in place."""
import pytest
import torch

import newton_schulz_04_amd as ns
from newton_schulz_04_amd import _q8

FP32, BF16 = torch.float32, torch.bfloat16


def test_tensors_that_require_grad_are_refused_in_grad_mode():
    """(Before any device is looked at.)"""
    x = torch.ones((3, 4), requires_grad=True)
    cuda = torch.device("cuda", 0)
    with pytest.raises(ValueError, match="requires grad.*no_grad"):
        _q8._matrix(x, "every matrix", FP32, cuda)
    # not without grad mode: then the device is what is wrong with it
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        _q8._matrix(x, "every matrix", FP32, cuda)


class Layer(torch.autograd.Function):
    """A linear layer written from the calls."""

    @staticmethod
    def forward(ctx, x, weight):
        xq, wq = ns.quantize_rows([x], pow2=True), ns.quantize_rows([weight], pow2=True)
        ctx.save_for_backward(*xq[0], *wq[0])
        return ns.q8_matmul(xq, wq, dtype=FP32)[0]

    @staticmethod
    def backward(ctx, dy):
        xq, xs, wq, ws = ctx.saved_tensors
        dy = [dy.to(BF16)]
        dx, = ns.q8_grad_input(dy, [(wq, ws)])
        dw, = ns.q8_grad_weight(dy, [(xq, xs)], [torch.empty(wq.shape, dtype=FP32, device=wq.device)])
        return dx.to(FP32), dw


@pytest.mark.gpu
def test_a_layer_of_the_calls():
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((33, 40), generator=g, device="cuda").requires_grad_()
    w = torch.randn((24, 40), generator=g, device="cuda").requires_grad_()
    seed = torch.randn((33, 24), generator=g, device="cuda").to(BF16).float()
    (Layer.apply(x, w) * seed).sum().backward()
    with torch.no_grad():
        (wq, ws), (xq, xs) = *ns.quantize_rows([w], pow2=True), *ns.quantize_rows([x], pow2=True)
    wide_w, wide_x = wq.double() * ws.double()[:, None], xq.double() * xs.double()[:, None]
    d = seed.double()
    # sums of exact products in fp32 (24 or 33 terms and 40 for tile edges), then the output
    dx, dw = d @ wide_w, d.T.contiguous() @ wide_x
    assert bool(((x.grad.double() - dx).abs() <= dx.abs() * 2.0 ** -8 + (d.abs() @ wide_w.abs()) * 64 * 2.0 ** -23).all())
    assert bool(((w.grad.double() - dw).abs() <= (d.abs().T.contiguous() @ wide_x.abs()) * 74 * 2.0 ** -23).all())


@pytest.mark.gpu
def test_refusals_on_the_gpu():
    x = torch.ones((3, 4), device="cuda", requires_grad=True)
    q, s = torch.zeros((3, 4), dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda")
    grad_s = torch.ones(3, device="cuda", requires_grad=True)
    dy = torch.ones((3, 5), dtype=BF16, device="cuda")
    out = torch.ones((5, 4), device="cuda", requires_grad=True)
    for call in (lambda: ns.quantize_rows([x]), lambda: ns.dequantize_rows([(q, grad_s)]),
                 lambda: ns.q8_matmul([(q, grad_s)], [(q, s)]), lambda: ns.q8_matmul([(q, s)], [(q, grad_s)]),
                 lambda: ns.q8_matmul([(q, s)], [(q, s)], dtype=FP32,
                                      out=[torch.ones((3, 3), device="cuda", requires_grad=True)]),
                 lambda: ns.q8_grad_input([dy[:, :3].clone().requires_grad_()], [(q, s)]),
                 lambda: ns.q8_grad_weight([dy.clone().requires_grad_()], [(q, s)], [out.detach()]),
                 lambda: ns.q8_grad_weight([dy], [(q, s)], [out])):
        with pytest.raises(ValueError, match="requires grad"):
            call()
        with torch.no_grad():
            call()


@pytest.mark.gpu
def test_writes_are_changes_in_place():
    """A tensor that a backward pass still needs cannot change unnoticed."""
    q, s = torch.ones((3, 4), dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda")
    dy = torch.ones((3, 5), dtype=BF16, device="cuda")
    a = torch.ones((), device="cuda", requires_grad=True)
    for make, write in (((5, 4), lambda t: ns.q8_grad_weight([dy], [(q, s)], [t], beta=1.0)),
                        ((3, 3), lambda t: ns.q8_matmul([(q, s)], [(q, s)], dtype=FP32, out=[t])),
                        ((3, 4), lambda t: ns.q8_grad_input([dy[:, :3].contiguous()], [(q, s)], out=[t]))):
        t = torch.ones(make, dtype=BF16 if make == (3, 4) else FP32, device="cuda")
        loss = (a * t).sum()
        write(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        version = t._version
        write(t)
        assert t._version == version + 1
