"""Autograd does not see these calls: an input that waits for a gradient is refused, instead of a
result without one."""
import pytest
import torch

import bit_gathered_quantized_amd as bgq

CALLS = {
    "x of grouped_matmul": lambda t: bgq.grouped_matmul(t, t.detach()),
    "w of grouped_matmul": lambda t: bgq.grouped_matmul(t.detach(), t),
    "dy of grouped_matmul_dw": lambda t: bgq.grouped_matmul_dw(t, t.detach()),
    "x of grouped_matmul_dw": lambda t: bgq.grouped_matmul_dw(t.detach(), t),
    "x of mx_quantize": lambda t: bgq.mx_quantize(t),
}


@pytest.mark.parametrize("call", CALLS.values(), ids=list(CALLS))
def test_inputs_that_wait_for_a_gradient(call):
    leaf = torch.zeros(8, 64, dtype=torch.bfloat16).requires_grad_()
    for t in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="gradient"):
            call(t)
        for quiet in (torch.no_grad, torch.inference_mode):
            with quiet(), pytest.raises(ValueError, match="CUDA"):  # past that check: it wants GPU tensors
                call(t)
    with pytest.raises(ValueError, match="CUDA"):
        call(leaf.detach())


@pytest.mark.gpu
def test_an_autograd_function_around_the_products():
    """Inside a Function's forward and backward grad mode is off, so the calls are taken, and its gradients are
    those of the formula."""
    from grouped_util import F64, check, gradient, offsets_of, product

    class Experts(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, offsets):
            ctx.save_for_backward(x, w, offsets)
            return bgq.grouped_matmul(x, w, offsets)

        @staticmethod
        def backward(ctx, dy):
            x, w, offsets = ctx.saved_tensors
            return bgq.grouped_matmul(dy, w, offsets, transpose=True), bgq.grouped_matmul_dw(dy, x, offsets), None

    g = torch.Generator(device="cuda").manual_seed(0)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    offsets = offsets_of([5, 0, 20])
    x, w, dy = normal(25, 64).requires_grad_(), normal(3, 40, 64).requires_grad_(), normal(25, 40)
    y = Experts.apply(x, w, offsets)
    y.backward(dy)
    check(y.detach(), *product(x.detach(), w.detach(), offsets), 64)
    check(x.grad, *product(dy, w.detach().transpose(1, 2), offsets), 40)
    check(w.grad, *gradient(dy, x.detach(), offsets), 20)
    with pytest.raises(ValueError, match="gradient"):
        bgq.grouped_matmul(x, w, offsets)
    with torch.no_grad():
        assert torch.equal(bgq.grouped_matmul(x, w, offsets), y)
