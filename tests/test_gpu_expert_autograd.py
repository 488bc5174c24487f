"""GPU tests of the expert operators' wrappers where autograd is on: values as
without it, and a backward pass that raises instead of leaving a gradient out."""
import pytest
import torch

from fp4_block_scaled_route_b200 import moe

pytestmark = pytest.mark.gpu


def test_results_are_the_same_and_their_backward_pass_raises():
    gen = torch.Generator("cuda").manual_seed(1)
    x, dy = (torch.randn(40, n, generator=gen, device="cuda").bfloat16() for n in (72, 136))
    w = torch.randn(3, 136, 72, generator=gen, device="cuda").bfloat16()
    off = torch.tensor([0, 10, 10, 40], dtype=torch.int32, device="cuda")
    inv = torch.randperm(40, generator=gen, device="cuda").int()
    g = torch.rand(20, 2, generator=gen, device="cuda")

    def calls():
        return (moe.grouped_gemm(x, w, off), moe.grouped_gemm_dgrad(dy, w, off), moe.grouped_gemm_wgrad(dy, x, off),
                moe.permute(x, inv, 1), moe.combine(x, inv, g), moe.combine_backward(x[:20], x, inv, g)[0])
    plain = calls()
    for t in (x, dy, w, g):
        t.requires_grad_()
    for a, b in zip(plain, calls()):
        assert torch.equal(a, b) and b.requires_grad
        with pytest.raises(NotImplementedError, match="no autograd formula"):
            b.float().sum().backward()
    with torch.no_grad():
        for a, b in zip(plain, calls()):
            assert torch.equal(a, b) and not b.requires_grad


def test_an_own_autograd_function_of_the_calls():
    """A caller's Function around the calls sees none of this: its forward and backward run without recording."""
    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, off):
            ctx.save_for_backward(x, w, off)
            return moe.grouped_gemm(x, w, off, out_dtype=torch.float32)

        @staticmethod
        def backward(ctx, dy):
            x, w, off = ctx.saved_tensors
            dy = dy.to(x.dtype)
            return moe.grouped_gemm_dgrad(dy, w, off), moe.grouped_gemm_wgrad(dy, x, off), None

    gen = torch.Generator("cuda").manual_seed(2)
    x, c = (torch.randn(50, n, generator=gen, device="cuda").bfloat16() for n in (104, 72))
    w = torch.randn(4, 72, 104, generator=gen, device="cuda").bfloat16()
    off = torch.tensor([0, 0, 7, 49, 50], dtype=torch.int32, device="cuda")
    x.requires_grad_(), w.requires_grad_()
    (Product.apply(x, w, off) * c.float()).sum().backward()
    x64, w64 = (t.detach().double().requires_grad_() for t in (x, w))
    o = off.tolist()
    sum(((x64[a:b] @ w64[e].T) * c[a:b].double()).sum() for e, (a, b) in enumerate(zip(o, o[1:]))).backward()
    for got, ref in ((x.grad, x64.grad), (w.grad, w64.grad)):
        # rounded once to bf16 (half a step, 2^-8 of the value); the fp32 sums of up to 104 products add far less
        assert float((got.double() - ref).norm()) <= 2.0 ** -8 * float(ref.norm())
