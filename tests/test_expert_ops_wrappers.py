"""CPU tests of what the torch wrappers of the expert operators refuse before
they reach the library."""
import pytest
import torch

from fp4_block_scaled_route_b200 import moe


def rows(n=4, cols=32):
    return torch.zeros(n, cols)


W, OFF, PERM = torch.zeros(2, 16, 32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)


@pytest.mark.parametrize("call,name", [
    (lambda: moe.grouped_gemm(rows(), W, None), "offsets"),
    (lambda: moe.grouped_gemm_dgrad(rows(cols=16), W, None), "offsets"),
    (lambda: moe.grouped_gemm_wgrad(rows(cols=16), rows(), None), "offsets"),
    (lambda: moe.permute(rows(), None, 2), "perm"),
    (lambda: moe.combine(rows(), None, k=2), "inv"),
    (lambda: moe.combine(rows(), None, torch.zeros(2, 2)), "inv"),
    (lambda: moe.combine_backward(rows(), rows(), None, torch.zeros(2, 2)), "inv"),
    (lambda: moe.combine_backward(rows(), rows(), PERM, None), "topk_w"),
], ids=["product", "input_gradient", "weight_gradient", "permute", "combine_unweighted", "combine", "combine_gradient",
        "combine_gradient_weights"])
def test_a_missing_argument_is_named(call, name):
    with pytest.raises(ValueError, match=f"{name} is None"):
        call()
