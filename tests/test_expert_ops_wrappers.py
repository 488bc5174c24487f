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


BIG = 2 ** 32 + 4    # its low 32 bits are 4


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


def index(n):
    return meta(n, dtype=torch.int32)


@pytest.mark.parametrize("call", [
    lambda: moe.grouped_gemm(meta(BIG, 32), meta(2, 16, 32), index(3)),
    lambda: moe.grouped_gemm(meta(4, 32), meta(2, BIG, 32), index(3)),
    lambda: moe.grouped_gemm_dgrad(meta(BIG, 16), meta(2, 16, 32), index(3)),
    lambda: moe.grouped_gemm_wgrad(meta(BIG, 16), meta(BIG, 32), index(3)),
    lambda: moe.grouped_gemm_wgrad(meta(4, 16), meta(4, 32), index(BIG)),
    lambda: moe.quant_int8(meta(BIG, 32)),
    lambda: moe.quant_int8(meta(4, 32), perm=index(BIG), k=2),
    lambda: moe.quant_int8(meta(4, 32), perm=index(8), k=2 ** 32 + 2),
    lambda: moe.int8_gemm(meta(BIG, 32, dtype=torch.int8), meta(BIG), meta(16, 32, dtype=torch.int8), meta(16)),
    lambda: moe.permute(meta(BIG, 32), index(8), 2),
    lambda: moe.permute(meta(4, 32), index(BIG), 2),
    lambda: moe.permute(meta(4, 32), index(8), 2 - 2 ** 32),
    lambda: moe.combine(meta(BIG, 32), index(8), k=2),
    lambda: moe.combine(meta(8, 32), index(2 * BIG), k=2),
    lambda: moe.combine(meta(8, 32), index(0), k=2 ** 32 + 2),
    lambda: moe.combine_backward(meta(BIG, 32), meta(8, 32), index(2 * BIG), meta(BIG, 2)),
])
def test_sizes_past_32_bits_are_refused(call):
    """ctypes passes the low 32 bits of a size: such a call would work on the first few rows without a word."""
    with pytest.raises(moe.MoeError) as e:
        call()
    assert e.value.status == moe.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("k,n_shared", [(0, 0), (0, 1), (-1, 1), (2, -2), (2, -1)])
def test_slots_that_no_token_has_are_refused(k, n_shared):
    """The number of tokens is that of the slots by k + n_shared."""
    with pytest.raises(ValueError, match="k is"):
        moe.combine(rows(), PERM, k=k, n_shared=n_shared)


class OnAnotherGpu:
    """Ids [2, 2] as route() sees a tensor of cuda:1."""
    shape, device, dtype, is_cuda = torch.Size((2, 2)), torch.device("cuda", 1), torch.int32, True

    def numel(self):
        return 4

    def is_contiguous(self):
        return True

    def get_device(self):
        return 1

    def data_ptr(self):
        raise AssertionError("reached the library")


def test_route_refuses_ids_of_another_gpu():
    """The context's workspace lies on its own GPU."""
    layer = object.__new__(moe.MoeLayer)
    layer.E, layer.k, layer.n_shared, layer.device, layer.ctx = 4, 2, 0, 0, None
    with pytest.raises(ValueError, match="topk_ids is on cuda:1, not on cuda:0"):
        layer.route(OnAnotherGpu())
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        layer.route(torch.zeros(2, 2, dtype=torch.int32))
