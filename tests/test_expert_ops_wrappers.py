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


# ---- autograd ---------------------------------------------------------------------
def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


# name -> (call of (inputs, results), shapes of the inputs that may record a gradient, shapes of the results)
BF16, INT8 = torch.bfloat16, torch.int8
CALLS = {
    "grouped_gemm": (lambda i, o: moe.grouped_gemm(i[0], i[1], OFF, out=o[0]), [(4, 32), (2, 16, 32)], [(4, 16)], BF16),
    "grouped_gemm_dgrad": (lambda i, o: moe.grouped_gemm_dgrad(i[0], i[1], OFF, out=o[0]), [(4, 16), (2, 16, 32)], [(4, 32)], BF16),
    "grouped_gemm_wgrad": (lambda i, o: moe.grouped_gemm_wgrad(i[0], i[1], OFF, out=o[0]), [(4, 16), (4, 32)], [(2, 16, 32)], BF16),
    "quant_int8": (lambda i, o: moe.quant_int8(i[0], out=z(4, 32, dtype=INT8), scale=o[0])[1], [(4, 32)], [(4,)], BF16),
    "int8_gemm": (lambda i, o: moe.int8_gemm(z(4, 32, dtype=INT8), i[0], z(16, 32, dtype=INT8), i[1], out=o[0]), [(4,), (16,)],
                  [(4, 16)], torch.float32),
    "permute": (lambda i, o: moe.permute(i[0], PERM, 2, out=o[0]), [(2, 32)], [(4, 32)], BF16),
    "combine": (lambda i, o: moe.combine(i[0], PERM, i[1], out=o[0]), [(4, 32), (2, 2)], [(2, 32)], torch.float32),
    "combine_unweighted": (lambda i, o: moe.combine(i[0], PERM, k=2, out=o[0]), [(4, 32)], [(2, 32)], BF16),
    "combine_backward": (lambda i, o: moe.combine_backward(i[0], i[1], PERM, i[2], dy=o[0], dtopk_w=o[1]),
                         [(2, 32), (4, 32), (2, 2)], [(4, 32), (2, 2)], torch.float32),
}


class Accepts:
    """A library that takes every call and computes nothing."""
    def __getattr__(self, name):
        return lambda *a: moe.MOE_OK


@pytest.fixture
def no_library(monkeypatch):
    """The wrappers on CPU tensors, up to the library's door."""
    monkeypatch.setattr(moe, "lib", Accepts)
    monkeypatch.setattr(moe, "_on", lambda *a: None)
    monkeypatch.setattr(moe, "_call", lambda what, dev, stream, body: body(0))


def tensors(name):
    _, ins, outs, dtype = CALLS[name]
    f32 = ("quant_int8",)
    return [z(*s, dtype=dtype) for s in ins], [z(*s, dtype=torch.float32 if name in f32 else dtype) for s in outs]


@pytest.mark.parametrize("name", CALLS)
def test_a_backward_pass_through_a_result_raises(no_library, name):
    call = CALLS[name][0]
    for which in range(len(CALLS[name][1])):
        ins, outs = tensors(name)
        ins[which].requires_grad_()
        got = call(ins, outs)
        got = got if isinstance(got, tuple) else (got,)
        # dtopk_w does not depend on topk_w, nor dy on y
        linked = [g for i, g in enumerate(got) if name != "combine_backward" or (i, which) not in ((1, 2), (0, 1))]
        assert linked and all(g.requires_grad for g in linked)
        for g, o in zip(got, outs):
            assert g.data_ptr() == o.data_ptr() and g.stride() == o.stride()
            assert o.grad_fn is None and not o.requires_grad   # a buffer that is used again gathers no graph
        for g in linked:
            with pytest.raises(NotImplementedError, match="no autograd formula"):
                g.float().sum().backward()


@pytest.mark.parametrize("name", CALLS)
def test_calls_without_gradients_stay_outside_of_autograd(no_library, name):
    call = CALLS[name][0]
    for grad in (False, True):
        ins, outs = tensors(name)
        for i in ins:
            i.requires_grad_(grad)
        with torch.set_grad_enabled(not grad):
            got = call(ins, outs)
        for g, o in zip(got if isinstance(got, tuple) else (got,), outs):
            assert g is o and not g.requires_grad and g.grad_fn is None


@pytest.mark.parametrize("name", CALLS)
def test_a_graph_that_kept_an_overwritten_tensor_notices(no_library, name):
    call = CALLS[name][0]
    ins, outs = tensors(name)
    leaves = [torch.ones_like(o, requires_grad=True) for o in outs]
    kept = [leaf * o for leaf, o in zip(leaves, outs)]     # the product's backward reads o
    call(ins, outs)
    for k in kept:
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            k.float().sum().backward()


def test_status_of_the_operators_without_a_gpu():
    if not torch.cuda.is_available():
        assert moe.moe_ops_status(None) == moe.MOE_ERR_CUDA
