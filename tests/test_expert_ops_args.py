"""Refusals of the expert operators' C entry points: argument checks come
before any device work, so they run (and are tested) without a GPU."""
import ctypes

import pytest
import torch

from fp4_block_scaled_route_b200 import build as moe_build
from fp4_block_scaled_route_b200 import moe

OK, BAD, UNS, CUDA = moe.MOE_OK, moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_CUDA
A = 1 << 20      # an aligned address that is never dereferenced: every call here is refused or has no GPU


@pytest.fixture(scope="module", autouse=True)
def built():
    moe_build.build()


def grouped(fn, **kw):
    a = dict(dtype=0, out_dtype=0, E=2, P=4, N=16, K=32, offsets=A, x=A, ldx=None, w=A, ldw=None, stride_w=None, y=A,
             ldy=None, st=None, stream=None)
    a.update(kw)
    fwd = fn is moe.moe_grouped_gemm
    a["ldx"] = (a["K"] if fwd else a["N"]) if a["ldx"] is None else a["ldx"]
    a["ldy"] = (a["N"] if fwd else a["K"]) if a["ldy"] is None else a["ldy"]
    a["ldw"] = a["K"] if a["ldw"] is None else a["ldw"]
    a["stride_w"] = a["N"] * a["ldw"] if a["stride_w"] is None else a["stride_w"]
    return fn(*a.values())


PRODUCTS = pytest.mark.parametrize("fn", [moe.moe_grouped_gemm, moe.moe_grouped_gemm_dgrad],
                                   ids=["forward", "input_gradient"])


@PRODUCTS
def test_grouped_refusals(fn):
    for kw, want in [(dict(dtype=2), UNS), (dict(dtype=9), UNS), (dict(out_dtype=1), UNS), (dict(out_dtype=3), UNS),
                     (dict(E=0), BAD), (dict(E=1025), UNS), (dict(P=-1), BAD), (dict(P=(1 << 24) + 1), UNS),
                     (dict(N=0), BAD), (dict(K=0), BAD), (dict(N=(1 << 20) + 8), UNS), (dict(K=(1 << 20) + 8), UNS),
                     (dict(x=None), BAD), (dict(w=None), BAD), (dict(y=None), BAD), (dict(offsets=None), BAD),
                     (dict(x=A + 8), BAD), (dict(w=A + 2), BAD), (dict(y=A + 4), BAD), (dict(offsets=A + 2), BAD),
                     (dict(st=A + 1), BAD), (dict(ldx=36), BAD), (dict(ldy=36), BAD), (dict(ldx=8), BAD), (dict(ldy=8), BAD),
                     (dict(ldw=36), BAD), (dict(ldw=24), BAD), (dict(stride_w=8), BAD), (dict(stride_w=516), BAD),
                     (dict(ldx=1 << 40), BAD), (dict(stride_w=1 << 40), BAD)]:
        assert grouped(fn, **kw) == want, kw
    assert grouped(fn, P=0, x=None, y=None, w=None, offsets=None) == OK
    if not torch.cuda.is_available():
        assert grouped(fn) == CUDA
        assert grouped(fn, E=1, stride_w=0) == CUDA      # one expert: its stride is not looked at


def test_weight_gradient_refusals():
    def call(**kw):
        a = dict(dtype=0, out_dtype=0, E=2, P=4, N=16, K=32, offsets=A, dy=A, lddy=16, x=A, ldx=32, dw=A, st=None,
                 stream=None)
        a.update(kw)
        return moe.moe_grouped_gemm_wgrad(*a.values())
    for kw, want in [(dict(dtype=2), UNS), (dict(out_dtype=1), UNS), (dict(E=0), BAD), (dict(E=1025), UNS),
                     (dict(P=-1), BAD), (dict(P=(1 << 24) + 1), UNS), (dict(dw=None), BAD), (dict(dw=A + 8), BAD),
                     (dict(dy=None), BAD), (dict(x=None), BAD), (dict(offsets=None), BAD), (dict(dy=A + 2), BAD),
                     (dict(x=A + 2), BAD), (dict(lddy=12), BAD), (dict(lddy=20), BAD), (dict(ldx=24), BAD),
                     (dict(K=20, ldx=24), BAD), (dict(K=36, ldx=40), BAD), (dict(st=A + 2), BAD)]:
        assert call(**kw) == want, kw
    if not torch.cuda.is_available():
        assert call() == CUDA
        assert call(K=36, ldx=40, out_dtype=2) == CUDA   # fp32 rows of 36 are whole 16-byte pieces


def test_int8_refusals():
    def call(**kw):
        a = dict(out=0, E=2, P=4, N=16, K=32, offsets=A, q=A, ldq=32, qs=A, w=A, ldw=32, sw=512, ws=A, y=A, ldy=16,
                 st=None, stream=None)
        a.update(kw)
        return moe.moe_int8_gemm(*a.values())
    for kw, want in [(dict(out=3), UNS), (dict(out=-1), UNS), (dict(K=131072, ldq=131072, ldw=131072), UNS),
                     (dict(qs=None), BAD), (dict(ws=None), BAD), (dict(qs=A + 2), BAD), (dict(offsets=None), BAD),
                     (dict(ldq=40), BAD), (dict(ldw=40), BAD), (dict(ldy=12), BAD), (dict(out=2, ldy=18), BAD),
                     (dict(q=A + 8), BAD), (dict(E=0), BAD), (dict(E=1025), UNS)]:
        assert call(**kw) == want, kw
    assert call(P=0, q=None, qs=None, w=None, ws=None, y=None) == OK
    if not torch.cuda.is_available():
        assert call() == CUDA
        assert call(E=1, offsets=None, sw=0) == CUDA


def test_row_operator_refusals():
    def permute(**kw):
        a = dict(dtype=0, rows=8, H=32, T=4, k=2, x=A, ldx=32, perm=A, y=A, ldy=32, stream=None)
        a.update(kw)
        return moe.moe_permute(*a.values())

    def quant(**kw):
        a = dict(dtype=0, rows=8, K=32, T=4, k=2, x=A, ldx=32, perm=A, q=A, ldq=32, s=A, stream=None)
        a.update(kw)
        return moe.moe_quant_int8(*a.values())

    def combine(**kw):
        a = dict(dtype=0, rows=8, H=32, T=4, k=2, n_shared=0, y=A, ldy=32, inv=A, w=A, out=A, ldo=32, stream=None)
        a.update(kw)
        return moe.moe_combine(*a.values())

    def backward(**kw):
        a = dict(dtype=0, rows=8, H=32, T=4, k=2, n_shared=0, dout=A, ldd=32, y=A, ldy=32, inv=A, w=A, dy=A, lddy=32,
                 dw=A, stream=None)
        a.update(kw)
        return moe.moe_combine_backward(*a.values())
    for fn in (permute, quant, combine, backward):
        assert fn(dtype=3) == UNS and fn(dtype=-1) == UNS
        assert fn(rows=-1) == BAD and fn(T=-1) == BAD and fn(k=0) == BAD and fn(k=33) == UNS
        assert fn(rows=(1 << 24) + 1) == UNS and fn(T=(1 << 24) + 1) == UNS
    for fn in (permute, combine, backward):
        assert fn(H=0) == BAD and fn(H=(1 << 20) + 8) == UNS
    assert quant(dtype=2) == UNS and quant(K=0) == BAD
    for fn, names in ((permute, ("x", "perm", "y")), (quant, ("x", "q", "s")), (combine, ("y", "inv", "out")),
                      (backward, ("dout", "y", "inv", "w", "dy", "dw"))):
        for n in names:
            assert fn(**{n: None}) == BAD, (fn, n)
            assert fn(**{n: A + 2}) == BAD, (fn, n)
    for fn, names in ((permute, ("ldx", "ldy")), (quant, ("ldx", "ldq")), (combine, ("ldy", "ldo")),
                      (backward, ("ldd", "ldy", "lddy"))):
        for n in names:
            assert fn(**{n: 24}) == BAD and fn(**{n: 36}) == BAD, (fn, n)
    assert combine(n_shared=2) == UNS and combine(n_shared=-1) == BAD and backward(n_shared=2) == UNS
    assert quant(perm=None) == BAD          # 8 rows of 4 tokens
    assert permute(rows=0, x=None) == OK and quant(rows=0, x=None) == OK
    assert permute(T=0, x=None) == OK and combine(T=0, y=None) == OK and backward(T=0, y=None) == OK
    assert moe.moe_route(None, 1, A, A, A, A, A, None) == BAD


def test_wrappers_refuse_before_the_library():
    """torch-level mistakes raise ValueError naming the argument."""
    x, w, off = torch.zeros(4, 32), torch.zeros(2, 16, 32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        moe.grouped_gemm(x, w, off)
    with pytest.raises(ValueError, match="x has shape"):
        moe.grouped_gemm(torch.zeros(4, 24), w, off)
    with pytest.raises(ValueError, match="offsets has shape"):
        moe.grouped_gemm(x, w, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match=r"not \[E, N, K\]"):
        moe.grouped_gemm(x, w[0], off)
    with pytest.raises(ValueError, match="rows are not contiguous"):
        moe.grouped_gemm(torch.zeros(32, 4).T, w, off)
    with pytest.raises(ValueError, match="not supported"):
        moe.grouped_gemm(x.double(), w, off)
    with pytest.raises(ValueError, match="dy has shape"):
        moe.grouped_gemm_dgrad(x, w, off)
    with pytest.raises(ValueError, match="x has shape"):
        moe.grouped_gemm_wgrad(x, torch.zeros(5, 32), off)
    with pytest.raises(ValueError, match="one matrix without offsets"):
        moe.int8_gemm(x, x[:, 0], w, w[:, :, 0])
    with pytest.raises(ValueError, match="k has to be given"):
        moe.combine(x, off)
    with pytest.raises(ValueError, match="inv"):
        moe.combine(x, off, torch.zeros(4, 2))
    assert isinstance(moe.lib(), ctypes.CDLL)
