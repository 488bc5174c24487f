"""GPU tests of very long contractions, against sums in fp64.

The tensor cores truncate each addition to an accumulator, always towards
zero, so with terms of one sign the error grows with the number of additions
and does not average out.  An accumulator therefore takes a bounded number of
them, and the segments' sums are added with rounding.

Tolerance, for terms of one sign, relative to the sum: an addition takes 16
products and the accumulator, aligned to the largest of them and cut there at
24 bits or more, so each loses less than one unit in the last place, 2^-23 of
the partial sum, and the total as much again when it is cut: 17 + 1 units.  The
partial sums of a segment grow evenly, so they average half of it, with 2 % for
the unevenness of random terms.  A segment has 128 steps of 64 elements into
fp16 (512 additions) and 512 into bf16 (2048 additions): 512 / 2 * 18 * 2^-23 *
1.02 = 5.6e-4 and 2.2e-3.  The segments' own additions round 128 times at most,
2^-24 each, and the output once.  (One accumulator over these lengths is off by
1.5e-3 on fp16.)"""
import numpy as np
import pytest
import torch

from fp4_block_scaled_route_b200 import moe
from tests.test_gpu_grouped import WAYS

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
LOSS = {t: n / 2 * 18 * 2.0 ** -23 * 1.02 + 128 * 2.0 ** -24 for t, n in ((FP16, 512), (BF16, 2048))}
TYPES = pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def positive(gen, *shape, dtype, scale=1.0):
    return ((torch.rand(*shape, generator=gen, device="cuda") + 0.5) * scale).to(dtype)


def check(got, ref):
    """got against ref, whose terms have one sign."""
    err = ((got.double() - ref) / ref).abs()
    assert bool((err <= torch.finfo(got.dtype).eps / 2 + LOSS[got.dtype]).all()), float(err.max())


# rows of each group, features; by what computes them
@TYPES
@pytest.mark.parametrize("counts,M", [([300], 264), ([200, 0, 150], 136), ([40, 1, 70], 6000), ([5], 72), ([50], 200),
                                      ([300], 2056), ([200, 0, 150], 2056)],
                         ids=["large_shared", "large_groups_shared", "one_cta", "few_rows_shared", "shared", "pairs",
                              "pairs_handed_out"])
def test_long_products(dtype, counts, M):
    K = 1 << 20 if M < 1000 else 1 << 18
    off = offsets_of(counts)
    P, E = sum(counts), len(counts)
    gen = torch.Generator("cuda").manual_seed(P)
    x = positive(gen, P, K, dtype=dtype)
    w = positive(gen, E, M, K, dtype=dtype, scale=2.0 ** -8)
    ref = torch.cat([x[a:b].double() @ w[e].double().T for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:]))])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = moe.grouped_gemm(x, w, off, status=status)
    check(y, ref)
    assert torch.equal(y, moe.grouped_gemm(x, w, off))
    wt = w.transpose(1, 2).contiguous()   # the input gradient's contraction runs over w's rows
    del w
    check(moe.grouped_gemm_dgrad(x, wt, off, status=status), ref)
    assert int(status) == 0


@TYPES
@pytest.mark.parametrize("counts,N,K", [([262149, 8192, 8193, 0, 16385, 3, 32768, 40000] + [0, 70] * 16, 256, 256),
                                        ([16384, 8191, 24577] * 20, 136, 200), ([1 << 19], 200, 256), ([1 << 18, 5], 40, 72)],
                         ids=["whole_tiles", "several_tiles_a_pair", "shared_by_four", "shared_by_two_groups"])
def test_weight_gradients_of_long_groups(dtype, counts, N, K):
    off = offsets_of(counts)
    P = sum(counts)
    gen = torch.Generator("cuda").manual_seed(N)
    x = positive(gen, P, K, dtype=dtype)
    dy = positive(gen, P, N, dtype=dtype, scale=2.0 ** -8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dw = moe.grouped_gemm_wgrad(dy, x, off, status=status)
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        if a == b:
            assert not dw[e].any()
        else:
            check(dw[e], dy[a:b].double().T @ x[a:b].double())
    assert torch.equal(dw, moe.grouped_gemm_wgrad(dy, x, off)) and int(status) == 0


# The 2-norm that the kernels' comments state for fp32 results of terms of random signs, 1.0e-6 (bf16) and 1.3e-6 (fp16),
# with half as much again: whatever the length, since the segments' own additions round by 2^-24 (6e-8) each.  One
# accumulator over 7168 elements is off by 6.6e-6, a result rounded to fp16 by 2e-4.
NORM = 2e-6


@TYPES
@pytest.mark.parametrize("counts,N,K", [([32768] + [0] * 7, 256, 256), ([0, 20001, 3, 11000, 0, 70], 200, 136)],
                         ids=["all_in_one", "uneven"])
def test_shared_weight_gradients_into_fp32_of_uneven_groups(dtype, counts, N, K):
    """How many pairs share a tile's rows goes by the average group; the accuracy of a longer one may not."""
    off = offsets_of(counts)
    P = sum(counts)
    gen = torch.Generator("cuda").manual_seed(N)
    dy, x = (torch.randn(P, n, generator=gen, device="cuda").to(dtype) for n in (N, K))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dw = moe.grouped_gemm_wgrad(dy, x, off, out_dtype=FP32, status=status)
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        ref = dy[a:b].double().T @ x[a:b].double()
        assert float((dw[e].double() - ref).norm()) <= NORM * float(ref.norm()), e
    assert torch.equal(dw, moe.grouped_gemm_wgrad(dy, x, off, out_dtype=FP32)) and int(status) == 0


def norms_fit(got, ref):
    assert float((got.double() - ref).norm()) <= NORM * float(ref.norm())


@TYPES
@pytest.mark.parametrize("counts,N,K", [*WAYS.values(), ([3, 0, 9], 1032, 7176), ([60], 1032, 7176), ([700, 40, 300], 1032, 7176),
                                        ([130, 257, 500, 0, 64] * 3, 1032, 7176)],
                         ids=[*WAYS, "few_7176", "some_7176", "few_large_7176", "pairs_7176"])
def test_products_into_fp32_in_the_2_norm(dtype, counts, N, K):
    """Elementwise bounds have to allow for every addition's worst case; the 2-norm shows what the additions do."""
    off = offsets_of(counts)
    gen = torch.Generator("cuda").manual_seed(N + K)
    x, w = (torch.randn(*s, generator=gen, device="cuda").to(dtype) for s in ((sum(counts), K), (len(counts), N, K)))
    ref = torch.cat([x[a:b].double() @ w[e].double().T for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:]))])
    norms_fit(moe.grouped_gemm(x, w, off, out_dtype=FP32), ref)
    norms_fit(moe.grouped_gemm_dgrad(x, w.transpose(1, 2).contiguous(), off, out_dtype=FP32), ref)


@TYPES
@pytest.mark.parametrize("counts,N,K", [([5000, 1, 1030, 0, 2048, 1024], 264, 1160), ([9001], 1800, 2056), ([4096], 136, 200),
                                        ([20000] * 3, 520, 2056), ([300, 7, 0, 900] * 20, 136, 264)])
def test_weight_gradients_into_fp32_in_the_2_norm(dtype, counts, N, K):
    off = offsets_of(counts)
    gen = torch.Generator("cuda").manual_seed(N + K)
    dy, x = (torch.randn(sum(counts), n, generator=gen, device="cuda").to(dtype) for n in (N, K))
    dw = moe.grouped_gemm_wgrad(dy, x, off, out_dtype=FP32)
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        norms_fit(dw[e], dy[a:b].double().T @ x[a:b].double())
