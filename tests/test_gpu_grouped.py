"""GPU tests of the ragged grouped products (moe_grouped_gemm, its two
gradients) and the int8 product against the definitions in fp64.

Tolerance of a 16-bit product, per element, with A = sum of |terms| over the
contraction of length R: every product of two 16-bit values is exact in fp32;
the tensor cores add R of them with at most one unit in the last place
(2^-23, truncation allowed) of a partial sum, which A bounds, per addition;
then one rounding to the output type (eps / 2 relative, half the smallest
subnormal below the normal range).  Int8 sums are exact; converting the sum
and the two scale products round three times (2^-24 each), then the output
once.
"""
import numpy as np
import pytest
import torch

from fp4_block_scaled_route_b200 import moe

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TINY = {BF16: 2.0 ** -133, FP16: 2.0 ** -24, FP32: 2.0 ** -149}  # smallest subnormals


def offsets_of(counts, start=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + start, dtype=torch.int32, device="cuda")


def randn(gen, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def tol16(ref, A, R, out):
    return torch.finfo(out).eps / 2 * ref.abs() + (R + 16) * 2.0 ** -23 * A * 1.01 + TINY[out]


def check(got, ref, tol):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    bad = err > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((err / tol).max()))


def forward64(x, w, off, contract="k"):
    """(ref, A) of the forward (contract k) or the input gradient (contract n)."""
    eq = "pk,nk->pn" if contract == "k" else "pn,nk->pk"
    cols = w.shape[1] if contract == "k" else w.shape[2]
    ref = torch.zeros(x.shape[0], cols, dtype=torch.float64, device="cuda")
    A = torch.zeros_like(ref)
    o = off.tolist()
    for e in range(len(o) - 1):
        s = slice(o[e], o[e + 1])
        ref[s] = torch.einsum(eq, x[s].double(), w[e].double())
        A[s] = torch.einsum(eq, x[s].double().abs(), w[e].double().abs())
    return ref, A


def wgrad64(dy, x, off):
    o = off.tolist()
    ref = torch.stack([dy[o[e]:o[e + 1]].double().T @ x[o[e]:o[e + 1]].double() for e in range(len(o) - 1)])
    A = torch.stack([dy[o[e]:o[e + 1]].double().abs().T @ x[o[e]:o[e + 1]].double().abs()
                     for e in range(len(o) - 1)])
    return ref, A


GROUPS = {
    "one_row": [1],
    "empty_between": [0, 5, 0, 17, 0],
    "sixteen": [16, 16, 15, 17],
    "ragged": [130, 0, 1, 64, 129, 31],
    "one_large": [700],
    "large_and_rare": [520, 3, 0, 257],
    "many": [(7 * i) % 5 for i in range(300)],
    "most": [(i % 97 == 0) * 3 for i in range(1024)],
}
SIZES = [(128, 64), (8, 8), (136, 72), (264, 200), (384, 520)]


@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (FP16, FP32)], ids=["bf16", "fp16_fp32"])
def test_forward_and_input_gradient(groups, N, K, dtype, out):
    counts = GROUPS[groups]
    off = offsets_of(counts)
    P, E = sum(counts), len(counts)
    gen = torch.Generator("cuda").manual_seed(P * 1000 + N + K)
    w = randn(gen, E, N, K, dtype=dtype)
    x = randn(gen, P, K, dtype=dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = moe.grouped_gemm(x, w, off, out_dtype=out, status=status)
    ref, A = forward64(x, w, off)
    check(y, ref, tol16(ref, A, K, out))
    dy = randn(gen, P, N, dtype=dtype)
    dx = moe.grouped_gemm_dgrad(dy, w, off, out_dtype=out, status=status)
    ref, A = forward64(dy, w, off, "n")
    check(dx, ref, tol16(ref, A, N, out))
    assert int(status) == 0


@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (FP16, FP32)], ids=["bf16", "fp16_fp32"])
def test_weight_gradient(groups, N, K, dtype, out):
    counts = GROUPS[groups]
    off = offsets_of(counts)
    P = sum(counts)
    gen = torch.Generator("cuda").manual_seed(P * 1000 + N + K)
    dy, x = randn(gen, P, N, dtype=dtype), randn(gen, P, K, dtype=dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dw = moe.grouped_gemm_wgrad(dy, x, off, out_dtype=out, status=status)
    ref, A = wgrad64(dy, x, off)
    check(dw, ref, tol16(ref, A, max(counts), out))
    assert int(status) == 0
    for e, c in enumerate(counts):
        if c == 0:
            assert not dw[e].any()


@pytest.mark.parametrize("dtype,out", [(FP16, FP16), (BF16, FP32)], ids=["fp16", "bf16_fp32"])
def test_long_contractions_and_wide_tiles(dtype, out):
    """Several full tiles in each direction, and more stages than the pipeline holds."""
    counts = [300, 0, 1100, 2]
    off = offsets_of(counts)
    P, E, N, K = sum(counts), len(counts), 1160, 2056
    gen = torch.Generator("cuda").manual_seed(5)
    w, x, dy = (randn(gen, *s, dtype=dtype) for s in ((E, N, K), (P, K), (P, N)))
    w *= 0.05
    ref, A = forward64(x, w, off)
    check(moe.grouped_gemm(x, w, off, out_dtype=out), ref, tol16(ref, A, K, out))
    ref, A = forward64(dy, w, off, "n")
    check(moe.grouped_gemm_dgrad(dy, w, off, out_dtype=out), ref, tol16(ref, A, N, out))
    dy *= 0.05
    ref, A = wgrad64(dy, x, off)
    check(moe.grouped_gemm_wgrad(dy, x, off, out_dtype=out), ref, tol16(ref, A, max(counts), out))


@pytest.mark.parametrize("rows", [3, 40, 600], ids=["few", "some", "many"])
def test_rows_outside_the_groups(rows):
    """Rows before the first and behind the last group hold NaN: outputs there stay, and nothing leaks."""
    counts = [rows, 0, rows + 5]
    start, tail = 11, 13
    off = offsets_of(counts, start)
    P, E, N, K = sum(counts) + start + tail, 3, 72, 136
    gen = torch.Generator("cuda").manual_seed(rows)
    w, x, dy = (randn(gen, *s, dtype=BF16) for s in ((E, N, K), (P, K), (P, N)))
    outside = torch.ones(P, dtype=torch.bool, device="cuda")
    outside[start:P - tail] = False
    x[outside] = float("nan")
    dy[outside] = float("inf")
    for fn, a, cols, contract in ((moe.grouped_gemm, x, N, "k"), (moe.grouped_gemm_dgrad, dy, K, "n")):
        y = torch.full((P, cols), 7.0, dtype=BF16, device="cuda")
        fn(a, w, off, out=y)
        assert (y[outside] == 7.0).all()
        ref, A = forward64(a, w, off, contract)
        held = ~outside
        check(y[held], ref[held], tol16(ref, A, w.shape[2 if contract == "k" else 1], BF16)[held])
    ref, A = wgrad64(dy, x, off)
    check(moe.grouped_gemm_wgrad(dy, x, off), ref, tol16(ref, A, max(counts), BF16))


def test_a_groups_nan_stays_in_its_group():
    """A NaN row of one group must not reach the groups whose tiles load it beside their own rows."""
    counts = [5, 1, 20, 3]
    off = offsets_of(counts)
    P, E, N, K = sum(counts), 4, 136, 200
    gen = torch.Generator("cuda").manual_seed(2)
    w, x, dy = (randn(gen, *s, dtype=FP16) for s in ((E, N, K), (P, K), (P, N)))
    x[5] = float("nan")
    dy[5] = float("inf")
    w[1, 3, 7] = float("nan")
    y = moe.grouped_gemm(x, w, off)
    assert torch.isnan(y[5]).all()
    keep = [i for i in range(P) if i != 5]
    ref, A = forward64(x, w, off)
    check(y[keep], ref[keep], tol16(ref, A, K, FP16)[keep])
    dx = moe.grouped_gemm_dgrad(dy, w, off)
    ref, A = forward64(dy, w, off, "n")
    check(dx[keep], ref[keep], tol16(ref, A, N, FP16)[keep])
    dw = moe.grouped_gemm_wgrad(dy, x, off)
    assert torch.isnan(dw[1]).all()
    ref, A = wgrad64(dy, x, off)
    check(dw[[0, 2, 3]], ref[[0, 2, 3]], tol16(ref, A, max(counts), FP16)[[0, 2, 3]])


def test_strided_operands():
    """Row strides longer than the rows, halves of a joint matrix, a window of its columns."""
    counts = [9, 33, 0, 70]
    off = offsets_of(counts)
    P, E, N, K = sum(counts), 4, 72, 104
    gen = torch.Generator("cuda").manual_seed(3)
    joint = randn(gen, E, 2 * N, K + 24, dtype=BF16)
    big_x, big_dy = randn(gen, P, K + 40, dtype=BF16), randn(gen, P, N + 8, dtype=BF16)
    x, dy = big_x[:, 8:8 + K], big_dy[:, :N]
    for w in (joint[:, N:, :K], joint[:, :N, 8:8 + K]):
        out = torch.full((P, N + 16), 3.0, dtype=FP32, device="cuda")
        moe.grouped_gemm(x, w, off, out=out[:, 8:8 + N])
        ref, A = forward64(x, w, off)
        check(out[:, 8:8 + N], ref, tol16(ref, A, K, FP32))
        assert (out[:, :8] == 3.0).all() and (out[:, 8 + N:] == 3.0).all()
        ref, A = forward64(dy, w, off, "n")
        check(moe.grouped_gemm_dgrad(dy, w, off), ref, tol16(ref, A, N, BF16))
    ref, A = wgrad64(dy, x, off)
    check(moe.grouped_gemm_wgrad(dy, x, off), ref, tol16(ref, A, max(counts), BF16))


@pytest.mark.parametrize("N,K", [(129, 104), (65, 40), (7, 24)])
def test_odd_widths_within_aligned_rows(N, K):
    """Any N or K, as long as the row strides are multiples of 16 bytes."""
    counts = [20, 90]
    off = offsets_of(counts)
    gen = torch.Generator("cuda").manual_seed(4)
    P = sum(counts)
    K1 = K - 3
    w = randn(gen, 2, N, K, dtype=FP16)[:, :, :K1]
    x = randn(gen, P, K, dtype=FP16)[:, :K1]
    ldn = (N + 7) // 8 * 8
    y = torch.full((P, ldn), 9.0, dtype=FP16, device="cuda")
    moe.grouped_gemm(x, w, off, out=y[:, :N])
    ref, A = forward64(x, w, off)
    check(y[:, :N], ref, tol16(ref, A, K1, FP16))
    assert (y[:, N:] == 9.0).all()
    dy = randn(gen, P, ldn, dtype=FP16)[:, :N]
    dx = torch.full((P, K), 9.0, dtype=FP16, device="cuda")
    moe.grouped_gemm_dgrad(dy, w, off, out=dx[:, :K1])
    ref, A = forward64(dy, w, off, "n")
    check(dx[:, :K1], ref, tol16(ref, A, N, FP16))
    assert (dx[:, K1:] == 9.0).all()


@pytest.mark.parametrize("off", [[0, 5, 4, 10], [-1, 3, 6, 10], [0, 5, 8, 11], [4, 2, 2, 2], [0, 2 ** 31 - 1, 3, 10]],
                         ids=["falling", "negative", "past_the_rows", "start_falls", "huge"])
def test_unusable_offsets_compute_nothing(off):
    P, E, N, K = 10, 3, 16, 64
    x = torch.ones(P, K, dtype=BF16, device="cuda")
    w = torch.ones(E, N, K, dtype=BF16, device="cuda")
    dy = torch.ones(P, N, dtype=BF16, device="cuda")
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    for call, shape in ((lambda out, st: moe.grouped_gemm(x, w, o, out=out, status=st), (P, N)),
                        (lambda out, st: moe.grouped_gemm_dgrad(dy, w, o, out=out, status=st), (P, K)),
                        (lambda out, st: moe.grouped_gemm_wgrad(dy, x, o, out=out, status=st), (E, N, K))):
        out = torch.full(shape, 5.0, dtype=BF16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(out, status)
        assert int(status) == 1 and (out == 5.0).all()
        call(out, None)   # no status word: still nothing computed
        torch.cuda.synchronize()
        assert (out == 5.0).all()


# Shapes that reach every way a call is tiled on 148 SMs: rows per tile, shares
# of the contraction, pairs, pieces of the last wave, units handed out at run time.
WAYS = {
    "rows16_split8": ([7], 520, 4160),
    "rows16_split8_at_most": ([16], 1912, 4104),
    "rows16_split4": ([3, 0, 9], 1160, 2056),
    "rows16_split2": ([3, 2, 9], 2056, 1032),
    "rows32_split4": ([17], 4096, 2056),
    "rows32_split2": ([20, 5, 12, 9], 1032, 1096),
    "rows64_split4": ([60], 136, 3080),
    "rows64_split2": ([64], 4232, 1544),
    "rows64_few_large": ([300, 0, 41], 264, 2056),
    "rows64_short": ([9, 3], 4000, 136),
    "rows64_many": ([13, 9, 20, 2, 10], 2056, 1992),
    "rows64": ([31, 33, 20, 40], 1032, 328),
    "rows64_two_tiles": ([1, 100, 0, 130, 5], 2056, 1032),
    "pairs": ([300, 500, 65, 129], 2056, 520),
    "pairs_pieces": ([2048], 1288, 648),
    "pairs_handed_out": ([700, 3, 333, 0, 512, 1100], 2824, 2056),
    "pairs_handed_out_few_units": ([257, 64, 130, 0, 0, 0, 1], 1544, 2120),
}


@pytest.mark.parametrize("way", WAYS)
def test_every_tiling(way):
    counts, N, K = WAYS[way]
    off = offsets_of(counts)
    P, E = sum(counts), len(counts)
    gen = torch.Generator("cuda").manual_seed(N)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w, x = randn(gen, E, N, K, dtype=BF16), randn(gen, P, K, dtype=BF16)
    y = moe.grouped_gemm(x, w, off, out_dtype=FP32, status=status)
    ref, A = forward64(x, w, off)
    check(y, ref, tol16(ref, A, K, FP32))
    assert torch.equal(y, moe.grouped_gemm(x, w, off, out_dtype=FP32))   # no sum depends on timing
    # the gradient's contraction runs over w's rows: the same tiling with the sizes exchanged
    wt = w.transpose(1, 2).contiguous()
    dx = moe.grouped_gemm_dgrad(x, wt, off, out_dtype=FP32, status=status)
    check(dx, ref, tol16(ref, A, K, FP32))
    K8 = 2 * (K // 16 * 16)   # as many steps of 128 bytes
    q = torch.randint(-128, 128, (P, K8), generator=gen, device="cuda", dtype=torch.int8)
    w8 = torch.randint(-128, 128, (E, N, K8), generator=gen, device="cuda", dtype=torch.int8)
    s, c = torch.rand(P, generator=gen, device="cuda"), torch.rand(E, N, generator=gen, device="cuda")
    for out in (BF16, FP32):
        y = moe.int8_gemm(q, s, w8, c, offsets=off, out_dtype=out, status=status)
        check_int8(y, int8_64(q, s, w8, c, off), out)
    assert int(status) == 0


@pytest.mark.parametrize("counts", [[3, 0, 9], [60], [700, 40, 300], [130, 257, 500, 0, 64] * 3], ids=["few", "some", "few_large", "pairs"])
def test_long_contractions_into_fp32(counts):
    """fp32 results add up segments of 1024: the truncated additions of a segment, and one rounding per segment."""
    off = offsets_of(counts)
    P, E, N, K = sum(counts), len(counts), 1032, 7176
    gen = torch.Generator("cuda").manual_seed(31)
    w, x = randn(gen, E, N, K, dtype=BF16), randn(gen, P, K, dtype=BF16)
    ref, A = forward64(x, w, off)
    tol = (1024 + 16 + 8) * 2.0 ** -23 * A
    check(moe.grouped_gemm(x, w, off, out_dtype=FP32), ref, tol)
    check(moe.grouped_gemm_dgrad(x, w.transpose(1, 2).contiguous(), off, out_dtype=FP32), ref, tol)


def test_long_groups_into_fp32():
    """The same for weight gradients, over groups of many rows and short ones."""
    for counts, N, K in (([5000, 1, 1030, 0, 2048, 1024], 264, 1160), ([9001], 1800, 2056), ([4096], 136, 200)):
        off = offsets_of(counts)
        P = sum(counts)
        gen = torch.Generator("cuda").manual_seed(32)
        dy, x = randn(gen, P, N, dtype=BF16), randn(gen, P, K, dtype=BF16)
        ref, A = wgrad64(dy, x, off)
        dw = moe.grouped_gemm_wgrad(dy, x, off, out_dtype=FP32)
        check(dw, ref, (1024 + 16 + 9) * 2.0 ** -23 * A + TINY[FP32])
        assert torch.equal(dw, moe.grouped_gemm_wgrad(dy, x, off, out_dtype=FP32))


def test_weight_gradient_tilings():
    """Whole waves of tiles, halves of the last wave, more experts than the larger pipeline has room for, and few tiles
    whose rows two or four pairs share (some of them without any)."""
    gen = torch.Generator("cuda").manual_seed(12)
    for counts, N, K in (([200, 0, 77], 1800, 3336), ([64] * 37, 264, 520), ([3, 0, 1, 20] * 130, 136, 72),
                         ([5000], 520, 392), ([2100], 136, 200), ([1, 0, 4000, 63], 264, 136), ([1300, 1000], 504, 776),
                         ([3001], 40, 8), ([1, 4099, 70, 2111] * 5, 520, 1032)):
        off = offsets_of(counts)
        P = sum(counts)
        dy, x = randn(gen, P, N, dtype=FP16), randn(gen, P, K, dtype=FP16)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        dw = moe.grouped_gemm_wgrad(dy, x, off, out_dtype=FP32, status=status)
        ref, A = wgrad64(dy, x, off)
        check(dw, ref, tol16(ref, A, max(counts), FP32))
        assert torch.equal(dw, moe.grouped_gemm_wgrad(dy, x, off, out_dtype=FP32)) and int(status) == 0
        dw = moe.grouped_gemm_wgrad(dy, x, off)
        check(dw, ref, tol16(ref, A, max(counts), FP16))


def test_more_than_2_to_31_elements():
    """Rows that start past 2^31 elements, of the operands and of the outputs."""
    P, K, N, n = 263000, 8200, 16, 300     # P * K = 2.16e9
    x = torch.zeros(P, K, dtype=BF16, device="cuda")
    gen = torch.Generator("cuda").manual_seed(13)
    x[-n:] = randn(gen, n, K, dtype=BF16)
    w = randn(gen, 2, N, K, dtype=BF16)
    off = torch.tensor([0, P - n // 2, P], dtype=torch.int32, device="cuda")
    tail = torch.tensor([0, n // 2, n], dtype=torch.int32, device="cuda")
    y = moe.grouped_gemm(x, w, off, out_dtype=FP32)
    ref, A = forward64(x[-n:], w, tail)
    check(y[-n:], ref, tol16(ref, A, K, FP32))
    assert not y[:-n].any()
    dw = moe.grouped_gemm_wgrad(y.to(BF16), x, off, out_dtype=FP32)
    ref, A = wgrad64(y[-n:].to(BF16), x[-n:], tail)
    check(dw, ref, tol16(ref, A, n, FP32))
    moe.grouped_gemm_dgrad(y.to(BF16), w, off, out=x)
    ref, A = forward64(y[-n:].to(BF16), w, tail, "n")
    check(x[-n:], ref, tol16(ref, A, N, BF16))
    q, s = moe.quant_int8(x)
    q2, s2 = moe.quant_int8(x[-n:].contiguous())
    assert torch.equal(q[-n:], q2) and torch.equal(s[-n:], s2)
    perm = torch.arange(P, dtype=torch.int32, device="cuda").flip(0).contiguous()
    moved = moe.permute(x, perm, 1)
    assert torch.equal(moved[:n], x[-n:].flip(0))
    back = moe.combine(moved, perm, k=1)
    assert torch.equal(back[-n:], x[-n:])


def test_no_rows():
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    w = torch.ones(3, 16, 64, dtype=BF16, device="cuda")
    x, dy = (torch.empty(0, n, dtype=BF16, device="cuda") for n in (64, 16))
    assert moe.grouped_gemm(x, w, off).shape == (0, 16)
    assert moe.grouped_gemm_dgrad(dy, w, off).shape == (0, 64)
    dw = torch.full((3, 16, 64), 4.0, dtype=BF16, device="cuda")
    moe.grouped_gemm_wgrad(dy, x, off, out=dw)
    assert not dw.any()
    # rows, but none in a group
    x, dy = (torch.full((5, n), float("nan"), dtype=BF16, device="cuda") for n in (64, 16))
    y = torch.full((5, 16), 4.0, dtype=BF16, device="cuda")
    moe.grouped_gemm(x, w, off, out=y)
    assert (y == 4.0).all()
    dw.fill_(4.0)
    moe.grouped_gemm_wgrad(dy, x, off, out=dw)
    assert not dw.any()


def test_gradients_against_differences():
    """The gradients of sum(y * c) agree with central differences of the fp64 product (which is linear, so the
    difference quotient is exact up to rounding)."""
    counts = [4, 0, 6]
    off = offsets_of(counts)
    P, E, N, K = 10, 3, 24, 40
    gen = torch.Generator("cuda").manual_seed(8)
    w, x, c = (randn(gen, *s, dtype=BF16) for s in ((E, N, K), (P, K), (P, N)))
    dx = moe.grouped_gemm_dgrad(c, w, off, out_dtype=FP32)
    dw = moe.grouped_gemm_wgrad(c, x, off, out_dtype=FP32)

    def loss(xx, ww):
        return sum((torch.einsum("pk,nk->pn", xx[a:b], ww[e]) * c[a:b].double()).sum()
                   for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])))
    for p, k in ((0, 0), (3, 39), (9, 17)):
        d = torch.zeros(P, K, dtype=torch.float64, device="cuda")
        d[p, k] = 0.5
        diff = loss(x.double() + d, w.double()) - loss(x.double() - d, w.double())
        assert abs(float(dx[p, k]) - float(diff)) <= 1e-4 * (1 + abs(float(diff)))
    for e, n, k in ((0, 0, 0), (2, 23, 39), (1, 5, 5)):
        d = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
        d[e, n, k] = 0.5
        diff = loss(x.double(), w.double() + d) - loss(x.double(), w.double() - d)
        assert abs(float(dw[e, n, k]) - float(diff)) <= 1e-4 * (1 + abs(float(diff)))


def test_captured_and_replayed_with_new_offsets():
    """One captured graph follows the device's offsets and inputs."""
    P, E, N, K = 96, 6, 136, 264
    gen = torch.Generator("cuda").manual_seed(6)
    w = randn(gen, E, N, K, dtype=BF16)
    x, dy = torch.zeros(P, K, dtype=BF16, device="cuda"), torch.zeros(P, N, dtype=BF16, device="cuda")
    off = offsets_of([16] * E)
    y, dx = torch.zeros(P, N, dtype=BF16, device="cuda"), torch.zeros(P, K, dtype=BF16, device="cuda")
    dw = torch.zeros(E, N, K, dtype=BF16, device="cuda")

    def step():
        moe.grouped_gemm(x, w, off, out=y)
        moe.grouped_gemm_dgrad(dy, w, off, out=dx)
        moe.grouped_gemm_wgrad(dy, x, off, out=dw)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for counts in ([96, 0, 0, 0, 0, 0], [1, 2, 3, 40, 49, 1], [0, 0, 0, 0, 0, 0], [20, 20, 20, 0, 20, 16]):
        off.copy_(offsets_of(counts))
        x.copy_(randn(gen, P, K, dtype=BF16))
        dy.copy_(randn(gen, P, N, dtype=BF16))
        y.zero_(), dx.zero_()
        graph.replay()
        ref, A = forward64(x, w, off)
        check(y, ref, tol16(ref, A, K, BF16))
        ref, A = forward64(dy, w, off, "n")
        check(dx, ref, tol16(ref, A, N, BF16))
        ref, A = wgrad64(dy, x, off)
        check(dw, ref, tol16(ref, A, max(counts), BF16))


def test_two_streams_at_once():
    """Calls share nothing: results on two streams equal the ones computed alone, bit for bit."""
    gen = torch.Generator("cuda").manual_seed(7)
    sets = []
    for counts in ([200, 30, 0, 400], [3, 1, 0, 9]):
        off, P = offsets_of(counts), sum(counts)
        x, w, dy = (randn(gen, *s, dtype=BF16) for s in ((P, 1032), (4, 520, 1032), (P, 520)))
        sets.append((x, w, dy, off))

    def outputs(x, w, dy, off, stream=None):
        return (moe.grouped_gemm(x, w, off, stream=stream), moe.grouped_gemm_dgrad(dy, w, off, stream=stream),
                moe.grouped_gemm_wgrad(dy, x, off, stream=stream))
    alone = [outputs(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        both = [outputs(*s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            for u, v in zip(a, b):
                assert torch.equal(u, v)


def test_two_graphs_replayed_at_once():
    """Two captured graphs of the same calls run side by side: there is no shared workspace."""
    gen = torch.Generator("cuda").manual_seed(17)
    counts = [40, 0, 7, 300, 21]
    off, P, E, N, K = offsets_of(counts), sum(counts), len(counts), 520, 2056
    sets, graphs = [], []
    for i in range(2):
        x, w, dy = randn(gen, P, K, dtype=BF16), randn(gen, E, N, K, dtype=BF16), randn(gen, P, N, dtype=BF16)
        w8 = torch.randint(-128, 128, (E, N, K + 8), generator=gen, device="cuda", dtype=torch.int8)[:, :, :K]

        def step(x=x, w=w, dy=dy, w8=w8):
            q, s = moe.quant_int8(x)   # (rows of K = 2056 bytes, padded to a multiple of 16)
            return (moe.grouped_gemm(x, w, off), moe.grouped_gemm_dgrad(dy, w, off), moe.grouped_gemm_wgrad(dy, x, off),
                    moe.int8_gemm(q, s, w8, torch.ones(E, N, device="cuda"), offsets=off))
        alone = step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        sets.append((alone, out, torch.cuda.Stream(), step))   # (step keeps the graph's inputs alive)
        graphs.append(g)
    for _ in range(5):
        for g, (_, out, st, _) in zip(graphs, sets):
            with torch.cuda.stream(st):
                for t in out:
                    t.zero_()
                g.replay()
        torch.cuda.synchronize()
        for alone, out, _, _ in sets:
            for a, b in zip(alone, out):
                assert torch.equal(a, b)


# ---- int8 ----------------------------------------------------------------------
def int8_64(q, s, w, c, off):
    y = torch.zeros(q.shape[0], w.shape[1], dtype=torch.float64, device="cuda")
    o = off.tolist()
    for e in range(len(o) - 1):
        r = slice(o[e], o[e + 1])
        y[r] = (q[r].double() @ w[e].double().T) * s[r].double()[:, None] * c[e].double()
    return y


def check_int8(y, ref, out):
    check(y, ref, ref.abs() * (torch.finfo(out).eps / 2 + 4 * 2.0 ** -24) + TINY[out])


@pytest.mark.parametrize("groups", GROUPS)
@pytest.mark.parametrize("N,K", [(128, 128), (8, 16), (136, 272), (392, 528)])
@pytest.mark.parametrize("out", [BF16, FP16, FP32], ids=["bf16", "fp16", "fp32"])
def test_int8_experts(groups, N, K, out):
    counts = GROUPS[groups]
    off = offsets_of(counts)
    P, E = sum(counts), len(counts)
    gen = torch.Generator("cuda").manual_seed(P + N + K)
    q = torch.randint(-128, 128, (P, K), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (E, N, K), generator=gen, device="cuda", dtype=torch.int8)
    s = torch.rand(P, generator=gen, device="cuda") * 0.01 + 1e-3
    c = torch.rand(E, N, generator=gen, device="cuda") * 0.01 + 1e-3
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = moe.int8_gemm(q, s, w, c, offsets=off, out_dtype=out, status=status)
    check_int8(y, int8_64(q, s, w, c, off), out)
    assert int(status) == 0


@pytest.mark.parametrize("P", [1, 5, 17, 100, 513])
@pytest.mark.parametrize("N,K", [(64, 16), (1000, 2064)])
def test_int8_dense(P, N, K):
    gen = torch.Generator("cuda").manual_seed(P)
    q = torch.randint(-128, 128, (P, K), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    s, c = (torch.rand(n, generator=gen, device="cuda") * 0.01 for n in (P, N))
    y = moe.int8_gemm(q, s, w, c)
    assert y.dtype == BF16
    check_int8(y, int8_64(q, s, w[None], c[None], torch.tensor([0, P])), BF16)


def test_int8_sums_fill_32_bits():
    """The largest K with every product at its extreme: +-128 * 128 * K is exact."""
    K = 131056
    q = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((16, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    w[2, ::2] = 127
    one = torch.ones(16, device="cuda")
    y = moe.int8_gemm(q, one[:3], w, one, out_dtype=FP32)
    check_int8(y, int8_64(q, one[:3], w[None], one[None], torch.tensor([0, 3])), FP32)


def test_int8_row_without_a_finite_scale():
    """A row that held an infinity or a NaN has scale NaN and zero codes: its products are NaN, the others' are not."""
    x = torch.randn(9, 160, device="cuda").to(FP16)
    x[3, 7] = float("inf")
    x[8, 0] = float("nan")
    q, s = moe.quant_int8(x)
    w = torch.randint(-128, 128, (40, 160), device="cuda", dtype=torch.int8)
    c = torch.ones(40, device="cuda")
    y = moe.int8_gemm(q, s, w, c)
    assert torch.isnan(y[[3, 8]]).all()
    keep = [0, 1, 2, 4, 5, 6, 7]
    check_int8(y[keep], int8_64(q, s, w[None], c[None], torch.tensor([0, 9]))[keep], BF16)


def test_groups_that_cover_few_of_many_rows():
    """Most of the launch's room for tiles stays unused: one small group, or none, in many rows."""
    P, E, N, K = 60000, 4, 1032, 2056
    gen = torch.Generator("cuda").manual_seed(21)
    x, w = randn(gen, P, K, dtype=BF16), randn(gen, E, N, K, dtype=BF16)
    for off in ([100, 100, 400, 407, 407], [0, 0, 0, 0, 0], [P, P, P, P, P]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        y = torch.full((P, N), 2.0, dtype=FP32, device="cuda")
        moe.grouped_gemm(x, w, o, out=y)
        ref, A = forward64(x[:512], w, o.clamp(max=512))
        held = slice(off[0], off[-1])
        check(y[held], ref[held], tol16(ref, A, K, FP32)[held])
        assert (y[:off[0]] == 2.0).all() and (y[off[-1]:] == 2.0).all()


FIRST_CALLS_CAPTURED = """
import sys
import torch
from fp4_block_scaled_route_b200 import moe
x, w = torch.randn(300, 2056, device="cuda").bfloat16(), torch.randn(3, 264, 2056, device="cuda").bfloat16()
off = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device="cuda")
perm = torch.arange(300, dtype=torch.int32, device="cuda")
g = torch.rand(150, 2, device="cuda")
w8, c = torch.ones(264, 2064, dtype=torch.int8, device="cuda"), torch.ones(264, device="cuda")
def step():
    y = moe.grouped_gemm(x, w, off)
    q, s = moe.quant_int8(x)
    return (y, moe.grouped_gemm_dgrad(y, w, off), moe.grouped_gemm_wgrad(y, x, off), moe.permute(x, perm, 1),
            moe.combine(y, perm, g), *moe.combine_backward(y[:150], y, perm, g),
            moe.int8_gemm(q, s, w8[:, :2056], c))
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
sys.exit(0 if all(torch.equal(a, b) for a, b in zip(out, step())) else 1)
"""


def test_first_calls_of_a_process_are_captured():
    """Nothing that a first call sets up is refused while a stream is being captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_int8_strides_and_rows_outside():
    counts = [3, 0, 40]
    off = offsets_of(counts, 2)
    P, N, K = 50, 72, 144
    gen = torch.Generator("cuda").manual_seed(9)
    big = torch.randint(-128, 128, (P, K + 32), generator=gen, device="cuda", dtype=torch.int8)
    wj = torch.randint(-128, 128, (3, 2 * N, K + 16), generator=gen, device="cuda", dtype=torch.int8)
    q, w = big[:, 16:16 + K], wj[:, :N, :K]
    s, c = torch.rand(P, generator=gen, device="cuda"), torch.rand(3, N, generator=gen, device="cuda")
    s[0] = float("nan")
    y = torch.full((P, N + 8), 2.0, dtype=FP32, device="cuda")
    moe.int8_gemm(q, s, w, c, offsets=off, out=y[:, :N])
    ref = int8_64(q, s, w, c, off)
    check_int8(y[2:45, :N], ref[2:45], FP32)
    assert (y[:2] == 2.0).all() and (y[45:] == 2.0).all() and (y[:, N:] == 2.0).all()
