"""GPU tests of the row movement (moe_route, moe_permute, moe_combine and its
gradients) and of moe_quant_int8 against their definitions.

Tolerances: permute and the quantised codes are exact.  A combined value is
k + 1 fused multiply-adds in fp32 (2^-24 of a partial sum each, bounded by
the sum of magnitudes) and one rounding to the output type; a weight gradient
is a sum of H products in fp32, at most H additions and one rounding per
product.
"""
import numpy as np
import pytest
import torch

from fp4_block_scaled_route_b200 import moe

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=["bf16", "fp16", "fp32"])
TINY = {BF16: 2.0 ** -133, FP16: 2.0 ** -24, FP32: 2.0 ** -149}


def route_numpy(ids, E, n_shared=0):
    """(counts, offsets, perm, inv) of ids [T, k]; ids outside [0, E) drop their slot."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    S = T * k
    held = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(held, flat, E), kind="stable")[: held.sum()]
    counts = np.bincount(flat[held], minlength=E)
    if n_shared:
        counts = np.append(counts, T)
        order = np.concatenate([order, S + np.arange(T)])
    P = S + n_shared * T
    perm = np.full(P, -1)
    perm[: len(order)] = order
    inv = np.full(P, -1)
    inv[order] = np.arange(len(order))
    return counts, np.concatenate([[0], np.cumsum(counts)]), perm, inv


def make(T, k, E, n_shared=0, drop=False, seed=0):
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    if drop:
        ids[rng.random((T, k)) < 0.3] = -1
        ids[0] = E  # a token all of whose slots are dropped
    arrays = [torch.tensor(a, dtype=torch.int32, device="cuda") for a in route_numpy(ids, E, n_shared)]
    return ids, arrays


@pytest.mark.parametrize("T,k,E,n_shared", [(1, 1, 1, 0), (5, 2, 8, 0), (70, 8, 64, 1), (300, 4, 160, 0),
                                            (1100, 8, 32, 1)])
@pytest.mark.parametrize("drop", [False, True], ids=["all", "dropped"])
def test_route(T, k, E, n_shared, drop):
    ids, ref = make(T, k, E, n_shared, drop, seed=T)
    layer = moe.MoeLayer(256, 128, E, k, max_T=max(T, 4), n_shared=n_shared)
    got = layer.route(torch.tensor(ids, device="cuda"))
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    st = layer.device_status()
    assert st == (moe.MOE_ERR_BAD_ROUTING if drop else moe.MOE_OK)
    counts, offsets, perm, inv = layer.route(torch.empty(0, k, dtype=torch.int32, device="cuda"))
    assert not counts.any() and not offsets.any() and perm.numel() == inv.numel() == 0
    layer.close()


def test_route_leaves_the_last_forwards_record():
    from fp4_block_scaled_route_b200 import synth
    cfg = synth.CONFIGS[0]
    L = synth.make_layer(cfg, 3, device="cuda")
    layer = moe.MoeLayer(L.H, L.I, L.E, L.k, L.wfmt, max_T=L.T)
    out = layer.forward(L.x, L.ids, L.topk_w, L.w13, L.s13, L.w2, L.s2)
    before = layer.routing(L.T)
    layer.route((L.ids + 1) % L.E)
    for a, b in zip(before, layer.routing(L.T)):
        assert np.array_equal(a, b)
    again = layer.forward(L.x, L.ids, L.topk_w, L.w13, L.s13, L.w2, L.s2)
    torch.cuda.synchronize()
    assert torch.allclose(out.float(), again.float(), rtol=2e-2, atol=1e-3)
    layer.close()


SHAPES = pytest.mark.parametrize("T,k,E,H,n_shared", [(1, 1, 1, 8, 0), (3, 2, 4, 136, 1), (40, 8, 16, 264, 0),
                                                      (9, 32, 40, 72, 1), (200, 3, 8, 1032, 1), (5, 4, 8, 7168, 0)])


@TYPES
@SHAPES
@pytest.mark.parametrize("drop", [False, True], ids=["all", "dropped"])
def test_permute_and_combine(dtype, T, k, E, H, n_shared, drop):
    _, (counts, offsets, perm, inv) = make(T, k, E, n_shared, drop, seed=T + H)
    gen = torch.Generator("cuda").manual_seed(H)
    x = torch.randn(T, H, generator=gen, device="cuda").to(dtype)
    P, held = perm.numel(), int(offsets[-1])
    xp = torch.full((P, H), 5.0, dtype=dtype, device="cuda")
    moe.permute(x, perm, k, out=xp)
    slot = perm.long()
    token = torch.where(slot < T * k, slot // k, slot - T * k)
    assert torch.equal(xp[:held], x[token[:held]])
    assert (xp[held:] == 5.0).all()

    y = torch.randn(P, H, generator=gen, device="cuda").to(dtype)
    y[held:] = float("nan")   # rows no slot names
    g = torch.randn(T, k, generator=gen, device="cuda")
    eps = torch.finfo(dtype).eps / 2
    for gw in (g, None):
        out = moe.combine(y, inv, gw, k=k, n_shared=n_shared)
        ref = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        A = torch.zeros_like(ref)
        for j in range(k + n_shared):
            at = inv[:T * k].view(T, k)[:, j].long() if j < k else inv[T * k:].long()
            wt = torch.ones(T, device="cuda") if (gw is None or j >= k) else gw[:, j]
            term = torch.where((at >= 0)[:, None], wt.double()[:, None] * y[at.clamp(min=0)].double(), 0.0)
            ref += term
            A += term.abs()
        assert ((out.double() - ref).abs() <= eps * ref.abs() + (k + 2) * 2.0 ** -24 * A * 1.01 + TINY[dtype]).all()


@TYPES
@SHAPES
@pytest.mark.parametrize("drop", [False, True], ids=["all", "dropped"])
def test_combine_backward(dtype, T, k, E, H, n_shared, drop):
    _, (counts, offsets, perm, inv) = make(T, k, E, n_shared, drop, seed=T + H)
    gen = torch.Generator("cuda").manual_seed(H)
    P, held = perm.numel(), int(offsets[-1])
    dout = torch.randn(T, H, generator=gen, device="cuda").to(dtype)
    y = torch.randn(P, H, generator=gen, device="cuda").to(dtype)
    y[held:] = float("nan")
    g = torch.randn(T, k, generator=gen, device="cuda")
    dy = torch.full((P, H), 5.0, dtype=dtype, device="cuda")
    _, dg = moe.combine_backward(dout, y, inv, g, n_shared=n_shared, dy=dy)
    assert (dy[held:] == 5.0).all()
    eps = torch.finfo(dtype).eps / 2
    for j in range(k + n_shared):
        at = inv[:T * k].view(T, k)[:, j].long() if j < k else inv[T * k:].long()
        ok = at >= 0
        ref = dout.double() * (g[:, j].double()[:, None] if j < k else 1.0)
        got = dy[at.clamp(min=0)].double()
        # one product rounded to fp32, then to the type
        assert ((got - ref).abs() <= (eps + 2.0 ** -24) * 1.01 * ref.abs() + TINY[dtype])[ok].all()
        if j < k:
            terms = torch.where(ok[:, None], dout.double() * y[at.clamp(min=0)].double(), 0.0)
            tol = (H + 1) * 2.0 ** -24 * terms.abs().sum(1) * 1.01
            assert ((dg[:, j].double() - terms.sum(1)).abs() <= tol).all()
            assert not dg[:, j][~ok].any()


def test_combine_gradients_against_differences():
    """combine is linear in y and in the weights, so central differences of it in fp64 are its gradients."""
    T, k, E, H = 6, 3, 5, 40
    _, (_, offsets, perm, inv) = make(T, k, E, drop=True, seed=3)
    gen = torch.Generator("cuda").manual_seed(9)
    y, dout = torch.randn(T * k, H, generator=gen, device="cuda"), torch.randn(T, H, generator=gen, device="cuda")
    g = torch.randn(T, k, generator=gen, device="cuda")
    dy, dg = moe.combine_backward(dout, y, inv, g)
    at, ok = inv.view(T, k).long().clamp(min=0), (inv.view(T, k) >= 0).double()

    def loss(yy, gg):
        return ((gg * ok)[..., None] * yy[at]).sum(1).mul(dout.double()).sum()
    for p, h in ((0, 0), (3, 39), (int(offsets[-1]) - 1, 17)):
        d = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        d[p, h] = 0.5
        diff = float(loss(y.double() + d, g.double()) - loss(y.double() - d, g.double()))
        assert abs(float(dy[p, h]) - diff) <= 1e-5 * (1 + abs(diff))
    for t, j in ((0, 0), (2, 1), (5, 2)):
        d = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        d[t, j] = 0.5
        diff = float(loss(y.double(), g.double() + d) - loss(y.double(), g.double() - d))
        assert abs(float(dg[t, j]) - diff) <= 1e-5 * (1 + abs(diff))


@TYPES
def test_row_strides_and_odd_widths(dtype):
    T, k, E, H = 13, 3, 6, 37
    _, (_, _, perm, inv) = make(T, k, E, seed=1)
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(T, 64, generator=gen, device="cuda").to(dtype)[:, 8:8 + H]
    xp = torch.full((T * k, 48), 5.0, dtype=dtype, device="cuda")
    moe.permute(x, perm, k, out=xp[:, :H])
    assert torch.equal(xp[:, :H], x[perm.long() // k]) and (xp[:, H:] == 5.0).all()
    out = torch.full((T, 40), 5.0, dtype=dtype, device="cuda")
    moe.combine(xp[:, :H], inv, k=k, out=out[:, :H])
    # k equal terms
    assert ((out[:, :H].double() - k * x.double()).abs() <= torch.finfo(dtype).eps * k * x.double().abs()).all()
    assert (out[:, H:] == 5.0).all()
    g = torch.rand(T, k, generator=gen, device="cuda")
    dy = torch.full((T * k, 40), 5.0, dtype=dtype, device="cuda")
    moe.combine_backward(x, xp[:, :H], inv, g, dy=dy[:, :H])
    ref = x[perm.long() // k].double() * g.flatten()[perm.long()].double()[:, None]
    assert ((dy[:, :H].double() - ref).abs() <= torch.finfo(dtype).eps * ref.abs() + TINY[dtype]).all()
    assert (dy[:, H:] == 5.0).all()


def test_slots_outside_are_skipped():
    """Permutation entries that name no slot, and inverse entries that name no row, touch nothing."""
    T, k, H = 4, 2, 16
    x = torch.randn(T, H, device="cuda")
    perm = torch.tensor([0, -5, 8, 2 ** 31 - 1, 11, 12, 7], dtype=torch.int32, device="cuda")
    y = torch.full((7, H), 5.0, device="cuda")
    moe.permute(x, perm, k, out=y)
    assert torch.equal(y[0], x[0]) and torch.equal(y[2], x[0]) and torch.equal(y[4], x[3]) and torch.equal(y[6], x[3])
    assert (y[[1, 3, 5]] == 5.0).all()
    inv = torch.tensor([0, 7, -1, 2 ** 31 - 1, 6, -2 ** 31, 3, 1], dtype=torch.int32, device="cuda")
    y = torch.randn(7, H, device="cuda")
    out = moe.combine(y, inv, k=k)
    assert torch.equal(out[0], y[0]) and not out[1].any() and torch.equal(out[2], y[6])
    dy = torch.full((7, H), 5.0, device="cuda")
    _, dg = moe.combine_backward(x, y, inv, torch.ones(T, k, device="cuda"), dy=dy)
    assert torch.equal(dy[0], x[0]) and torch.equal(dy[6], x[2]) and torch.equal(dy[3], x[3]) and torch.equal(dy[1], x[3])
    assert (dy[[2, 4, 5]] == 5.0).all() and not dg.flatten()[[1, 2, 3, 5]].any()
    q = torch.full((7, H), 5, dtype=torch.int8, device="cuda")
    s = torch.full((7,), 5.0, device="cuda")
    moe.quant_int8(x.to(BF16), perm=perm, k=k, out=q, scale=s)
    assert (q[[1, 3, 5]] == 5).all() and (s[[1, 3, 5]] == 5.0).all() and torch.equal(q[0], q[2])


def test_the_same_row_twice():
    """combine may read a row for several slots, and permute a token for several rows."""
    y = torch.randn(3, 40, device="cuda")
    inv = torch.tensor([2, 2, 0, 2], dtype=torch.int32, device="cuda")
    g = torch.tensor([[0.5, 0.25], [2.0, -1.0]], device="cuda")
    out = moe.combine(y, inv, g)
    ref = torch.stack([0.75 * y[2].double(), 2 * y[0].double() - y[2].double()])
    assert ((out.double() - ref).abs() <= 4 * 2.0 ** -24 * (y[2].abs() + 2 * y[0].abs()).double()).all()
    perm = torch.tensor([5, 5, 4], dtype=torch.int32, device="cuda")
    assert torch.equal(moe.permute(y, perm, 2), y[[2, 2, 2]])


def test_infinite_weights_and_values_are_kept_apart():
    """A token's NaN or infinity reaches that token's output only."""
    T, k, H = 3, 2, 24
    y = torch.randn(T * k, H, device="cuda")
    y[1, 3] = float("inf")
    y[4, 5] = float("nan")
    inv = torch.arange(T * k, dtype=torch.int32, device="cuda")
    g = torch.rand(T, k, device="cuda") + 0.1
    out = moe.combine(y, inv, g)
    ref = (g[..., None].double() * y.view(T, k, H).double()).sum(1)
    assert torch.equal(torch.isnan(out), torch.isnan(ref)) and torch.equal(torch.isinf(out), torch.isinf(ref))
    fine = torch.isfinite(ref)
    assert torch.allclose(out.double()[fine], ref[fine], rtol=1e-6, atol=1e-6)


# ---- row quantisation -----------------------------------------------------------------
def quant64(x):
    """Codes and scales by the definition; every quotient 127 x / amax of 16-bit values is far from a tie unless it
    is one, so fp64 decides it exactly."""
    v = x.double()
    amax = v.abs().amax(1)
    q = torch.where(amax[:, None] > 0, 127.0 * v / amax.clamp(min=1e-300)[:, None], 0.0).round()
    s = torch.where(amax > 0, (amax / 127.0).float(), 1.0)
    return q.to(torch.int8), s


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("T,K", [(1, 1), (3, 16), (7, 72), (33, 1032), (5, 7168), (2, 20000), (600, 136)])
def test_quant_int8(dtype, T, K):
    gen = torch.Generator("cuda").manual_seed(T * 7 + K)
    ld = (K + 15) // 16 * 16
    x = torch.randn(T, ld, generator=gen, device="cuda").to(dtype)[:, :K]
    x[0] *= 1e-3
    x[-1, K // 2] = 60.0
    q = torch.full((T, ld), 99, dtype=torch.int8, device="cuda")
    _, s = moe.quant_int8(x, out=q[:, :K])
    rq, rs = quant64(x)
    assert torch.equal(q[:, :K], rq) and (q[:, K:] == 99).all()
    assert torch.equal(s, rs)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_quant_int8_every_quotient_near_a_tie(dtype):
    """Rows whose values run through every multiple of amax / 254: the ties themselves and their neighbours."""
    rows = []
    for top in (1.0, 127.0, 254.0, 1.9921875, 100.0, 3.0, 0.007):
        t = torch.tensor(top, dtype=dtype)
        n = torch.arange(-254, 255, dtype=torch.float64) * (float(t) / 254.0)
        v = n.to(dtype)
        bits = v.view(torch.int16)
        near = torch.stack([v, (bits + 1).view(dtype), (bits - 1).view(dtype)]).flatten()
        near = near[near.abs() <= float(t)][:1500]
        row = torch.zeros(1528, dtype=dtype)
        row[: near.numel()] = near
        row[-1] = t
        rows.append(row)
    x = torch.stack(rows).cuda()
    q, s = moe.quant_int8(x)
    rq, rs = quant64(x)
    assert torch.equal(q, rq) and torch.equal(s, rs)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_quant_int8_special_rows(dtype):
    x = torch.ones(7, 64, dtype=dtype, device="cuda")
    x[1] = 0.0
    x[2, 5] = float("inf")
    x[3, 63] = float("-inf")
    x[4, 0] = float("nan")
    x[5] = torch.finfo(dtype).smallest_normal / 4    # subnormal
    x[5, 1] = torch.finfo(dtype).smallest_normal / 2
    x[6] = torch.finfo(dtype).max
    x[6, 3] = -torch.finfo(dtype).max / 2
    q, s = moe.quant_int8(x)
    assert not q[1].any() and s[1] == 1.0
    assert not q[2:5].any() and torch.isnan(s[2:5]).all()
    rq, rs = quant64(x[[0, 1, 5, 6]])
    assert torch.equal(q[[0, 1, 5, 6]], rq) and torch.equal(s[[0, 1, 5, 6]], rs)


def test_quant_int8_in_expert_order():
    T, k, E, K = 37, 4, 8, 144
    _, (_, _, perm, _) = make(T, k, E, n_shared=1, drop=True, seed=5)
    x = torch.randn(T, K, device="cuda").to(BF16)
    q = torch.full((perm.numel(), K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((perm.numel(),), 9.0, device="cuda")
    moe.quant_int8(x, perm=perm, k=k, out=q, scale=s)
    rq, rs = quant64(x)
    slot = perm.long()
    held = slot >= 0
    token = torch.where(slot < T * k, slot // k, slot - T * k).clamp(min=0)
    assert torch.equal(q[held], rq[token][held]) and torch.equal(s[held], rs[token][held])
    assert (q[~held] == 99).all() and (s[~held] == 9.0).all()
