"""GPU tests of the expert operators used together: route, permute, grouped
products, combine, and the way back; and the int8 experts between the same
routing steps.

Tolerances: every operator rounds its output to bf16 once.  bf16 keeps 8
significant bits, so neighbours are 2^-7 of the lower power of two apart and a
rounding is off by at most half of that, 2^-8 of the value; the layer is a chain of them, so an output is off by the sum over the
steps of 2^-8 times the magnitudes that pass through the step (computed in
fp64 from absolute values), and the elementwise steps between the products,
done by torch in bf16, add one such rounding each."""
import pytest
import torch

from fp4_block_scaled_route_b200 import moe

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
U = torch.finfo(BF16).eps / 2 * 1.05   # 2^-8, with room for the fp32 sums (2^-23 * length)


def layer64(x, w13, w2, ids, g):
    """The layer in fp64 autograd from its definition, and its magnitudes (every term's absolute value)."""
    T, H = x.shape
    I = w2.shape[2]
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    for j in range(ids.shape[1]):
        for e in ids[:, j].unique().tolist():
            t = (ids[:, j] == e).nonzero().flatten()
            h = x[t] @ w13[e].T
            a = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
            out = out.index_add(0, t, g[t, j, None] * (a @ w2[e].T))
            hm = x[t].detach().abs() @ w13[e].detach().abs().T
            # silu has slope at most 1.1 and |silu(v)| <= |v|
            am = 1.1 * hm[:, :I] * hm[:, I:]
            mag.index_add_(0, t, g[t, j, None].detach().abs() * (am @ w2[e].detach().abs().T))
    return out, mag


def inputs(T, H, I, E, k, seed, spread):
    gen = torch.Generator("cuda").manual_seed(seed)

    def rnd(*s, scale=1.0):
        return (torch.randn(*s, generator=gen, device="cuda") * scale).to(BF16)
    x = rnd(T, H)
    w13, w2 = rnd(E, 2 * I, H, scale=H ** -0.5), rnd(E, H, I, scale=I ** -0.5)
    score = torch.rand(T, E, generator=gen, device="cuda") + spread * torch.arange(E, device="cuda") / E
    ids = score.topk(k, dim=1).indices.int()
    g = torch.softmax(torch.randn(T, k, generator=gen, device="cuda"), 1)
    return x, w13, w2, ids, g, rnd(T, H)


@pytest.mark.parametrize("T,H,I,E,k,spread", [(1, 128, 128, 8, 2, 0.0), (33, 256, 128, 8, 2, 0.0),
                                              (150, 256, 384, 12, 3, 2.0), (700, 512, 128, 4, 2, 0.5)])
def test_bf16_layer_forward_and_backward(T, H, I, E, k, spread):
    x, w13, w2, ids, g, dout = inputs(T, H, I, E, k, T, spread)
    layer = moe.MoeLayer(H, I, E, k, max_T=T)
    counts, off, perm, inv = layer.route(ids)

    xp = moe.permute(x, perm, k)
    h = moe.grouped_gemm(xp, w13, off)
    gate, up = h[:, :I], h[:, I:]
    act = torch.nn.functional.silu(gate) * up
    y = moe.grouped_gemm(act, w2, off)
    out = moe.combine(y, inv, g)

    dy, dg = moe.combine_backward(dout, y, inv, g)
    dact = moe.grouped_gemm_dgrad(dy, w2, off)
    dw2 = moe.grouped_gemm_wgrad(dy, act, off)
    sg = torch.sigmoid(gate.float())
    dh = torch.empty_like(h)
    dh[:, :I] = (dact.float() * up.float() * sg * (1 + gate.float() * (1 - sg))).to(BF16)
    dh[:, I:] = (dact.float() * gate.float() * sg).to(BF16)
    dxp = moe.grouped_gemm_dgrad(dh, w13, off)
    dw13 = moe.grouped_gemm_wgrad(dh, xp, off)
    dx = moe.combine(dxp, inv, k=k)
    assert layer.device_status() == moe.MOE_OK
    layer.close()

    leaves = [t.double().requires_grad_() for t in (x, w13, w2)] + [g.double().requires_grad_()]
    ref, mag = layer64(*leaves[:3], ids, leaves[3])
    ref.backward(dout.double())
    # x -> h, act (two elementwise roundings), y, out: five roundings of what mag bounds
    assert ((out.double() - ref).abs() <= 6 * U * mag + 1e-30).all()
    # the gradients pass through at most as many rounded steps each way; their own magnitudes vary by element, so
    # they are held to the same relative error in the 2-norm, where independent roundings add in squares
    for got, leaf in zip((dx, dw13, dw2, dg), (leaves[0], leaves[1], leaves[2], leaves[3])):
        assert ((got.double() - leaf.grad).norm() <= 8 * U * leaf.grad.norm()).all()


@pytest.mark.parametrize("T,H,I,E,k,spread", [(1, 128, 128, 8, 2, 0.0), (90, 256, 384, 12, 3, 2.0)])
def test_int8_layer(T, H, I, E, k, spread):
    x, w13, w2, ids, g, _ = inputs(T, H, I, E, k, T + 1, spread)

    def channels(w):
        c = w.float().abs().amax(2) / 127
        return (w.float() / c[..., None]).round().to(torch.int8), c
    q13, c13 = channels(w13)
    q2, c2 = channels(w2)
    layer = moe.MoeLayer(H, I, E, k, max_T=T)
    _, off, perm, inv = layer.route(ids)
    q, s = moe.quant_int8(x, perm=perm, k=k)
    h = moe.int8_gemm(q, s, q13, c13, offsets=off)
    act = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
    qa, sa = moe.quant_int8(act)
    y = moe.int8_gemm(qa, sa, q2, c2, offsets=off)
    out = moe.combine(y, inv, g)
    layer.close()
    # the same chain from the definitions in fp64, on the operators' own rounded inputs of each step
    grp = torch.repeat_interleave(torch.arange(E, device="cuda"), off.diff().long())
    h64 = torch.einsum("pk,pnk->pn", q.double(), q13[grp].double()) * s.double()[:, None] * c13[grp].double()
    assert bool(((h.double() - h64).abs() <= U * h64.abs()).all())
    y64 = torch.einsum("pk,pnk->pn", qa.double(), q2[grp].double()) * sa.double()[:, None] * c2[grp].double()
    assert ((y.double() - y64).abs() <= U * y64.abs()).all()
    o64 = (g.double()[..., None] * y[inv.long()].double().view(T, k, H)).sum(1)
    bound = U * o64.abs() + (k + 2) * 2.0 ** -24 * (g.double()[..., None] * y[inv.long()].double().view(T, k, H).abs()).sum(1)
    assert ((out.double() - o64).abs() <= bound).all()
    # and against the unquantised layer: 8-bit rounding of rows and weights, a few percent in the 2-norm
    ref, _ = layer64(x.double(), w13.double(), w2.double(), ids, g.double())
    assert (out.double() - ref).norm() <= 0.05 * ref.norm()
    assert torch.equal(moe.int8_gemm(q, s, q13, c13, offsets=off), h)   # integer sums: bit for bit again


def test_the_whole_step_in_one_graph():
    """Route to combine captured once, replayed with new tokens and routings."""
    T, H, I, E, k = 24, 256, 128, 8, 2
    x, w13, w2, ids, g, dout = inputs(T, H, I, E, k, 5, 0.0)
    layer = moe.MoeLayer(H, I, E, k, max_T=T)

    def step():
        _, off, perm, inv = layer.route(ids)
        xp = moe.permute(x, perm, k)
        h = moe.grouped_gemm(xp, w13, off)
        y = moe.grouped_gemm(torch.nn.functional.silu(h[:, :I]) * h[:, I:], w2, off)
        dy, dg = moe.combine_backward(dout, y, inv, g)
        return moe.combine(y, inv, g), dg, moe.grouped_gemm_wgrad(dy, xp, off)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (11, 12):
        new = inputs(T, H, I, E, k, seed, 1.0)
        for old, v in zip((x, ids, g, dout), (new[0], new[3], new[4], new[5])):
            old.copy_(v)
        graph.replay()
        got = [t.clone() for t in captured]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    layer.close()
