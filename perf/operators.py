"""Cases of the expert operators: ragged grouped products with their gradients,
8-bit integer products with token and channel scales, and the row movement
between token order and expert order.

Each case names an operator (``op``), its sizes and its types.  ``run`` computes
it from elementary torch operations, or, with ``own`` set, through
``fp4_block_scaled_route_b200.moe``.  Rows are routed: T tokens choose k of E
experts, and the P = T * k chosen slots are sorted by expert (position p holds
slot ``perm[p]`` = t * k + j, ``inv`` is the inverse, expert e owns positions
``offsets[e] .. offsets[e + 1] - 1``).

==================  =====================================================
product             y[p] = x[p] W_e^T             x [P, K], W [E, N, K]
input_gradient      dx[p] = dy[p] W_e             dy [P, N]
weight_gradient     dW_e = sum_p dy[p]^T x[p]     over the rows p of e
int8                s[t] = amax|x[t]| / 127, q = round(127 x / amax),
                    y[p, n] = s[p] c[e, n] sum_k q[p, k] w[e, n, k]
                    (E = 0: one matrix for all rows, in token order)
permute             xp[p] = x[perm[p] / k]
combine             out[t] = sum_j g[t, j] y[inv[t, j]]
combine_gradient    dy[inv[t, j]] = g[t, j] dout[t],
                    dg[t, j] = sum_h dout[t, h] y[inv[t, j], h]
==================  =====================================================
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
PRODUCTS = ("product", "input_gradient", "weight_gradient")
ROWS = ("permute", "combine", "combine_gradient")


def listed():
    return [
        # one decode step of a small layer: a handful of rows over eight experts, all latency
        dict(name="product_tiny", op="product", T=4, k=2, E=8, N=128, K=256, type="fp16", out="fp16", routing="uniform"),
        # the down projection of a decode batch over many experts: one or two rows each, the weights' stream is the cost
        dict(name="product_decode", op="product", T=32, k=8, E=256, N=7168, K=2048, type="bf16", out="bf16", routing="uniform"),
        # gate and up projection of a prefill or training batch with popular and rare experts: bound by the tensor cores
        dict(name="product_prefill", op="product", T=4096, k=8, E=32, N=4096, K=7168, type="bf16", out="bf16", routing="zipf"),
        # backward of the same projection for a smaller batch whose rows fill no whole tiles
        dict(name="input_gradient", op="input_gradient", T=1000, k=6, E=32, N=4096, K=7168, type="fp16", out="fp16", routing="zipf"),
        # weight gradients of a training step, kept in the weights' type
        dict(name="weight_gradient", op="weight_gradient", T=2048, k=8, E=32, N=2048, K=7168, type="bf16", out="bf16", routing="uniform"),
        # weight gradients in fp32 of a small layer with odd sizes, some experts with few rows or none
        dict(name="weight_gradient_odd", op="weight_gradient", T=250, k=4, E=64, N=392, K=1032, type="fp16", out="fp32", routing="zipf"),
        # a dense layer in 8 bits while decoding a few sequences: one pass over its weights
        dict(name="int8_decode", op="int8", T=5, k=1, E=0, N=4096, K=7168, type="bf16", out="bf16", routing="uniform"),
        # the same kind of layer on a long prompt
        dict(name="int8_prefill", op="int8", T=4096, k=1, E=0, N=7168, K=2048, type="bf16", out="bf16", routing="uniform"),
        # experts in 8 bits for a decode batch, rows quantised while they are brought into expert order
        dict(name="int8_experts", op="int8", T=128, k=8, E=64, N=2048, K=7168, type="fp16", out="fp16", routing="uniform"),
        # a prompt's tokens into expert order
        dict(name="permute", op="permute", T=4096, k=8, E=32, K=7168, type="bf16", out="bf16", routing="zipf"),
        # the weighted sum of a prompt's expert outputs
        dict(name="combine", op="combine", T=4096, k=8, E=32, K=7168, type="bf16", out="bf16", routing="zipf"),
        # its gradients, for a training batch of odd length
        dict(name="combine_gradient", op="combine_gradient", T=1333, k=6, E=32, K=4096, type="fp16", out="fp16", routing="zipf"),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(PRODUCTS + PRODUCTS + ("int8", "int8") + ROWS)
    typ = rng.choice(("bf16", "fp16"))
    out = rng.choice((typ, typ, "fp32")) if op in PRODUCTS + ("int8",) else typ
    E = _spread(rng, 1, 256)
    if op == "int8" and rng.random() < 0.5:
        E = 0
    k = rng.randint(1, min(8, E)) if E else 1
    case = dict(op=op, T=_spread(rng, 1, 4096), k=k, E=E)
    if op in ROWS:
        case["K"] = _spread(rng, 128, 7168, 8)
    else:
        case["N"] = _spread(rng, 64, 7168, 8)
        case["K"] = _spread(rng, 64, 7168, 16 if op == "int8" else 8)
        # the weights of a whole layer stay below 2 Gi elements, the padded plain form below the largest listed case
        while max(E, 1) * case["N"] * case["K"] > 1 << 30:
            case["N"] = max(64, case["N"] // 16 * 8)
        cap = 1 << (38 if op == "int8" else 39)
        while case["T"] > 1 and case["T"] * max(E, 1) * case["N"] * case["K"] > cap:
            case["T"] = max(1, case["T"] // 2)
    case.update(type=typ, out=out, routing=rng.choice(("uniform", "zipf")))
    return case


def _popularity(case):
    """log popularity of the experts: flat, or falling as rank^-1."""
    E = case["E"]
    return [0.0 if case["routing"] == "uniform" else -math.log(1.0 + e) for e in range(E)]


def _touched(case):
    """Experts that get a row, as expected over routings."""
    w = [math.exp(v) for v in _popularity(case)]
    total = sum(w)
    return sum(1.0 - (1.0 - min(1.0, case["k"] * v / total)) ** case["T"] for v in w)


def work(case):
    T, k, E, K = case["T"], case["k"], case["E"], case["K"]
    P, i, o = T * k, SIZE[case["type"]], SIZE[case["out"]]
    op = case["op"]
    if op == "permute":
        return {"bytes": T * K * i + P * K * o + 4 * P, "flops": 0}
    if op == "combine":
        return {"bytes": P * K * i + T * K * o + 8 * P, "flops": 2 * P * K}
    if op == "combine_gradient":
        return {"bytes": T * K * i + 2 * P * K * i + 12 * P, "flops": 3 * P * K}
    N = case["N"]
    flops = 2 * P * N * K
    used = max(1.0, _touched(case)) if E else 1.0
    if op == "int8":
        return {"bytes": int(T * K * i + used * N * (K + 4) + P * N * o), "flops": flops}
    if op == "product":
        return {"bytes": int(P * K * i + used * N * K * i + P * N * o), "flops": flops}
    if op == "input_gradient":
        return {"bytes": int(P * N * i + used * N * K * i + P * K * o), "flops": flops}
    return {"bytes": P * (N + K) * i + E * N * K * o, "flops": flops}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    T, k, E, K = case["T"], case["k"], case["E"], case["K"]
    P, typ, op = T * k, TYPES[case["type"]], case["op"]
    state = dict(case=case, T=T, k=k, P=P, out=TYPES[case["out"]], offsets=None, perm=None, most=P)

    def normal(*shape, scale=1.0):
        # in the type itself: a layer's weights in fp32 would take twice the memory for a moment
        return torch.randn(*shape, generator=gen, device=dev, dtype=typ).mul_(scale)

    if E:
        noise = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device=dev).clamp(1e-9, 1 - 1e-7)))
        order = torch.randperm(E, generator=gen, device=dev)
        ids = (noise + torch.tensor(_popularity(case), device=dev)[order]).topk(k, dim=1).indices
        flat, perm = ids.flatten().sort(stable=True)
        inv = torch.empty_like(perm)
        inv[perm] = torch.arange(P, device=dev)
        counts = torch.zeros(E, dtype=torch.int64, device=dev).index_add_(0, flat, torch.ones_like(flat))
        offsets = torch.zeros(E + 1, dtype=torch.int64, device=dev)
        offsets[1:] = counts.cumsum(0)
        state.update(offsets=offsets.int(), perm=perm.int(), inv=inv.int().view(T, k), most=int(counts.max()),
                     used=counts.nonzero().flatten())
    if op in ROWS:
        logits = torch.randn(T, k, generator=gen, device=dev)
        state.update(g=torch.softmax(logits, 1).contiguous(), x=normal(T, K))
        if op != "permute":
            state["y"] = normal(P, K)
        return state
    N = case["N"]
    if op == "int8":
        # a few channels of the activations are far larger than the rest, as they are behind a norm
        loud = torch.where(torch.rand(K, generator=gen, device=dev) < 0.01, 12.0, 1.0).to(typ)
        state["x"] = normal(T, K) * loud
        w = torch.empty(max(E, 1), N, K, dtype=torch.int8, device=dev)
        for e in range(max(E, 1)):
            w[e] = torch.randn(N, K, generator=gen, device=dev, dtype=torch.bfloat16).mul_(34.0).round_().clamp_(-127, 127)
        state["w"] = w
        state["c"] = torch.exp(0.3 * torch.randn(max(E, 1), N, generator=gen, device=dev)) / (34.0 * math.sqrt(K))
        return state
    if op == "product":
        state["x"] = normal(P, K)
    elif op == "input_gradient":
        state["dy"] = normal(P, N)
    else:
        state["x"], state["dy"] = normal(P, K), normal(P, N)
    if op != "weight_gradient":
        state["w"] = normal(E, N, K, scale=1.0 / math.sqrt(K if op == "product" else N))
    return state


def _padded(state, experts=None):
    """Rows of each expert as a rectangle [experts, most], and which of its entries are rows."""
    off = state["offsets"].long()
    lo, hi = off[:-1], off[1:]
    if experts is not None:
        lo, hi = lo[experts], hi[experts]
    rows = lo[:, None] + torch.arange(state["most"], device=off.device)
    held = rows < hi[:, None]
    return rows.clamp(max=state["P"] - 1), held


def _plain_product(state, left, right, out_cols):
    """left rows [P, .] times each used expert's right [., out_cols], in 32 bits."""
    rows, held = _padded(state, state["used"])
    y = torch.bmm(left.float()[rows], right)
    result = torch.zeros(state["P"], out_cols, dtype=state["out"], device=left.device)
    result[rows[held]] = y[held].to(state["out"])
    return result


def _plain(state):
    op, k = state["case"]["op"], state["k"]
    if op == "product":
        w = state["w"][state["used"]].float()
        return _plain_product(state, state["x"], w.transpose(1, 2), w.shape[1])
    if op == "input_gradient":
        w = state["w"][state["used"]].float()
        return _plain_product(state, state["dy"], w, w.shape[2])
    if op == "weight_gradient":
        rows, held = _padded(state)
        dy = state["dy"].float()[rows] * held[..., None]
        return torch.bmm(dy.transpose(1, 2), state["x"].float()[rows]).to(state["out"])
    if op == "int8":
        x = state["x"].float()
        amax = x.abs().amax(1, keepdim=True)
        q = torch.round(x * 127.0 / amax.where(amax > 0, 1.0))
        s = torch.where(amax > 0, amax / 127.0, 1.0)
        # the integer sums pass 2^24, so they are taken in 64 bits
        if state["offsets"] is None:
            sums = q.double() @ state["w"][0].double().T
            return (sums * s * state["c"][0]).to(state["out"])
        rows, held = _padded(state, state["used"])
        token = state["perm"].long()[rows] // k
        sums = torch.bmm(q.double()[token], state["w"][state["used"]].double().transpose(1, 2))
        y = sums * s[token] * state["c"][state["used"]][:, None]
        result = torch.zeros(state["P"], sums.shape[2], dtype=state["out"], device=x.device)
        result[rows[held]] = y[held].to(state["out"])
        return result
    if op == "permute":
        return state["x"][state["perm"].long() // k]
    at = state["inv"].long()
    if op == "combine":
        return (state["y"][at].float() * state["g"][..., None]).sum(1).to(state["out"])
    # the tokens' rows are the gradient of the combined output here
    dout = state["x"].float()[:, None]
    dy = torch.empty_like(state["y"])
    dy[at.flatten()] = (dout * state["g"][..., None]).to(state["out"]).flatten(0, 1)
    return {"dy": dy, "dg": (dout * state["y"][at].float()).sum(2)}


def _framework(state):
    from fp4_block_scaled_route_b200 import moe
    op, out = state["case"]["op"], state["out"]
    if op == "product":
        return moe.grouped_gemm(state["x"], state["w"], state["offsets"], out_dtype=out)
    if op == "input_gradient":
        return moe.grouped_gemm_dgrad(state["dy"], state["w"], state["offsets"], out_dtype=out)
    if op == "weight_gradient":
        return moe.grouped_gemm_wgrad(state["dy"], state["x"], state["offsets"], out_dtype=out)
    if op == "int8":
        q, s = moe.quant_int8(state["x"], perm=state["perm"], k=state["k"])
        return moe.int8_gemm(q, s, state["w"], state["c"], offsets=state["offsets"], out_dtype=out)
    if op == "permute":
        return moe.permute(state["x"], state["perm"], state["k"])
    if op == "combine":
        return moe.combine(state["y"], state["inv"], state["g"])
    dy, dg = moe.combine_backward(state["x"], state["y"], state["inv"], state["g"])
    return {"dy": dy, "dg": dg}


def run(state):
    return _framework(state) if own else _plain(state)


def exact(case, seed):
    """The definitions in 64 bits, expert by expert and slot by slot."""
    state = prepare(case, seed)
    op, T, k, E = case["op"], case["T"], case["k"], case["E"]
    off = state["offsets"].tolist() if E else [0, T]
    spans = [(e, slice(off[e], off[e + 1])) for e in range(len(off) - 1) if off[e + 1] > off[e]]
    dev = state["w"].device if "w" in state else state["x"].device
    slot = state["perm"].long() if E else torch.arange(T, device=dev)
    if op == "product":
        y = torch.zeros(T * k, case["N"], dtype=torch.float64, device=dev)
        for e, rows in spans:
            y[rows] = torch.einsum("pk,nk->pn", state["x"][rows].double(), state["w"][e].double())
        return y
    if op == "input_gradient":
        dx = torch.zeros(T * k, case["K"], dtype=torch.float64, device=dev)
        for e, rows in spans:
            dx[rows] = torch.einsum("pn,nk->pk", state["dy"][rows].double(), state["w"][e].double())
        return dx
    if op == "weight_gradient":
        dw = torch.zeros(E, case["N"], case["K"], dtype=torch.float64, device=dev)
        for e, rows in spans:
            dw[e] = torch.einsum("pn,pk->nk", state["dy"][rows].double(), state["x"][rows].double())
        return dw
    if op == "int8":
        y = torch.zeros(T * k, case["N"], dtype=torch.float64, device=dev)
        for e, rows in spans:
            x = state["x"][slot[rows] // k].double()
            top = x.abs().max(dim=1).values
            q = torch.where(top[:, None] > 0, (127.0 * x) / top.clamp(min=1e-300)[:, None], 0.0).round()
            unit = torch.where(top > 0, top / 127.0, 1.0)
            y[rows] = torch.einsum("pk,nk->pn", q, state["w"][e].double()) * torch.outer(unit, state["c"][e].double())
        return y
    if op == "permute":
        return state["x"].double().index_select(0, slot // k)
    y, g = state["y"], state["g"].double()
    where = torch.empty(T * k, dtype=torch.int64, device=dev)
    where[slot] = torch.arange(T * k, device=dev)
    where = where.view(T, k)
    if op == "combine":
        out = torch.zeros(T, case["K"], dtype=torch.float64, device=dev)
        for j in range(k):
            out += g[:, j, None] * y[where[:, j]].double()
        return out
    dout = state["x"].double()
    dy = torch.zeros(T * k, case["K"], dtype=torch.float64, device=dev)
    dg = torch.zeros(T, k, dtype=torch.float64, device=dev)
    for j in range(k):
        dy[where[:, j]] = g[:, j, None] * dout
        dg[:, j] = torch.einsum("th,th->t", dout, y[where[:, j]].double())
    return {"dy": dy, "dg": dg}
