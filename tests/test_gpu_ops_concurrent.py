"""GPU tests of expert products that run beside each other: units handed out
at run time, contractions and groups of several segments, shared tiles.  Each
result equals the one computed alone, bit for bit."""
import numpy as np
import pytest
import torch

from fp4_block_scaled_route_b200 import moe

pytestmark = pytest.mark.gpu


def calls(seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def randn(*s, dtype):
        return torch.randn(*s, generator=gen, device="cuda").to(dtype)

    def offsets(counts):
        return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    many, long = [700, 3, 333, 0, 512, 1100], [20000, 0, 9000, 5]
    x, w, off = randn(sum(many), 2056, dtype=torch.bfloat16), randn(len(many), 1288, 2056, dtype=torch.bfloat16), offsets(many)
    x16, w16 = randn(200, 16400, dtype=torch.float16), randn(2, 2056, 16400, dtype=torch.float16)
    off16 = offsets([90, 110])
    a, b, off_long = randn(sum(long), 264, dtype=torch.float16), randn(sum(long), 520, dtype=torch.float16), offsets(long)
    return [lambda **k: moe.grouped_gemm(x, w, off, **k), lambda **k: moe.grouped_gemm(x, w, off, out_dtype=torch.float32, **k),
            lambda **k: moe.grouped_gemm(x16, w16, off16, **k), lambda **k: moe.grouped_gemm_wgrad(a, b, off_long, **k),
            lambda **k: moe.grouped_gemm_wgrad(a, b, off_long, out_dtype=torch.float32, **k)]


def test_on_three_streams_at_once():
    sets = [calls(s) for s in (1, 2, 3)]
    alone = [[f() for f in fs] for fs in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    moe.ops_status()
    for _ in range(6):
        got = [[] for _ in sets]
        for i in range(len(sets[0])):
            for fs, st, g in zip(sets, streams, got):
                g.append(fs[i](stream=st))
        torch.cuda.synchronize()
        for one, both in zip(alone, got):
            for p, q in zip(one, both):
                assert torch.equal(p, q)
    assert moe.ops_status() == moe.MOE_OK


def test_in_one_stream_back_to_back_and_replayed():
    """Each call starts before the one ahead of it in the stream is through."""
    fs = calls(4)
    alone = []
    for f in fs:
        alone.append(f())
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = [f() for f in fs for _ in range(2)]
    moe.ops_status()
    for _ in range(4):
        got = [f() for f in fs for _ in range(2)]
        graph.replay()
        torch.cuda.synchronize()
        for i, ref in enumerate(alone):
            for r in (got[2 * i], got[2 * i + 1], captured[2 * i], captured[2 * i + 1]):
                assert torch.equal(r, ref)
    assert moe.ops_status() == moe.MOE_OK
