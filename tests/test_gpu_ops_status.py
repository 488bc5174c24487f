"""GPU tests of the errors that the expert operators find on the device, in
calls without a status word of their own."""
import subprocess
import sys
import os

import pytest
import torch

from fp4_block_scaled_route_b200 import moe

pytestmark = pytest.mark.gpu

E, N, K, P = 3, 16, 64, 10


def make(off):
    ones = torch.ones
    return (ones(P, K, device="cuda").bfloat16(), ones(P, N, device="cuda").bfloat16(), ones(E, N, K, device="cuda").bfloat16(),
            torch.tensor(off, dtype=torch.int32, device="cuda"))


def calls(x, dy, w, off, **kw):
    q, s = moe.quant_int8(x)
    return {"product": lambda: moe.grouped_gemm(x, w, off, **kw), "input_gradient": lambda: moe.grouped_gemm_dgrad(dy, w, off, **kw),
            "weight_gradient": lambda: moe.grouped_gemm_wgrad(dy, x, off, **kw),
            "int8": lambda: moe.int8_gemm(q, s, torch.ones_like(w, dtype=torch.int8), torch.ones(E, N, device="cuda"), offsets=off, **kw)}


@pytest.mark.parametrize("name", ["product", "input_gradient", "weight_gradient", "int8"])
def test_unusable_offsets_are_told_once(name):
    moe.ops_status()
    calls(*make([0, 3, 3, 10]))[name]()
    assert moe.ops_status() == moe.MOE_OK
    calls(*make([0, 5, 4, 10]))[name]()
    assert moe.ops_status() == moe.MOE_ERR_BAD_ROUTING
    assert moe.ops_status() == moe.MOE_OK


def test_a_callers_word_takes_the_errors_of_its_calls():
    moe.ops_status()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for f in calls(*make([0, 5, 8, 11]), status=status).values():
        f()
    assert int(status) == 1 and moe.ops_status() == moe.MOE_OK


def test_errors_of_other_streams_and_of_replays():
    moe.ops_status()
    args = make([0, 3, 3, 10])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(*make([-1, 3, 3, 10]))["product"]()
    assert moe.ops_status(side) == moe.MOE_ERR_BAD_ROUTING
    calls(*args)["product"]()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls(*args)["product"]()
    graph.replay()
    assert moe.ops_status() == moe.MOE_OK and bool((out == K).all())
    args[3].copy_(torch.tensor([0, 9, 3, 10]))
    graph.replay()
    assert moe.ops_status() == moe.MOE_ERR_BAD_ROUTING
    assert moe.ops_status() == moe.MOE_OK


FIRST_CALL_CAPTURED = """
import torch
from fp4_block_scaled_route_b200 import moe
x, w = torch.ones(10, 64, device="cuda").bfloat16(), torch.ones(3, 16, 64, device="cuda").bfloat16()
off = torch.tensor([0, 5, 4, 10], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    moe.grouped_gemm(x, w, off)
graph.replay()
assert moe.ops_status() == moe.MOE_ERR_BAD_ROUTING and moe.ops_status() == moe.MOE_OK
"""


def test_first_call_of_a_process_is_captured():
    """The device's word is found while a stream is being captured."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
