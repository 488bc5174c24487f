"""Which way each shape of the GPU tests is tiled: the rules of grouped_tile
and Units, compiled for the host from the kernels' own source, at a B200's 148
SMs; and GPU cases for the ways that those shapes do not reach."""
import os
import subprocess

import numpy as np
import pytest
import torch

from tests.test_gpu_grouped import WAYS
from tests.test_grouped_units import CSRC, between

MAIN = r"""
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include "moe_ops.h"
#undef __device__
#undef __forceinline__
#define __device__
#define __forceinline__ inline
using std::max;
using std::min;
namespace moe {
%s
}
using namespace moe;
// kind, M, R, then the groups' rows -> rows of a tile, CTAs of an MMA, shares, handed out, cut
int main(int, char** v) {
  const int kind = atoi(v[1]);
  GroupedParams p{};
  p.M = atoi(v[2]);
  p.R = atoi(v[3]);
  for (char** a = v + 4; *a; ++a) {
    ++p.E;
    p.P += atoi(*a);
  }
  const GroupedTile t = grouped_tile(p, kind, 148);
  int tiles = 0;
  for (char** a = v + 4; *a; ++a) tiles += (atoi(*a) + t.rows - 1) / t.rows;
  const int NT = (p.M + 128 * t.ctas - 1) / (128 * t.ctas), teams = t.running / (t.ctas * t.split);
  int cut = 0;
  if (t.ctas == 2) cut = Units::make<256, 2>(tiles * NT, NT, teams).cut;
  if (t.split > 1 && t.grid < tiles * NT * t.split) return 1;  // a cluster has one tile
  if (t.grid > t.running && t.split == 1 && t.grid < 2 * Units::make<256, 2>(tiles * NT, NT, teams).total) return 1;
  printf("%%d %%d %%d %%d %%d\n", t.rows, t.ctas, t.split, t.ctas == 2 && t.grid > t.running, cut);
  return 0;
}
"""


@pytest.fixture(scope="module")
def way(tmp_path_factory):
    with open(os.path.join(CSRC, "moe_grouped.cu")) as f:
        g = f.read()
    parts = [between(g, "constexpr int kBand", "\n"), between(g, "constexpr int kSplitChunks", "struct Tile {"),
             between(g, "struct Units {", "// Unit u -> group"), between(g, "GroupedTile grouped_tile(", "template <int KIND>\nstatic")]
    d = tmp_path_factory.mktemp("ways")
    (d / "ways.cpp").write_text(MAIN % "\n".join(parts))
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", os.path.join(os.path.dirname(os.path.dirname(CSRC)), "include"),
                    "-I", cuda, "-o", str(d / "ways"), str(d / "ways.cpp")], check=True, timeout=120)

    def run(counts, M, R, kind=0):
        r = subprocess.run([str(d / "ways"), *map(str, (kind, M, R, *counts))], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, (counts, M, R)
        return tuple(map(int, r.stdout.split()))
    return run


# rows of a tile, CTAs of an MMA, CTAs that share its contraction, handed out at run time, last wave cut into 2^n pieces
TILED = {
    "rows16_split8": (16, 1, 8, 0, 0),
    "rows16_split8_at_most": (16, 1, 8, 0, 0),
    "rows16_split4": (16, 1, 4, 0, 0),
    "rows16_split2": (16, 1, 2, 0, 0),
    "rows32_split4": (32, 1, 4, 0, 0),
    "rows32_split2": (32, 1, 2, 0, 0),
    "rows64_split4": (64, 1, 4, 0, 0),
    "rows64_split2": (64, 1, 2, 0, 0),
    "rows64_few_large": (64, 1, 4, 0, 0),
    "rows64_short": (64, 1, 1, 0, 0),
    "rows64_many": (64, 1, 1, 0, 0),
    "rows64": (64, 1, 1, 0, 0),
    "rows64_two_tiles": (64, 1, 1, 0, 0),
    "pairs": (256, 2, 1, 0, 0),
    "pairs_pieces": (256, 2, 1, 0, 0),     # 48 tiles of 74 pairs: no piece, in spite of its name
    "pairs_handed_out": (256, 2, 1, 1, 3),
    "pairs_handed_out_few_units": (256, 2, 1, 1, 1),
}
# Rows of the groups, N, K, cut, handed out: pairs whose last wave is whole or cut in 2, 4 and 8 pieces
PIECES = {
    "dealt_out_halves": ([1024], 1288, 648, 1, 0),
    "dealt_out_quarters": ([777], 1000, 648, 2, 0),
    "dealt_out_eighths": ([513], 520, 1000, 3, 0),
    "dealt_out_second_wave": ([256 * 13], 1544, 520, 2, 0),
    "dealt_out_groups": ([300, 0, 257, 1, 500], 1160, 1000, 1, 0),
    "handed_out_halves": ([2000, 1, 255], 600, 2056, 1, 1),
    "handed_out_whole": ([700, 300], 2056, 2120, 0, 1),
    "handed_out_second_wave": ([1000, 0, 1300, 256], 1800, 2056, 2, 1),
}


@pytest.mark.parametrize("name", WAYS)
def test_ways_are_reached(way, name):
    counts, N, K = WAYS[name]
    assert way(counts, N, K) == TILED[name]
    assert way(counts, N, 2 * (K // 16 * 16), 2) == TILED[name]   # 8-bit: as many steps of 128 bytes


@pytest.mark.parametrize("name", PIECES)
def test_pieces_are_reached(way, name):
    counts, N, K, cut, handed = PIECES[name]
    assert way(counts, N, K) == (256, 2, 1, handed, cut)


BF16, FP32 = torch.bfloat16, torch.float32


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("name", PIECES)
def test_pieces(name, out):
    """Every element of these ways against fp64: products, input gradients and 8-bit products.

    Tolerances: a 16-bit product is exact in fp32, each of its R additions loses at most one unit in the last place of a
    partial sum (2^-23, truncation allowed, and as much for its product where that is cut), then the output is rounded
    once; 8-bit sums are exact, and the int-to-float conversion and two scale products round by 2^-24 each."""
    from fp4_block_scaled_route_b200 import moe
    counts, N, K, _, _ = PIECES[name]
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    spans = list(zip(off.tolist(), off.tolist()[1:]))
    P, E = sum(counts), len(counts)
    gen = torch.Generator("cuda").manual_seed(N + K)
    x, w = (torch.randn(*s, generator=gen, device="cuda").to(BF16) for s in ((P, K), (E, N, K)))
    ref = torch.cat([x[a:b].double() @ w[e].double().T for e, (a, b) in enumerate(spans)])
    mag = torch.cat([x[a:b].double().abs() @ w[e].double().abs().T for e, (a, b) in enumerate(spans)])
    step = torch.finfo(out).eps / 2
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    guard = torch.full((P + 1, (N + 15) // 16 * 16), 7.0, dtype=out, device="cuda")
    moe.grouped_gemm(x, w, off, out=guard[:P, :N], status=status)
    dx = moe.grouped_gemm_dgrad(x, w.transpose(1, 2).contiguous(), off, out_dtype=out, status=status)
    for y in (guard[:P, :N], dx):
        assert bool(((y.double() - ref).abs() <= step * ref.abs() + 2 * K * 2.0 ** -23 * mag).all())
        assert float((y.double() - ref).norm()) <= (2 * step if out == BF16 else 2e-6) * float(ref.norm())
    assert bool((guard[P:] == 7.0).all()) and bool((guard[:, N:] == 7.0).all())
    K8 = 2 * (K // 16 * 16)
    q = torch.randint(-128, 128, (P, K8), generator=gen, device="cuda", dtype=torch.int8)
    w8 = torch.randint(-128, 128, (E, N, K8), generator=gen, device="cuda", dtype=torch.int8)
    s, c = torch.rand(P, generator=gen, device="cuda") + 0.1, torch.rand(E, N, generator=gen, device="cuda") + 0.1
    y = moe.int8_gemm(q, s, w8, c, offsets=off, out_dtype=out, status=status)
    ref = torch.cat([(q[a:b].double() @ w8[e].double().T) * s[a:b, None].double() * c[e].double() for e, (a, b) in enumerate(spans)])
    assert bool(((y.double() - ref).abs() <= (step + 4 * 2.0 ** -24) * ref.abs()).all())
    assert int(status) == 0
