"""CPU check of how the grouped products deal out their work: the units of
moe_grouped.cu and moe_wgrad.cu, compiled for the host from the kernels' own
source, cover every output element exactly once, for random groups, sizes and
numbers of CTAs."""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_block_scaled_route_b200", "csrc")

MAIN = r"""
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <vector>
#define __device__
#define __forceinline__ inline
using std::max;
using std::min;
%s
static bool wgrad(int E, int N, int K, int teams, const std::vector<int>& off) {
  const int TN = (N + 255) / 256, TC = (K + 127) / 128;
  std::vector<int> hit((size_t)E * TN * TC, 0);
  for (int t = 0; t < teams; ++t) {
    WWalk w(off.data(), E, N, K, t, teams);
    WUnit u;
    while (w.take(u, teams)) {
      if (u.k0 >= K) continue;
      if (u.e < 0 || u.e >= E || u.n0 %% 256 || u.n0 >= N || u.k0 %% 128) return false;
      if (u.lo != off[u.e] || u.hi != off[u.e + 1]) return false;
      for (int b = 0; b < u.nb; ++b) hit[((size_t)u.e * TN + u.n0 / 256) * TC + u.k0 / 128 + b]++;
    }
  }
  for (int h : hit) if (h != 1) return false;
  return true;
}
template <int BN, int CG>
static bool grouped(int E, int M, int teams, const std::vector<int>& off) {
  constexpr int BM = 128 * CG;
  const int NT = (M + BM - 1) / BM;
  std::vector<int> tile(E + 1, 0);
  for (int e = 0; e < E; ++e) tile[e + 1] = tile[e] + (off[e + 1] - off[e] + BN - 1) / BN;
  const Units w = Units::make<BN, CG>(tile[E] * NT, NT, teams);
  // (a launch leaves room for the tiles and one wave of pieces)
  if (w.total > tile[E] * NT + teams) return false;
  std::vector<int> hit((size_t)(off[E] + 1) * NT, 0);
  for (int t = 0; t < teams; ++t) {
    int e = 0;
    for (int u = t; u < w.total; u += teams) {
      const Tile x = tile_of<BN, BM>(u, w, off.data(), tile.data(), e);
      if (x.rows <= 0) continue;
      if (x.rows > BN || x.m0 %% BM || x.m0 >= M || x.p0 < off[x.e] || x.p0 + x.rows > off[x.e + 1]) return false;
      for (int r = 0; r < x.rows; ++r) hit[(size_t)(x.p0 + r) * NT + x.m0 / BM]++;
    }
  }
  for (int p = off[0]; p < off[E]; ++p)
    for (int n = 0; n < NT; ++n) if (hit[(size_t)p * NT + n] != 1) return false;
  return true;
}
int main() {
  for (int it = 0; it < 6000; ++it) {
    const int E = 1 + rand() %% 9, teams = 1 + rand() %% 80, top = it %% 3 ? 90 : 900;
    std::vector<int> off(E + 1, rand() %% 4);
    for (int e = 0; e < E; ++e) off[e + 1] = off[e] + (rand() %% 3 ? rand() %% top : 0);
    const int N = 1 + rand() %% 1500, K = 8 * (1 + rand() %% 200);
    if (!wgrad(E, N, K, teams, off)) return printf("weight gradient: E %%d N %%d K %%d teams %%d\n", E, N, K, teams), 1;
    if (!grouped<16, 1>(E, N, teams, off) || !grouped<64, 1>(E, N, teams, off) || !grouped<256, 2>(E, N, teams, off))
      return printf("product: E %%d M %%d teams %%d\n", E, N, teams), 1;
  }
  puts("ok");
  return 0;
}
"""


def between(text, start, stop):
    m = re.search(re.escape(start) + r".*?(?=" + re.escape(stop) + ")", text, flags=re.S)
    assert m, (start, stop)
    return m.group(0)


def test_every_output_element_is_computed_once(tmp_path):
    with open(os.path.join(CSRC, "moe_wgrad.cu")) as f:
        w = f.read()
    with open(os.path.join(CSRC, "moe_grouped.cu")) as f:
        g = f.read()
    parts = [between(w, "constexpr int kWM", "// SPLIT: p.split pairs"),
             between(g, "constexpr int kBand", "\n"), between(g, "struct Tile {", "template <int KIND>"),
             between(g, "struct Units {", "template <int KIND, int BN, int CG, bool SPLIT>\n__global__")]
    src, exe = tmp_path / "units.cpp", tmp_path / "units"
    src.write_text(MAIN % "\n".join(parts))
    subprocess.run(["g++", "-std=c++17", "-O2", "-o", str(exe), str(src)], check=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
