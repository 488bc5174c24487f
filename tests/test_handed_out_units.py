"""CPU checks of the units that a running pair of CTAs takes off the grid,
compiled for the host from the kernels' own source: whatever the order in
which clusters start or are taken, every unit is computed once, with its own
rows and features."""
import os
import subprocess

from tests.test_grouped_units import CSRC, between

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
static void shuffle(std::vector<int>& v, int window) {
  for (size_t i = 0; i < v.size(); ++i) std::swap(v[i], v[min(v.size() - 1, i + rand() %% window)]);
}
// A grid of `clusters`, of which `room` run at once.
static bool run(int total, int clusters, int room, int window) {
  std::vector<int> queue(clusters), hit(clusters, 0);
  for (int i = 0; i < clusters; ++i) queue[i] = i;
  shuffle(queue, window);
  size_t head = 0;
  struct Pair { int unit; bool left, first; };
  std::vector<Pair> pairs;
  while (head < queue.size() || !pairs.empty()) {
    while ((int)pairs.size() < room && head < queue.size()) pairs.push_back({queue[head++], true, true});
    const size_t i = rand() %% pairs.size();
    Pair& p = pairs[i];
    bool asked_too_often = false;
    auto ask = [&](int* v) {
      asked_too_often |= !p.left;
      if (head == queue.size()) return false;
      *v = queue[head++];
      return true;
    };
    if (!p.first || p.unit >= total) p.unit = next_handed(ask, total, p.left);
    p.first = false;
    if (asked_too_often) return false;
    if (p.unit < total) ++hit[p.unit];
    else pairs.erase(pairs.begin() + i);
  }
  for (int u = 0; u < clusters; ++u) if (hit[u] != (u < total)) return false;
  return true;
}
template <int BN, int CG>
static bool tiles(int E, int M, int teams, const std::vector<int>& off) {
  const int NT = (M + 128 * CG - 1) / (128 * CG);
  std::vector<int> tile(E + 1, 0);
  for (int e = 0; e < E; ++e) tile[e + 1] = tile[e] + (off[e + 1] - off[e] + BN - 1) / BN;
  const Units w = Units::make<BN, CG>(tile[E] * NT, NT, teams);
  int kept = 0;
  for (int i = 0; i < 200 && w.total; ++i) {
    const int u = rand() %% w.total;
    int fresh = 0;
    const Tile a = tile_of<BN, 128 * CG>(u, w, off.data(), tile.data(), fresh);
    const Tile b = tile_of<BN, 128 * CG>(u, w, off.data(), tile.data(), kept);
    if (a.e != b.e || a.m0 != b.m0 || a.p0 != b.p0 || a.rows != b.rows) return false;
  }
  return true;
}
int main() {
  for (int it = 0; it < 3000; ++it) {
    const int total = rand() %% 120, clusters = total + rand() %% 100 + 1;
    if (!run(total, clusters, 1 + rand() %% 20, it %% 3 ? 1 + rand() %% 40 : clusters))
      return printf("units: %%d of %%d\n", total, clusters), 1;
    const int E = 1 + rand() %% 9;
    std::vector<int> off(E + 1, rand() %% 4);
    for (int e = 0; e < E; ++e) off[e + 1] = off[e] + (rand() %% 3 ? rand() %% 900 : 0);
    const int M = 1 + rand() %% 1500, teams = 1 + rand() %% 80;
    if (!tiles<64, 1>(E, M, teams, off) || !tiles<256, 2>(E, M, teams, off)) return printf("tiles: E %%d M %%d\n", E, M), 1;
  }
  puts("ok");
  return 0;
}
"""


def test_units_in_any_order(tmp_path):
    with open(os.path.join(CSRC, "moe_grouped.cu")) as f:
        g = f.read()
    with open(os.path.join(CSRC, "moe_grouped.cuh")) as f:
        h = f.read()
    parts = [between(g, "constexpr int kBand", "\n"), between(g, "struct Tile {", "template <int KIND>"),
             between(g, "struct Units {", "template <int KIND, int BN, int CG, bool SPLIT>\n__global__"),
             between(h, "template <typename Ask>", "\n// ---- groups")]
    src, exe = tmp_path / "units.cpp", tmp_path / "units"
    src.write_text(MAIN % "\n".join(parts))
    subprocess.run(["g++", "-std=c++17", "-O2", "-o", str(exe), str(src)], check=True, timeout=120)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
