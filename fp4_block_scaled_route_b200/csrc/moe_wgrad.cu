// moe_wgrad.cu -- weight gradients of the ragged grouped product:
// dW_e[n, k] = sum over the rows p of group e of dy[p, n] x[p, k].
//
// What bounds it: for long groups the tensor cores and the loads that feed
// them (dense, 8192 rows into 4096 x 7168: 324 to 363 us, 1.48 to 1.32
// PFLOP/s; cuBLAS 333 to 360), for groups of a few hundred rows also the
// result's way out (32 groups of 512 rows into 2048 x 7168 bf16, 940 MB: 497
// us), for short ones that alone (64 groups of 16 rows into 392 x 1032 fp32,
// 104 MB: 37 us, 2.9 TB/s; a fill reaches 6.2).
#include <type_traits>

#include "moe_grouped.cuh"

namespace moe {
namespace {

// A pair of CTAs computes 256 output rows n by 256 columns k: each holds 128
// of the rows (accumulators in its tensor memory, double-buffered) and loads
// half of both operands.  The contraction runs over the group's rows, so both
// operands have their output index contiguous (MN-major): a stage holds 64
// rows of 128 dy columns and of 128 x columns, in boxes of 64 columns whose
// rows are 128-byte lines.
//
// Warp 0 loads, warp 1 (of the even CTA) issues the MMAs, warp 2 fills in the
// rows of a group that do not make up a whole MMA step, warps 4-11 read the
// accumulators, round them and store them by TMA from shared memory.
// Stages: 6, or 5 when the offsets of very many experts take the room.
template <int STAGES_>
struct WCfg {
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr int BN = 256;
  static constexpr int CH = 64;        // rows per stage
  static constexpr int BOX = CH * 128;
  static constexpr int STAGE = 4 * BOX;  // dy: boxes 0, 1; x: boxes 2, 3
  static constexpr int STAGES = STAGES_;
  static constexpr int OUT = 32 * 128;  // per epilogue warp: a box of 32 rows of 128 bytes
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr int BARS = 512;
  static constexpr int SMEM = 1024 + STAGES * STAGE + EPI_WARPS * OUT + BARS;  // (+ the offsets)
  static constexpr int MAX_E = (232448 - SMEM) / 4 - 1;
  static_assert((4 * STAGES + 7) * 8 + 12 <= BARS && MAX_E > 0, "shared memory");
};

// An epilogue warp stores 32 rows of 128 bytes by TMA: v is a lane's row, k and
// n the first column and row.  Columns and rows past the ends are not written.
__device__ __forceinline__ void store_box(const CUtensorMap& tmO, uint8_t* box, const uint32_t* v, int k, int n, int e) {
  const int lane = threadIdx.x & 31;
  uint8_t* line = box + lane * 128;  // 16-byte piece i of a line sits at i ^ (lane & 7)
  tma_store_wait_read<0>();          // lane 0's store has read the box
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint4*>(line + ((i ^ (lane & 7)) * 16)) =
        make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) tma_store_3d(&tmO, box, k, n, e, policy_evict_normal());
}

// A warp's part of a tile into fp32 of a group of `rows` rows: the segments add
// up in 128 registers, then 32 rows n by `wide` columns k leave.  Returns the
// accumulators read, -1 when a wait gave up.
__device__ __forceinline__ int sum_tile(const CUtensorMap& tmO, uint32_t acc, int wide, int rows, int j, uint64_t* tfull,
                                        uint32_t tempty0, volatile int* abort, uint8_t* box, int k0, int cols, int n,
                                        int e) {
  float sum[4][32];
#pragma unroll
  for (int i = 0; i < 128; ++i) sum[i / 32][i % 32] = 0.0f;
  int taken = 0;
  for (; rows > 0; rows -= kSegment * 64, ++taken) {
    const int buf = (j + taken) & 1;
    if (!mbar_wait_warp(&tfull[buf], (uint32_t)((j + taken) >> 1) & 1u, abort)) return -1;
    tc_fence_after();
#pragma unroll
    for (int i = 0; i < 128; i += 16) {
      if (i >= wide) continue;
      float v[16];
      tmem_ld16(acc + buf * 256 + i, v);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 16; ++k) sum[i / 32][i % 32 + k] += v[k];
    }
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive_at(tempty0 + 8u * buf);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i * 32 >= wide || i * 32 >= cols) continue;
    uint32_t v[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(sum[i][k]);
    store_box(tmO, box, v, k0 + i * 32, n, e);
  }
  return taken;
}

// 16 columns of one accumulator added to another, for this warp's 32 lanes.
__device__ __forceinline__ void add_columns(uint32_t to, uint32_t from) {
  float a[16], b[16];
  tmem_ld16(to, a);
  tmem_ld16(from, b);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) a[i] += b[i];
  tmem_st16(to, a);
}

// Work of one pair: all features of an expert before the next column of
// tiles, all tiles of an expert before the next expert.  The units of the
// last, partial wave are halves of 128 columns when they still are one wave.
constexpr int kWM = 256, kWN = 256;  // rows and columns of a tile

struct WUnit {
  int e, lo, hi;  // expert, its rows
  int n0, k0, nb; // first row and column of the output, 128-column halves
};
struct WWalk {
  const int* s_off;
  int TN, per, K, whole, halves, total;
  int u, r, e;  // next unit; its place within expert e
  __device__ __forceinline__ WWalk(const int* off, int E, int N, int K_, int team, int teams) : s_off(off), K(K_) {
    TN = (N + kWM - 1) / kWM;
    per = TN * ((K + kWN - 1) / kWN);
    total = E * per;
    const int rem = total % teams;
    whole = total - rem;
    halves = rem * 2 <= teams;
    if (halves) total = whole + 2 * rem;
    u = team;
    r = team;
    e = 0;
  }
  __device__ __forceinline__ bool take(WUnit& t, int teams) {
    if (u >= total) return false;
    int at = r, half = 0;
    if (halves && u >= whole) {
      // (the walk passes `whole` once: r is u's place counted from expert e)
      half = (u - whole) & 1;
      at = r - (u - whole) + ((u - whole) >> 1);
    }
    int ee = e;
    while (at >= per) {
      at -= per;
      ++ee;
    }
    t.e = ee;
    t.lo = s_off[ee];
    t.hi = s_off[ee + 1];
    t.n0 = (at % TN) * kWM;
    t.k0 = (at / TN) * kWN;
    t.nb = K - t.k0 > 128 ? 2 : 1;
    if (halves && u >= whole) {
      t.nb = 1;
      t.k0 += half * 128;  // (past K: nothing is loaded, computed or stored)
    }
    u += teams;
    r += teams;
    if (u < whole)
      while (r >= per) {
        r -= per;
        ++e;
      }
    return true;
  }
};

// SPLIT: p.split pairs of a cluster share a tile's rows; each then sends the
// others their part of the columns of its sums, adds up its own part in the
// pairs' order, and stores it.
//
// The segments of a long group (see kSegment) add up in tensor memory: the first
// keeps its accumulator, the others take turns in the second, and the epilogue
// adds each to the first.  The MMAs wait meanwhile: 32768 rows into 2048 x 4096
// fp16, four segments, 372 -> 377 us.
//
// SUM: into fp32.  A group's segments add up in
// the epilogue's registers, for which the other warps leave some of theirs.
// 8192 rows into 2048 x 7168: 228 us (1.06 PFLOP/s), 277 when the segments add
// up in the result's memory, 223 with one segment (and 7e-6 off).
enum WMode { W_WHOLE, W_SPLIT, W_SUM };
constexpr int kSumRegs = 168, kSumRegsLow = 104, kSumRegsHigh = 200;  // at launch; warps 0-3; warps 4-11
static_assert(128 * kSumRegsLow + 256 * kSumRegsHigh <= 384 * kSumRegs, "registers of the launch");

template <int STAGES, WMode MODE>
__global__ void __launch_bounds__(WCfg<STAGES>::THREADS, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmX,
                 const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmY16,
                 const __grid_constant__ CUtensorMap tmX16, const WgradParams p) {
  using C = WCfg<STAGES>;
  constexpr bool SPLIT = MODE == W_SPLIT, SUM = MODE == W_SUM;
  static_assert(C::THREADS == 384, "register split");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out = smem + STAGES * C::STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(out + C::EPI_WARPS * C::OUT);  // (even CTA) both CTAs' bytes
  uint64_t* empty = full + STAGES;      // a commit to each CTA
  uint64_t* filled = empty + STAGES;    // (even CTA) both CTAs' warps 2 have filled in a stage's last rows
  uint64_t* fill = filled + STAGES;     // this CTA's warp 2 may fill in a stage's last rows
  uint64_t* tfull = fill + STAGES;      // a commit to each CTA
  uint64_t* tempty = tfull + 2;         // (even CTA) the epilogue warps of both CTAs
  uint64_t* ready = tempty + 2;         // (SPLIT) the other pairs' memory is free
  uint64_t* joined = ready + 1;         // (SPLIT) their sums are here
  uint64_t* done = joined + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* moved = abort + 1;  // units that warp 0 has come to
  int* s_off = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + C::BARS);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // rank: of the CTA in its pair; pair: of the pair in its cluster
  const int split = SPLIT ? p.split : 1;
  const int rank = (int)cluster_rank() & 1, pair = SPLIT ? (int)cluster_rank() >> 1 : 0;
  const uint32_t even = 2 * pair;                       // the pair's even CTA in the cluster
  const uint16_t both = (uint16_t)(3u << (2 * pair));   // its two CTAs
  const int team = blockIdx.x / (2 * split), teams = gridDim.x / (2 * split);
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&filled[s], 2);
      mbar_init(&fill[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * C::EPI_WARPS);
    }
    if (SPLIT) {
      mbar_init(ready, (split - 1) * C::EPI_WARPS);
      mbar_init(joined, (split - 1) * C::EPI_WARPS);
    }
    mbar_init(done, 1);
    *abort = 0;
    *moved = 0;
    mbar_fence_init();
    tma_prefetch_map(&tmY);
    tma_prefetch_map(&tmX);
    tma_prefetch_map(&tmO);
    tma_prefetch_map(&tmY16);
    tma_prefetch_map(&tmX16);
  }
  if (warp == 1) tmem_alloc_cg<2>(tmem_holder, C::TMEM_COLS);
  // everything above ran while the kernel before this one could still be
  // running; nothing of its results is read before this point
  griddep_wait();
  // unusable offsets (negative, falling, past P): nothing is computed
  int bad = 0;
  for (int e = threadIdx.x; e < p.E; e += C::THREADS) {
    const int lo = p.offsets[e], hi = p.offsets[e + 1];
    bad |= (lo < 0) | (hi < lo) | (hi > p.P);
    s_off[e] = lo;
    if (e == p.E - 1) s_off[p.E] = hi;
  }
  tc_fence_before();
  bad = __syncthreads_or(bad);
  cluster_sync_all();  // both CTAs' barriers exist before any signal crosses
  tc_fence_after();
  griddep_launch_dependents();  // (tensor memory is held: no later kernel can take it first)
  const uint32_t tmem = *tmem_holder;
  const int seg = segment_stages(p.out_type) * C::CH;  // rows that one accumulator takes
  // (a unit's place in the walk: the same for every role)
  WWalk walk(s_off, bad ? 0 : p.E, p.N, p.K, team, teams);
  // The next unit, with this pair's share of the rows: whole stages of them.
  auto take = [&](WUnit& t) {
    if (!walk.take(t, teams)) return false;
    if (SPLIT) {
      const int lo = t.lo, stages = (t.hi - lo + C::CH - 1) / C::CH;
      t.lo = min(t.hi, lo + (int)((long long)stages * pair / split) * C::CH);
      t.hi = min(t.hi, lo + (int)((long long)stages * (pair + 1) / split) * C::CH);
    }
    return true;
  };
  // Rows of a stage that TMA must not load as part of a 64-row box, because
  // those past the group's end, in the same 16-row MMA step, may hold anything
  // (NaN too) and have to be zero in both operands: such a stage's whole steps
  // come by TMA in boxes of 16 rows, the rest by warp 2.
  auto ragged = [](int held) { return held < C::CH && (held & 15); };

  if (SUM && warp < 4) regs_shrink<kSumRegsLow>();
  if (warp == 0) {
    const uint64_t pol = policy_evict_normal();
    const uint32_t full0 = mapa_rank(full, even);
    uint32_t armed = 0, st = 0, ph = 0;
    bool ok = true;
    WUnit t;
    while (ok && take(t)) {
      if (t.k0 >= p.K) continue;
      if (lane == 0) *moved = *moved + 1;
      __syncwarp();
      const int n0 = t.n0 + rank * 128, k0 = t.k0 + rank * 64 * t.nb, nb = t.nb;
      const uint32_t bytes = (2 + nb) * C::BOX;
      for (int row = t.lo; row < t.hi; row += C::CH) {
        ok = mbar_wait_warp(&empty[st], ph ^ 1u, abort);
        if (!ok) break;
        const uint32_t bar = full0 + 8u * st;
        uint8_t* a = smem + st * C::STAGE;
        const int held = t.hi - row, steps = ragged(held) ? held / 16 : 4;  // those that TMA loads
        if (elect_one()) {
          if (steps == 0) {
            if (rank == 0) mbar_arrive(&full[st]);
          } else if (rank == 0) {
            mbar_arrive_expect_tx(&full[st], 2 * (bytes / 4) * steps);
          }
          if (!ragged(held)) {
            tma_load_2d_pair(&tmY, bar, a, n0, row, pol);
            tma_load_2d_pair(&tmY, bar, a + C::BOX, n0 + 64, row, pol);
            tma_load_2d_pair(&tmX, bar, a + 2 * C::BOX, k0, row, pol);
            if (nb == 2) tma_load_2d_pair(&tmX, bar, a + 3 * C::BOX, k0 + 64, row, pol);
          } else {
            mbar_arrive(&fill[st]);
            for (int g = 0; g < steps; ++g) {
              uint8_t* ag = a + g * (C::BOX / 4);
              tma_load_2d_pair(&tmY16, bar, ag, n0, row + 16 * g, pol);
              tma_load_2d_pair(&tmY16, bar, ag + C::BOX, n0 + 64, row + 16 * g, pol);
              tma_load_2d_pair(&tmX16, bar, ag + 2 * C::BOX, k0, row + 16 * g, pol);
              if (nb == 2) tma_load_2d_pair(&tmX16, bar, ag + 3 * C::BOX, k0 + 64, row + 16 * g, pol);
            }
          }
        }
        armed |= 1u << st;
        if (++st == STAGES) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    // after an abort: the copies in flight land before the CTAs leave.
    // Stages below st were last armed with parity ph, the others before.
    if (*abort && rank == 0)
      for (uint32_t s = 0; s < STAGES; ++s)
        if (armed & (1u << s)) mbar_drain(&full[s], s < st ? ph : ph ^ 1u);
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    const uint32_t empty0 = smem_u32(empty), tfull0 = smem_u32(tfull);
    const uint64_t ad0 = sdesc_mn_sw128(smem_u32(smem), C::BOX);
    const uint64_t bd0 = sdesc_mn_sw128(smem_u32(smem) + 2 * C::BOX, C::BOX);
    uint32_t uses = 0;  // parity of each stage's next use of filled
    uint32_t st = 0, ph = 0, cur = 0, acc_ph = 0;  // next unit's accumulator; parity of each one's next use
    bool ok = true;
    WUnit next;
    bool more = take(next);
    while (more && ok) {
      const WUnit t = next;
      const int lo = t.lo, hi = t.hi, nb = t.nb;
      if (hi == lo || t.k0 >= p.K) {
        more = take(next);
        continue;
      }
      const uint32_t idesc = p.idesc | (uint32_t)(128 * nb >> 3) << 17;
      for (int row = lo; row < hi;) {  // segments
        const uint32_t buf = SUM || row == lo ? cur : cur ^ 1u;
        const int first = row, end = min(hi, row + seg);
        const uint32_t d = tmem + buf * C::BN;
        ok = mbar_wait_warp(&tempty[buf], ((acc_ph >> buf) & 1u) ^ 1u, abort);
        if (!ok) break;
        acc_ph ^= 1u << buf;
        if (SUM) cur ^= 1u;
        tc_fence_after();
        for (; row < end; row += C::CH) {
          const int held = min(C::CH, hi - row), steps = (held + 15) / 16;
          ok = mbar_wait_warp(&full[st], ph, abort);
          if (ok && ragged(hi - row)) {
            ok = mbar_wait_cluster(&filled[st], (uses >> st) & 1u, abort);
            ok = __all_sync(0xFFFFFFFFu, ok);
            uses ^= 1u << st;
          }
          if (!ok) break;
          tc_fence_after();
          const uint64_t off = st * (C::STAGE >> 4);
          if (steps == 4) {
            mma_steps4<false, 2>(d, ad0 + off, bd0 + off, 128, 128, idesc, row != first);
          } else {
            for (int kk = 0; kk < steps; ++kk)
              mma_f16_pair(d, ad0 + off + 128 * kk, bd0 + off + 128 * kk, idesc, (row != first) | (kk != 0));
          }
          mma_commit_all<2>(empty0 + 8u * st, both);
          if (++st == STAGES) {
            st = 0;
            ph ^= 1u;
          }
          // the next unit is looked up while the tensor cores have work
          if (row == lo) more = take(next);
        }
        if (!ok) break;
        mma_commit_all<2>(tfull0 + 8u * buf, both);
      }
      if (!SUM) cur ^= 1u;
    }
    mma_commit_all<2>(smem_u32(done), both);
    mbar_drain(done, 0);
    __syncwarp();
  } else if (warp == 2) {
    // The last rows of a group, when they do not fill a 16-row step, and zeros
    // behind them.  They are read into registers long before their stage is
    // free and written as soon as it is, so that they are there before the
    // stage's other rows.  (Zeroing the tail of a box that TMA loaded, after it
    // had landed, cost 10 % of the time at 512 rows a group.)
    const uint32_t filled0 = mapa_rank(filled, even);
    uint32_t st = 0, uses = 0;  // first stage of the unit; parity of each stage's next use of fill
    bool ok = true;
    WUnit t;
    while (ok && take(t)) {
      if (t.hi <= t.lo || t.k0 >= p.K) continue;
      const int rows = t.hi - t.lo, stages = (rows + C::CH - 1) / C::CH, held = rows - (stages - 1) * C::CH;
      const uint32_t s = (st + stages - 1) % STAGES;  // the last stage
      st = (st + stages) % STAGES;
      if (!ragged(held)) continue;
      const int first = held & ~15, count = held & 15, row0 = t.hi - count;
      const int n0 = t.n0 + rank * 128, k0 = t.k0 + rank * 64 * t.nb;
      // piece j of this lane: 16 bytes of one row of one box
      uint4 v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int i = j * 32 + lane, box = i >> 7, r = (i >> 3) & 15, c = (box & 1) * 64 + (i & 7) * 8;
        const int col = (box < 2 ? n0 : k0) + c, cols = box < 2 ? p.N : p.K;
        const uint16_t* src = box < 2 ? p.dy + (long long)(row0 + r) * p.lddy + col
                                      : p.x + (long long)(row0 + r) * p.ldx + col;
        v[j] = make_uint4(0, 0, 0, 0);
        if (r < count) {
          if (col + 8 <= cols) {
            v[j] = __ldg(reinterpret_cast<const uint4*>(src));
          } else if (col < cols) {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (col + k < cols) w[k / 2] |= (uint32_t)src[k] << (16 * (k & 1));
            v[j] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      // (units without such rows are passed over here, so the first one that has some may be far away)
      ok = mbar_wait_moving(&fill[s], (uses >> s) & 1u, abort, moved);
      if (!ok) break;
      uses ^= 1u << s;
      uint8_t* a = smem + s * C::STAGE + first * 128;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int i = j * 32 + lane, box = i >> 7, r = (i >> 3) & 15;
        // (`first` is a multiple of 16 lines: the swizzle goes by r alone)
        *reinterpret_cast<uint4*>(a + box * C::BOX + r * 128 + (((i & 7) ^ (r & 7)) * 16)) = v[j];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(filled0 + 8u * s);
    }
    __syncwarp();
  } else if (warp >= 4) {
    if (SUM) regs_grow<kSumRegsHigh>();
    // Two warps per quarter of the rows, one for each half of the columns; a
    // step is a box of 32 rows by 128 bytes.
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tempty0 = mapa_rank(tempty, even);
    uint8_t* box = out + (warp - 4) * C::OUT;
    const bool f32 = p.out_type == MOE_DT_FP32, bf = p.out_type == MOE_DT_BF16;
    bool ok = true;
    int j = 0;
    uint32_t cur = 0, acc_ph = 0;  // as in warp 1
    WUnit t;
    while (ok && take(t)) {
      if (t.k0 >= p.K) continue;
      const int n = t.n0 + rank * 128 + q * 32, wide = 64 * t.nb, k0 = t.k0 + half * wide;
      const bool none = t.hi == t.lo;
      if (SUM) {
        const int read = sum_tile(tmO, tmem + ((uint32_t)(q * 32) << 16) + half * wide, wide, t.hi - t.lo, j, tfull,
                                  tempty0, abort, box, k0, n < p.N ? p.K - k0 : 0, n, t.e);
        ok = read >= 0;
        j += read;
        continue;
      }
      const uint32_t buf = cur, quarter = tmem + ((uint32_t)(q * 32) << 16);
      if (!none) {
        ok = mbar_wait_warp(&tfull[buf], (acc_ph >> buf) & 1u, abort);
        if (!ok) break;
        acc_ph ^= 1u << buf;
        tc_fence_after();
        // the columns that this warp reads, of SPLIT's owners too
        const int blocks = 4 * t.nb / split;
        for (int left = t.hi - t.lo - seg; left > 0; left -= seg) {
          const uint32_t other = buf ^ 1u;
          ok = mbar_wait_warp(&tfull[other], (acc_ph >> other) & 1u, abort);
          if (!ok) break;
          acc_ph ^= 1u << other;
          tc_fence_after();
          for (int pr = 0; pr < split; ++pr)
            for (int b = 0; b < blocks; ++b) {
              const uint32_t at = quarter + ((2 * pr + half) * blocks + b) * 16;
              add_columns(at + buf * C::BN, at + other * C::BN);
            }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_at(tempty0 + 8u * other);
          __syncwarp();
        }
        if (!ok) break;
        cur ^= 1u;
      }
      if (SPLIT) {
        // Every pair owns 1 / split of the tile's columns, of which this warp
        // takes half, in blocks of 16.  A pair's sums go straight into the
        // owners' pipeline memory, which is free once their MMAs are done:
        // [sender][warp][block][register / 4][lane][4] words.
        const int part = 128 * t.nb / split, blocks = part / 32;
        uint32_t* sums = reinterpret_cast<uint32_t*>(smem);
        const uint32_t row_acc = quarter + buf * C::BN + half * (part / 2);
        auto sums_at = [&](int sender, int b) {
          return sums + (((sender * C::EPI_WARPS + (warp - 4)) * blocks + b) * 16 * 32) + lane * 4;
        };
        auto own = [&](int pr, int b, float (&v)[16]) {
          if (none) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0.0f;
          } else {
            tmem_ld16(row_acc + pr * part + b * 16, v);
            tmem_wait_ld();
          }
        };
        __syncwarp();
        for (int pr = 0; pr < split; ++pr)
          if (pr != pair && lane == 0) mbar_arrive_at(mapa_rank(ready, 2 * pr + rank));
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(ready, 0, abort));
        if (!ok) break;
        for (int pr = 0; pr < split; ++pr) {
          if (pr == pair) continue;
          for (int b = 0; b < blocks; ++b) {
            float v[16];
            own(pr, b, v);
            const uint32_t to = mapa_rank(sums_at(pair, b), 2 * pr + rank);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              st_cluster_v4(to + i * 512, __float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                            __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_at(mapa_rank(joined, 2 * pr + rank));
          __syncwarp();
        }
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(joined, 0, abort));
        if (!ok) break;
        for (int b = 0; b < blocks; ++b) {
          float mine[16], v[16];
          own(pair, b, mine);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0.0f;
          for (int pr = 0; pr < split; ++pr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float4 o = make_float4(mine[4 * i], mine[4 * i + 1], mine[4 * i + 2], mine[4 * i + 3]);
              if (pr != pair) o = *reinterpret_cast<const float4*>(sums_at(pr, b) + i * 128);
              v[4 * i] += o.x;
              v[4 * i + 1] += o.y;
              v[4 * i + 2] += o.z;
              v[4 * i + 3] += o.w;
            }
          }
          const int k = t.k0 + pair * part + half * (part / 2) + b * 16;
          const size_t at = ((size_t)t.e * p.N + n + lane) * p.K + k;
          // (K is a multiple of 16 bytes: no piece is partly inside)
          const int cols = n + lane < p.N ? p.K - k : 0;
          if (f32) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              if (i < cols)
                *reinterpret_cast<float4*>(static_cast<float*>(p.dw) + at + i) =
                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 16; i += 8)
              if (i < cols)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dw) + at + i) =
                    make_uint4(pack16(v[i], v[i + 1], bf), pack16(v[i + 2], v[i + 3], bf),
                               pack16(v[i + 4], v[i + 5], bf), pack16(v[i + 6], v[i + 7], bf));
          }
          __syncwarp();  // the next block's accumulators are read by the whole warp
        }
        break;  // a cluster has one tile
      }
      const uint32_t acc = quarter + buf * C::BN + half * wide;
      // The whole accumulator is read and rounded before anything is stored, so
      // that the MMAs of the tile after next can start (box by box: 32 groups
      // of 512 rows 536 us, so 498).
      uint32_t w[2][32];  // a box of 64 columns each
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t v[64];
        if (none || b * 64 >= wide) {
#pragma unroll
          for (int i = 0; i < 64; ++i) v[i] = 0;
        } else {
          tmem_ld32(acc + b * 64, reinterpret_cast<float*>(v));
          tmem_ld32(acc + b * 64 + 32, reinterpret_cast<float*>(v) + 32);
          tmem_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) w[b][i] = pack16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), bf);
      }
      if (!none) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(tempty0 + 8u * buf);
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (b * 64 < wide && k0 + b * 64 < p.K && n < p.N) store_box(tmO, box, w[b], k0 + b * 64, n, t.e);
    }
    tma_store_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  // neither CTA leaves while the other may still signal it or read its memory
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_cg<2>(tmem, C::TMEM_COLS);
  if (threadIdx.x == 0 && p.status) {
    if (*abort) atomicOr(p.status, DEV_TIMEOUT);
    if (bad) atomicOr(p.status, DEV_BAD_ROUTING);
  }
}

// The register split is only safe if the block is launched with the registers
// that it counts on.
template <int STAGES>
bool sum_fits() {
  static const bool fits = [] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, wgrad_kernel<STAGES, W_SUM>) == cudaSuccess && fa.numRegs >= kSumRegs;
  }();
  return fits;
}

}  // namespace

cudaError_t launch_wgrad(const CUtensorMap& ty, const CUtensorMap& tx, const CUtensorMap& to,
                         const CUtensorMap& ty16, const CUtensorMap& tx16, const WgradParams& p0, int sms,
                         cudaStream_t s) {
  WgradParams p = p0;
  p.idesc = idesc_f16(kWM, 0, p.fmt, 1, 1);  // N is set tile by tile
  // Few tiles of many rows: 2 or 4 pairs share a tile while each has kMinStages
  // stages and all are resident.  B200, 4096 rows into 512 x 512: 22.0 us
  // whole, 17.7 in two, 15.6 in four; 16384 into 1024 x 1024: 76 whole, 46 in
  // two; 1000 into 384 x 176 (16 stages): 8.9 whole, 11.0 in two.
  constexpr int kMinStages = 16;
  const long long tiles = (long long)p.E * ((p.N + kWM - 1) / kWM) * ((p.K + kWN - 1) / kWN);
  const int stages = (int)((p.P / p.E + 63) / 64);
  p.split = 1;
  // (into fp32 a share of a group of average length is one segment, see kSegment: longer ones add up faster in
  // registers)
  const int most = p.out_type == MOE_DT_FP32 ? 4 * kSegment : 1 << 20;
  while (p.split < 4 && stages <= most && tiles <= resident_clusters(p.split * 4, sms) && stages >= p.split * 2 * kMinStages)
    p.split *= 2;
  const int grid = p.split > 1 ? (int)tiles * p.split * 2 : sms / 2 * 2;
  auto go = [&](auto n) {
    using C = WCfg<n>;
    const size_t smem = C::SMEM + (p.E + 1) * sizeof(int32_t);
    if (p.split > 1)
      return launch_cluster<wgrad_kernel<n, W_SPLIT>>(grid, C::THREADS, smem, 2 * p.split, s, ty, tx, to, ty16, tx16, p);
    if (p.out_type != MOE_DT_FP32)
      return launch_cluster<wgrad_kernel<n, W_WHOLE>>(grid, C::THREADS, smem, 2, s, ty, tx, to, ty16, tx16, p);
    if (!sum_fits<n>()) return cudaErrorInvalidConfiguration;
    return launch_cluster<wgrad_kernel<n, W_SUM>>(grid, C::THREADS, smem, 2, s, ty, tx, to, ty16, tx16, p);
  };
  static_assert(WCfg<5>::MAX_E >= 1024, "every expert count has a variant");
  return p.E <= WCfg<6>::MAX_E ? go(std::integral_constant<int, 6>{}) : go(std::integral_constant<int, 5>{});
}

}  // namespace moe
