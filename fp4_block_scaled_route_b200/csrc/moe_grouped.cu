// moe_grouped.cu -- ragged grouped products with the weights on the MMA's M
// side: y[p, :] = x[p, :] W_e^T (forward), dx[p, :] = dy[p, :] W_e (input
// gradient), and the 8-bit integer product y[p, n] = s[p] c[e, n]
// sum_k q[p, k] w[e, n, k], for the rows p of every group e.
//
// Weights are the M operand and rows the N operand because a group has any
// number of rows: an MMA's N goes down to 16 (32 for a pair), so a group of a
// few rows costs little more than streaming its weights, and one kernel serves
// both a decode step and a prefill.  The contraction index of the rows is
// contiguous; that of the weights is too in the forward product (K-major
// tiles), and is their row index in the input gradient (MN-major tiles, no
// transposed copy).  Rows of other groups inside a tile are loaded, multiplied
// and not stored: they reach no other row's sums.
//
// What bounds it.  Few rows per group: the weights' stream from HBM (256
// experts, 256 rows, 7168 x 2048 bf16: 698 us, 6.9 TB/s).  Many: the tensor
// cores at the power limit.  Tiles are 256 x 256 on CTA pairs, because a pair
// moves 64 KB into shared memory per step where two CTAs alone move 96, and
// the L2 delivers little more than that: with a quarter of the loads left out
// the dense product took 320 us instead of 352.  32 ragged groups of 32768
// rows, 4096 x 7168: 1643 us, 1.17 PFLOP/s, about 1.1 GHz at 1000 W (cuBLAS
// sustains 1.40 on a dense product of that size); dense 8192 rows: 302 to 334
// us, 1.59 to 1.44 PFLOP/s (cuBLAS 303 to 326).  8-bit: 8192 x 4096 x 7168 159
// us, 3.0 POP/s.
#include "moe_grouped.cuh"

namespace moe {
namespace {

// Tiles of 128 * CG output features by BN rows.  CG = 1: one CTA; CG = 2: a
// pair of CTAs, each with half of the features and half of the rows' operand
// in its shared memory.  SPLIT (CG = 1): the CTAs of a cluster share a tile's
// contraction, and the first joins their partial sums in their order.
//
// Warp 0 loads both operands with TMA, warp 1 (of the even CTA) issues the
// MMAs, warps 4-11 read the accumulators (double-buffered in tensor memory)
// and store the result: as matrix fragments, turned through shared memory by
// stmatrix, so that a lane stores 16 bytes of a row instead of 2.  Stages fill
// the shared memory that is left: the loads' latency under load is about 3300
// cycles, six steps of a pair.
template <int KIND, int BN, int CG, bool SPLIT>
struct Cfg {
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr int CH = KIND == GG_INT8 ? 128 : 64;  // contraction elements per stage: 128 bytes
  static constexpr int BR = BN / CG;                     // rows of the tile that this CTA loads
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = BR * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int TABLE = (2 * (kMaxGroups + 3) + 32) * 4;
  static constexpr int BARS = 512;
  // the epilogue turns CB rows by 32 features per warp and step, through
  // rows of 64 bytes, 80 apart (no two of eight neighbours share a bank)
  static constexpr int CB = BN <= 32 ? 16 : 32;
  static constexpr int TURN = EPI_WARPS * CB * 80;
  // SPLIT: the partial sums of up to MAX_SPLIT - 1 other CTAs
  static constexpr int MAX_SPLIT = !SPLIT ? 1 : BN <= 32 ? 8 : 4;
  static constexpr int JOIN = (MAX_SPLIT - 1) * 128 * BN * 4;
  static constexpr int FIT = (232448 - 1024 - TABLE - BARS - TURN - JOIN) / STAGE;
  static constexpr int STAGES = FIT < 12 ? FIT : 12;
  static constexpr int TMEM_COLS = 2 * BN < 32 ? 32 : 2 * BN;
  static constexpr int SMEM = 1024 + STAGES * STAGE + TABLE + BARS + TURN + JOIN;
  static constexpr int BOX = 32;  // rows of a small box (pairs: tiles that are not full)
  static_assert((2 * STAGES + 13) * 8 + 8 + 16 <= BARS, "barriers");
  static_assert(BN % (16 * CG) == 0 && BN <= 256 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "tile");
  static_assert(!SPLIT || CG == 1, "clusters either pair up or share a contraction");
  static_assert(B_BYTES % 1024 == 0, "128-byte swizzle atoms");
};

// Row tiles of one group are taken in bands of this many, all features of a
// band before the next one, so that the CTAs running at one time share their
// rows and their weights in the L2 (bands of 2, 4 and 16: within 2 %).
constexpr int kBand = 8;

// A contraction of fewer steps (128 bytes each) is not split, and a share
// keeps kMinChunks.  Joining costs about 2 us; B200, 16 rows by 512 features:
// 8 steps 5.0 us whole and 6.1 in two, 16 steps 7.0 in two and 6.4 in four.
constexpr int kSplitChunks = 12, kMinChunks = 4;
// From this many steps on, few large tiles are cut into 64 rows and their
// contraction split instead of being given to pairs: 512 x 512 features, 16
// steps 10.4 us so and 8.2 on pairs; 300 x 256, 32 steps 9.1 and 11.3; 256 x
// 512, 112 steps 13.6 and 29.1.
constexpr int kFewChunks = 24;

// Units are handed out at run time from this many contraction steps on, when
// there are several groups (32 ragged groups of 32768 rows, 4096 features: 16
// steps 264 us dealt out and 286 handed out, 112 steps 1844 and 1650; one group
// of as many rows 1493 either way); a pair asks for its next unit kAhead steps
// before it is through loading the present one.
constexpr int kHandOutChunks = 32;
constexpr int kAhead = 12;
// Up to this many: a pair that looks for a unit may meet all the clusters past
// the last one (0.3 to 1 us each), while its other warps wait within their limit.
constexpr long long kMaxHandOut = 1LL << 18;

struct Tile {
  int e, m0, p0, rows;
};

template <int KIND>
__device__ __forceinline__ uint32_t add_as(uint32_t a, uint32_t b) {
  if (KIND == GG_INT8) return a + b;
  return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}

// The tiles as units of work for `teams` CTAs (or pairs): whole tiles while
// they fill the machine, and the tiles of the last, partial wave cut into
// 1 << cut pieces by rows when that still is one wave.
struct Units {
  int NT, whole, cut, total;
  template <int BN, int CG>
  static __device__ __forceinline__ Units make(int tiles, int NT, int teams) {
    Units w;
    w.NT = NT;
    const int rem = tiles % teams;
    w.whole = tiles - rem;
    w.cut = 0;
    if (CG == 2)
      while (w.cut < 3 && (BN >> (w.cut + 1)) >= 32 && (rem << (w.cut + 1)) <= teams) ++w.cut;
    w.total = w.whole + (rem << w.cut);
    return w;
  }
};

// Unit u -> group, first feature, first row, rows (none for a piece past the
// group's end).  e walks upwards with u, and starts again where u falls.
template <int BN, int BM>
__device__ __forceinline__ Tile tile_of(int u, const Units& w, const int* s_off, const int* s_tile, int& e) {
  const int NT = w.NT;
  int piece = 0, cut = 0;
  if (u >= w.whole && w.cut) {
    const int i = u - w.whole;
    cut = w.cut;
    piece = i & ((1 << cut) - 1);
    u = w.whole + (i >> cut);
  }
  const int v = u / NT;
  if (s_tile[e] > v) e = 0;
  while (s_tile[e + 1] <= v) ++e;
  const int local = u - s_tile[e] * NT, mt = s_tile[e + 1] - s_tile[e];
  const int band = local / (kBand * NT), in_band = local - band * kBand * NT;
  const int bw = min(kBand, mt - band * kBand);
  const int nt = in_band / bw, tt = band * kBand + in_band % bw;
  // Pairs: a group's tiles have equal rows, as near as 64 divides them, so
  // that they take equal time.  CTAs that share a group's rows and weights
  // then stay in step and find them in the L2.
  int width = BN, end = s_off[e + 1];
  const int lo = s_off[e];
  if (BM == 256) width = ((end - lo + mt - 1) / mt + 63) & ~63;
  Tile t;
  t.e = e;
  t.m0 = nt * BM;
  t.p0 = lo + tt * width;
  if (cut) {
    end = min(end, t.p0 + width);
    width = ((width >> cut) + 31) & ~31;
    t.p0 += piece * width;
  }
  t.rows = min(width, end - t.p0);
  return t;
}

template <int KIND, int BN, int CG, bool SPLIT>
__global__ void __launch_bounds__(Cfg<KIND, BN, CG, SPLIT>::THREADS, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const __grid_constant__ CUtensorMap tmXs, const GroupedParams p) {
  using C = Cfg<KIND, BN, CG, SPLIT>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int* s_off = reinterpret_cast<int*>(smem + STAGES * C::STAGE);
  int* s_tile = s_off + kMaxGroups + 3;
  int* s_scan = s_tile + kMaxGroups + 3;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE + C::TABLE);  // (even CTA's are used)
  uint64_t* empty = full + STAGES;   // a commit to each CTA
  uint64_t* tfull = empty + STAGES;  // a commit to each CTA
  uint64_t* tempty = tfull + 2;      // (even CTA) the epilogue warps of each CTA
  uint64_t* joined = tempty + 2;     // (SPLIT, first CTA) the other CTAs' epilogue warps
  uint64_t* done = joined + 1;
  // Units handed out in order (p.hand_out; see warp 2):
  uint64_t* handed = done + 1;   // [2] the next unit is in unit[] (each CTA)
  uint64_t* taken = handed + 2;  // [2] (even CTA) every reader of both CTAs has read it
  uint64_t* want = taken + 2;    // (even CTA) the producer nears the end of its unit
  uint64_t* answered = want + 1; // (even CTA) the hardware's answer is in
  volatile int* unit = reinterpret_cast<volatile int*>(answered + 1);  // [2]
  uint8_t* answer = reinterpret_cast<uint8_t*>(full) + C::BARS - 16;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(answered + 2);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 || SPLIT ? cluster_rank() : 0;
  const int split = SPLIT ? p.split : 1, size = CG * split;  // CTAs that work on a tile
  // handed-out units: the grid has a cluster per unit, and p.teams run at once
  const bool hand_out = CG == 2 && p.hand_out;
  const int team = blockIdx.x / size, teams = hand_out ? p.teams : gridDim.x / size;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], C::EPI_WARPS * CG);
    }
    if (SPLIT) mbar_init(joined, (split - 1) * C::EPI_WARPS);
    mbar_init(done, 1);
    if (CG == 2) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&handed[b], 1);
        mbar_init(&taken[b], 2 * (C::EPI_WARPS + 1) + 1);
      }
      mbar_init(want, 1);
      mbar_init(answered, 1);
    }
    *abort = 0;
    mbar_fence_init();
    tma_prefetch_map(&tmW);
    tma_prefetch_map(&tmX);
    if (CG == 2) tma_prefetch_map(&tmXs);
  }
  if (warp == 1) tmem_alloc_cg<CG>(tmem_holder, C::TMEM_COLS);
  // everything above ran while the kernel before this one could still be
  // running; nothing of its results is read before this point
  griddep_wait();
  tc_fence_before();
  const bool good = build_group_table<C::THREADS>(p.offsets, p.E, p.P, BN, s_off, s_tile, s_scan);
  if (CG == 2 || SPLIT) cluster_sync_all();  // the CTAs' barriers exist before any signal crosses
  tc_fence_after();
  griddep_launch_dependents();  // (tensor memory is held: no later kernel can take it first)
  const uint32_t tmem = *tmem_holder;
  const int NT = (p.M + 128 * CG - 1) / (128 * CG);
  const Units work = Units::make<BN, CG>(good ? s_tile[p.E] * NT : 0, NT, teams);
  const int chunks = (p.R + C::CH - 1) / C::CH;
  // this CTA's part of the contraction
  const int kb0 = SPLIT ? (int)((long long)chunks * rank / split) : 0;
  const int kb1 = SPLIT ? (int)((long long)chunks * (rank + 1) / split) : chunks;

  // contraction steps that one accumulator takes
  const int seg = KIND == GG_INT8 ? chunks : segment_stages(p.out_type);

  // The unit after u, for each warp that walks the units.
  const uint32_t taken0 = CG == 2 ? mapa_rank(taken, 0) : 0;
  int hand = 0;
  auto next_unit = [&](int u) {
    if (CG != 2 || !hand_out) return u + teams;
    const int b = hand & 1;
    const bool in = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(&handed[b], (uint32_t)(hand >> 1) & 1u, abort));
    const int v = in ? unit[b] : work.total;
    __syncwarp();
    if (lane == 0) mbar_arrive_at(taken0 + 8u * b);
    ++hand;
    return v;
  };
  // The first one: a cluster past the last unit may still be handed some.
  auto first_unit = [&]() { return CG == 2 && hand_out && team >= work.total ? next_unit(team) : team; };

  if (warp == 0) {
    const uint64_t pol_w = p.stream_w ? policy_evict_first() : policy_evict_normal();
    const uint64_t pol_x = policy_evict_normal();
    const uint32_t full0 = CG == 2 ? mapa_rank(full, 0) : smem_u32(full);
    uint32_t armed = 0, st = 0, ph = 0;
    bool ok = true;
    int e = 0;
    if (hand_out && rank == 0 && lane == 0 && team >= work.total) mbar_arrive(want);
    for (int u = first_unit(); u < work.total && ok; u = next_unit(u)) {
      const Tile t = tile_of<BN, 128 * CG>(u, work, s_off, s_tile, e);
      if (t.rows <= 0) {
        if (hand_out && rank == 0 && lane == 0) mbar_arrive(want);
        continue;
      }
      // the MMA covers the tile's rows rounded up; each CTA of a pair
      // holds half of them, in small boxes unless the tile is full
      const int n = CG == 2 ? (t.rows + 31) & ~31 : BN;
      const int boxes = CG == 1 || n == BN ? 0 : (n / 2 + C::BOX - 1) / C::BOX;
      const uint32_t bytes = CG == 1 || n == BN ? CG * C::STAGE : 2 * (C::A_BYTES + boxes * C::BOX * 128);
      const int half = CG == 2 ? (int)rank : 0;
      const int m0 = t.m0 + half * 128, p0 = t.p0 + half * (n / CG);
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = mbar_wait_warp(&empty[st], ph ^ 1u, abort);
        if (!ok) break;
        if (hand_out && rank == 0 && lane == 0 && kb == max(kb1 - kAhead, kb0)) mbar_arrive(want);
        uint8_t* a = smem + st * C::STAGE;
        const int r0 = kb * C::CH;
        if (elect_one()) {
          // the even CTA posts the bytes of both
          if (CG == 1 || rank == 0) mbar_arrive_expect_tx(&full[st], bytes);
          if constexpr (CG == 1) {
            if (KIND == GG_DGRAD) {
              tma_load_3d(&tmW, &full[st], a, m0, r0, t.e, pol_w);
              tma_load_3d(&tmW, &full[st], a + C::A_BYTES / 2, m0 + 64, r0, t.e, pol_w);
            } else {
              tma_load_3d(&tmW, &full[st], a, r0, m0, t.e, pol_w);
            }
            tma_load_2d(&tmX, &full[st], a + C::A_BYTES, r0, p0, pol_x);
          } else {
            const uint32_t bar = full0 + 8u * st;
            if (KIND == GG_DGRAD) {
              tma_load_3d_pair(&tmW, bar, a, m0, r0, t.e, pol_w);
              tma_load_3d_pair(&tmW, bar, a + C::A_BYTES / 2, m0 + 64, r0, t.e, pol_w);
            } else {
              tma_load_3d_pair(&tmW, bar, a, r0, m0, t.e, pol_w);
            }
            if (boxes == 0) tma_load_2d_pair(&tmX, bar, a + C::A_BYTES, r0, p0, pol_x);
            for (int b = 0; b < boxes; ++b)
              tma_load_2d_pair(&tmXs, bar, a + C::A_BYTES + b * C::BOX * 128, r0, p0 + b * C::BOX, pol_x);
          }
        }
        armed |= 1u << st;
        if (++st == STAGES) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    // after an abort: the copies in flight land before the CTAs leave (the
    // even CTA's barriers count both CTAs' bytes).  Stages below st were last
    // armed with parity ph, the others with the parity before.
    if (*abort && (CG == 1 || rank == 0))
      for (uint32_t s = 0; s < STAGES; ++s)
        if (armed & (1u << s)) mbar_drain(&full[s], s < st ? ph : ph ^ 1u);
    __syncwarp();
  } else if (warp == 1) {
    if (CG == 1 || rank == 0) {
      const uint32_t empty0 = smem_u32(empty), tfull0 = smem_u32(tfull), a0 = smem_u32(smem);
      const uint64_t ad0 = KIND == GG_DGRAD ? sdesc_mn_sw128(a0, C::A_BYTES / 2) : sdesc_k_sw128(a0);
      const uint64_t bd0 = sdesc_k_sw128(a0 + C::A_BYTES);
      // an instruction takes 32 bytes of the contraction, or 16 rows of 128 bytes
      constexpr uint64_t step_a = KIND == GG_DGRAD ? 128 : 2, step_b = 2;
      bool ok = true;
      uint32_t st = 0, ph = 0;
      int j = 0, e = 0, u = first_unit();
      Tile next = {};
      if (u < work.total) next = tile_of<BN, 128 * CG>(u, work, s_off, s_tile, e);
      while (u < work.total && ok) {
        const Tile t = next;
        if (!hand_out) u += teams;
        if (t.rows <= 0) {
          if (hand_out) u = next_unit(u);
          if (u < work.total) next = tile_of<BN, 128 * CG>(u, work, s_off, s_tile, e);
          continue;
        }
        const int n = (t.rows + 16 * CG - 1) & ~(16 * CG - 1);
        const uint32_t idesc = p.idesc | (uint32_t)(n >> 3) << 17;
        for (int kb = kb0; kb < kb1; ++j) {  // one accumulator each: segments
          const int buf = j & 1, first = kb, end = min(kb1, kb + seg);
          ok = mbar_wait_warp(&tempty[buf], ((uint32_t)(j >> 1) & 1u) ^ 1u, abort);
          if (!ok) break;
          tc_fence_after();
          for (; kb < end; ++kb) {
            ok = mbar_wait_warp(&full[st], ph, abort);
            if (!ok) break;
            tc_fence_after();
            const uint64_t off = st * (C::STAGE >> 4);
            mma_steps4<KIND == GG_INT8, CG>(tmem + buf * BN, ad0 + off, bd0 + off, step_a, step_b, idesc, kb != first);
            mma_commit_all<CG>(empty0 + 8u * st);
            if (++st == STAGES) {
              st = 0;
              ph ^= 1u;
            }
            // the next tile is looked up while the tensor cores have work
            if (!hand_out && kb == kb0 && u < work.total) next = tile_of<BN, 128 * CG>(u, work, s_off, s_tile, e);
          }
          if (!ok) break;
          mma_commit_all<CG>(tfull0 + 8u * buf);
        }
        if (hand_out) {
          u = next_unit(u);
          if (u < work.total) next = tile_of<BN, 128 * CG>(u, work, s_off, s_tile, e);
        }
      }
      mma_commit_all<CG>(smem_u32(done));
      mbar_drain(done, 0);
    }
    __syncwarp();
  } else if (CG == 2 && warp == 2) {
    // Pairs that share rows or weights find them in the L2 only while they run
    // in step.  With units dealt out beforehand the pairs drift apart over the
    // many tiles of ragged groups; here each pair takes the next unit just
    // before it needs it, so that neighbours in order are neighbours in time.
    // The even CTA's warp 2 asks the hardware and tells both CTAs.
    if (hand_out && rank == 0) {
      const uint32_t handed0 = mapa_rank(handed, 0), handed1 = mapa_rank(handed, 1);
      const uint32_t unit1 = mapa_rank(const_cast<const int*>(unit), 1);
      int asked = 0;
      bool left = true;
      auto ask = [&](int* v) {  // the next unit's number, or none left (false)
        if (lane == 0) {
          mbar_arrive_expect_tx(answered, 16);
          try_cancel(answer, answered);
        }
        __syncwarp();
        const bool in = mbar_wait_warp(answered, (uint32_t)asked++ & 1u, abort);
        const int block = in ? cancelled_block(answer) : -1;
        fence_proxy_async_smem();  // the answer is read before the next one may land on it
        __syncwarp();
        *v = block >= 0 ? block / 2 : work.total;
        return block >= 0;
      };
      for (int i = 0;; ++i) {
        const int b = i & 1;
        if (!mbar_wait_warp(want, (uint32_t)i & 1u, abort) ||
            !mbar_wait_warp(&taken[b], ((uint32_t)(i >> 1) & 1u) ^ 1u, abort))
          break;
        // (the clusters past the last unit are taken off the grid as well, so that they need not start, set up and
        // leave: offsets that cover few of the rows, or none, leave many)
        const int v = next_handed(ask, work.total, left);
        if (lane == 0) {
          unit[b] = v;
          asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(unit1 + 4u * b), "r"(v) : "memory");
          mbar_arrive_at(handed0 + 8u * b);
          mbar_arrive_at(handed1 + 8u * b);
        }
        __syncwarp();
        if (v >= work.total) break;
      }
      // (an answer still on its way lands before the CTA leaves)
      if (*abort && asked) mbar_drain(answered, (uint32_t)(asked - 1) & 1u);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // Two warps per quarter of the features share the tile's rows, CB by CB.
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tempty0 = CG == 2 ? mapa_rank(tempty, 0) : smem_u32(tempty);
    // SPLIT: [other CTA][warp][step][register / 4][lane][4] words
    constexpr int STEPS = (BN + 2 * C::CB - 1) / (2 * C::CB), NG = C::CB / 8;
    uint32_t* join = reinterpret_cast<uint32_t*>(smem + STAGES * C::STAGE + C::TABLE + C::BARS + C::TURN);
    constexpr int PER_WARP = STEPS * NG * 8 * 32, PER_CTA = 128 * BN;
    static_assert((BN < 2 * C::CB ? 4 : 8) * PER_WARP == PER_CTA, "partial sums");
    uint8_t* turn = smem + STAGES * C::STAGE + C::TABLE + C::BARS + (warp - 4) * C::CB * 80;
    const uint32_t turn_st = smem_u32(turn) + (lane & 7) * 80 + (lane >> 3) * 16;
    bool ok = true;
    int j = 0, e = 0;
    for (int u = first_unit(); u < work.total && ok; u = next_unit(u)) {
      const Tile t = tile_of<BN, 128 * CG>(u, work, s_off, s_tile, e);
      if (t.rows <= 0) continue;
      const int m0 = t.m0 + (CG == 2 ? (int)rank * 128 : 0) + q * 32;  // this warp's first feature
      // int8: the scales of the features this thread holds
      float cs[4];
      if (KIND == GG_INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = m0 + i * 8 + (lane >> 2);
          cs[i] = m < p.M ? __ldg(p.col_scale + (size_t)t.e * p.M + m) : 0.0f;
        }
      }
      // int8: a lane holds the scale of one of the step's rows, the next
      // step's loaded a step ahead
      auto scale_of = [&](int c) {
        return KIND == GG_INT8 && lane < C::CB && c + lane < t.rows ? __ldg(p.row_scale + t.p0 + c + lane) : 0.0f;
      };
      float next_scale = scale_of(half * C::CB);
      // Pairs into fp32, or of several segments: these add up in registers, a
      // lane holding one feature of all the warp's rows, so that a store is
      // 128 (or 64) bytes of one row.  (Into fp32, 32768 ragged rows
      // of 32 experts, 7168 -> 4096: 1777 us; 2290 when the segments add up in
      // the result's memory; 1757 with one segment.)
      if (STEPS > 1 && KIND != GG_INT8 && (p.out_type == MOE_DT_FP32 || chunks > seg)) {
        float s[STEPS][C::CB];
#pragma unroll
        for (int i = 0; i < STEPS * C::CB; ++i) s[i / C::CB][i % C::CB] = 0.0f;
        for (int left_kb = kb1 - kb0; left_kb > 0; left_kb -= seg, ++j) {
          const int buf = j & 1;
          ok = mbar_wait_warp(&tfull[buf], (uint32_t)(j >> 1) & 1u, abort);
          if (!ok) break;
          tc_fence_after();
          const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + buf * BN;
#pragma unroll
          for (int i = 0; i < STEPS * C::CB; i += 16) {
            const int c0 = (i / C::CB * 2 + half) * C::CB + i % C::CB;
            if (c0 >= t.rows) continue;
            float v[16];
            tmem_ld16(acc + c0, v);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) s[i / C::CB][i % C::CB + k] += v[k];
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_at(tempty0 + 8u * buf);
        }
        if (!ok) break;
        const size_t at = (size_t)t.p0 * p.ldy + m0 + lane;
#pragma unroll
        for (int i = 0; i < STEPS * C::CB; ++i) {
          const int c = (i / C::CB * 2 + half) * C::CB + i % C::CB;
          const float v = s[i / C::CB][i % C::CB];
          if (p.out_type == MOE_DT_FP32) {
            if (c < t.rows && m0 + lane < p.M) static_cast<float*>(p.y)[at + (size_t)c * p.ldy] = v;
          } else if (c < t.rows && m0 + lane < p.M)
            static_cast<uint16_t*>(p.y)[at + (size_t)c * p.ldy] = (uint16_t)pack16(v, 0.0f, p.out_type == MOE_DT_BF16);
        }
        __syncwarp();
        continue;
      }
      // The segments (one, but for long contractions) add up in registers:
      // tiles with several steps have left above.
      uint32_t f[2][NG * 4];
      for (int left_kb = kb1 - kb0, sg = 0; left_kb > 0; left_kb -= seg, ++sg, ++j) {
        const bool last = left_kb <= seg;
        const int buf = j & 1;
        ok = mbar_wait_warp(&tfull[buf], (uint32_t)(j >> 1) & 1u, abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + buf * BN;
        // the other CTAs' sums have arrived (data written by them: acquire)
        if (SPLIT && rank == 0 && last) {
          ok = mbar_wait_cluster(joined, 0, abort);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
        }
        for (int c0 = half * C::CB; c0 < t.rows && m0 < p.M; c0 += 2 * C::CB) {
          const int left = t.rows - c0;  // rows of this step: min(left, CB)
          if (STEPS == 1 && sg > 0) {
            uint32_t h[2][NG * 4];
            tmem_ld_16x256b<NG>(acc + c0, h[0]);
            tmem_ld_16x256b<NG>(acc + (16u << 16) + c0, h[1]);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < NG * 8; ++i)
              f[i / (NG * 4)][i % (NG * 4)] = add_as<KIND>(f[i / (NG * 4)][i % (NG * 4)], h[i / (NG * 4)][i % (NG * 4)]);
          } else {
            tmem_ld_16x256b<NG>(acc + c0, f[0]);
            tmem_ld_16x256b<NG>(acc + (16u << 16) + c0, f[1]);
            tmem_wait_ld();
          }
          if (STEPS == 1 && !last) continue;
          if (SPLIT) {
            uint32_t* at = join + (warp - 4) * PER_WARP + (c0 / (2 * C::CB)) * (NG * 8 * 32) + lane * 4;
            if (rank != 0) {
              const uint32_t to = mapa_rank(at + (rank - 1) * PER_CTA, 0);
#pragma unroll
              for (int i = 0; i < NG * 2; ++i) {
                const uint32_t* v = &f[i / NG][(i % NG) * 4];
                st_cluster_v4(to + i * 512, v[0], v[1], v[2], v[3]);
              }
              continue;
            }
            // in the CTAs' order, whatever order they finished in
            for (int r = 0; r < split - 1; ++r) {
#pragma unroll
              for (int i = 0; i < NG * 2; ++i) {
                const uint4 o = *reinterpret_cast<const uint4*>(at + r * PER_CTA + i * 128);
                uint32_t* v = &f[i / NG][(i % NG) * 4];
                v[0] = add_as<KIND>(v[0], o.x);
                v[1] = add_as<KIND>(v[1], o.y);
                v[2] = add_as<KIND>(v[2], o.z);
                v[3] = add_as<KIND>(v[3], o.w);
              }
            }
          }
          const float row_scale = next_scale;
          next_scale = scale_of(c0 + 2 * C::CB);
          const bool bf = p.out_type == MOE_DT_BF16;
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            uint32_t w[4];
            float rs[2];
            if (KIND == GG_INT8) {
#pragma unroll
              for (int h = 0; h < 2; ++h) rs[h] = __shfl_sync(0xFFFFFFFFu, row_scale, i * 8 + (lane & 3) * 2 + h);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {  // features 8 g .. 8 g + 7 of the warp's 32
              float a = __uint_as_float(f[g >> 1][i * 4 + (g & 1) * 2]);
              float b = __uint_as_float(f[g >> 1][i * 4 + (g & 1) * 2 + 1]);
              if (KIND == GG_INT8) {
                a = __fmul_rn(__fmul_rn((float)__float_as_int(a), rs[0]), cs[g]);
                b = __fmul_rn(__fmul_rn((float)__float_as_int(b), rs[1]), cs[g]);
              }
              if (p.out_type == MOE_DT_FP32) {
                // eight neighbouring lanes (l / 4) fill a 32-byte sector of one row
                const int m = m0 + g * 8 + (lane >> 2), c = i * 8 + (lane & 3) * 2;
                float* y = static_cast<float*>(p.y) + (size_t)(t.p0 + c0 + c) * p.ldy + m;
                if (m < p.M && c < left) y[0] = a;
                if (m < p.M && c + 1 < left) y[p.ldy] = b;
              } else {
                w[g] = pack16(a, b, bf);
              }
            }
            if (p.out_type == MOE_DT_FP32) continue;
            stmatrix_x4_trans(turn_st + i * 8 * 80, w[0], w[1], w[2], w[3]);
          }
          __syncwarp();  // the next step's accumulators are read by the whole warp
          if (p.out_type == MOE_DT_FP32) continue;
          uint16_t* y = static_cast<uint16_t*>(p.y) + (size_t)(t.p0 + c0) * p.ldy + m0;
#pragma unroll
          for (int i = 0; i < C::CB / 8; ++i) {
            const int c = i * 8 + (lane >> 2), part = (lane & 3) * 8;
            if (c < left && m0 + part < p.M) {
              const uint4 v = *reinterpret_cast<const uint4*>(turn + c * 80 + part * 2);
              uint16_t* to = y + c * p.ldy + part;
              if (m0 + part + 8 <= p.M) {
                *reinterpret_cast<uint4*>(to) = v;
              } else {
                const uint16_t* x = reinterpret_cast<const uint16_t*>(&v);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  if (m0 + part + k < p.M) to[k] = x[k];
              }
            }
          }
          __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (SPLIT && rank != 0 && last && lane == 0) mbar_arrive_at(mapa_rank(joined, 0));
        if (lane == 0) mbar_arrive_at(tempty0 + 8u * buf);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // no CTA of a cluster leaves while another may still signal it or use its memory
  if (CG == 2 || SPLIT) cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_cg<CG>(tmem, C::TMEM_COLS);
  if (threadIdx.x == 0 && p.status) {
    if (*abort) atomicOr(p.status, DEV_TIMEOUT);
    if (!good) atomicOr(p.status, DEV_BAD_ROUTING);
  }
}

template <int KIND, int BN, int CG, bool SPLIT>
cudaError_t launch(const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& txs, const GroupedParams& p,
                   int grid, cudaStream_t s) {
  using C = Cfg<KIND, BN, CG, SPLIT>;
  if (SPLIT && p.split > C::MAX_SPLIT) return cudaErrorInvalidValue;
  return launch_cluster<grouped_kernel<KIND, BN, CG, SPLIT>>(grid, C::THREADS, C::SMEM, SPLIT ? p.split : CG, s, tw, tx,
                        txs, p);
}

}  // namespace

GroupedTile grouped_tile(const GroupedParams& p, int kind, int sms) {
  const int chunks = (p.R + (kind == GG_INT8 ? 127 : 63)) / (kind == GG_INT8 ? 128 : 64);
  const long long groups = p.E < p.P ? p.E : p.P;  // that can have rows
  // most tiles there can be: ceil(c / rows) <= 1 + (c - 1) / rows in every group with c rows
  auto most = [&](int rows, int features) {
    return (groups + (p.P - groups) / rows) * (long long)((p.M + features - 1) / features);
  };
  // Few tiles: 2 to 8 CTAs share a tile's contraction while every share keeps
  // kMinChunks steps and all clusters, one for each tile, are resident at once.
  auto shares = [&](int rows) {
    int split = 1;
    while (chunks >= kSplitChunks && split < (rows <= 32 ? 8 : 4) &&
           most(rows, 128) <= resident_clusters(split * 2, sms) && chunks >= split * 2 * kMinChunks)
      split *= 2;
    return split;
  };
  // On one CTA without sharing, tiles have 64 rows; on pairs, 256.  B200, 64
  // groups, 2048 x 4096 bf16, us with 64 rows, 256 (and 32, 16): 4 rows a group
  // 157, 170 (162, 163), 24: 158, 177 (163, 211), 48: 162, 180 (204), 64: 182,
  // 182, 96: 218, 188, 128: 265, 193.
  const long long average = (p.P + p.E - 1) / p.E;
  GroupedTile t{64, 1, 1, sms, sms};
  if (average > 64 && !(chunks >= kFewChunks && shares(64) > 1)) {
    t.rows = 256;
    t.ctas = 2;
    t.grid = t.running = sms / 2 * 2;
    // a cluster for every unit there can be: tiles, and the pieces of the last wave
    const long long units = most(256, 256) + sms / 2;
    if (p.E > 1 && chunks >= kHandOutChunks && units <= kMaxHandOut) t.grid = (int)units * 2;
    return t;
  }
  // Shared tiles hold the group's rows when there is one group, else twice the
  // average, since routed groups vary; a lower tile leaves room for more stages
  // (8 rows by 4096 x 4096: 9.6 us in tiles of 16, 15.4 in tiles of 64).
  const long long want = p.E == 1 ? p.P : 2 * average;
  const int rows = want <= 16 ? 16 : want <= 32 ? 32 : 64;
  if ((t.split = shares(rows)) > 1) {
    t.rows = rows;
    t.grid = (int)most(rows, 128) * t.split;
  }
  return t;
}

template <int KIND>
static cudaError_t launch_kind(GroupedTile t, const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& txs,
                               const GroupedParams& p, cudaStream_t s) {
  switch (t.rows) {
    case 16: return launch<KIND, 16, 1, true>(tw, tx, txs, p, t.grid, s);
    case 32: return launch<KIND, 32, 1, true>(tw, tx, txs, p, t.grid, s);
    case 64:
      return t.split > 1 ? launch<KIND, 64, 1, true>(tw, tx, txs, p, t.grid, s)
                         : launch<KIND, 64, 1, false>(tw, tx, txs, p, t.grid, s);
    case 256: return launch<KIND, 256, 2, false>(tw, tx, txs, p, t.grid, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_grouped(int kind, GroupedTile t, const CUtensorMap& tw, const CUtensorMap& tx,
                           const CUtensorMap& txs, const GroupedParams& p0, cudaStream_t s) {
  GroupedParams p = p0;
  p.split = t.split;
  p.hand_out = t.ctas == 2 && t.grid > t.running;
  p.teams = t.running / t.ctas;
  // N is set tile by tile
  p.idesc = kind == GG_INT8 ? idesc_s8(128 * t.ctas, 0) : idesc_f16(128 * t.ctas, 0, p.fmt, kind == GG_DGRAD, 0);
  if (kind == GG_FWD) return launch_kind<GG_FWD>(t, tw, tx, txs, p, s);
  if (kind == GG_DGRAD) return launch_kind<GG_DGRAD>(t, tw, tx, txs, p, s);
  return launch_kind<GG_INT8>(t, tw, tx, txs, p, s);
}

}  // namespace moe
