// moe_grouped.cuh -- what the ragged grouped products (moe_grouped.cu,
// moe_wgrad.cu) share: operand descriptors, pair and cluster PTX, and the
// table of row tiles that every CTA builds from the groups' offsets.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "moe_internal.h"
#include "moe_ops.h"
#include "moe_ptx.cuh"

namespace moe {

// ---- TMA ----------------------------------------------------------------------
__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint64_t* bar, void* dst, int c0, int c1, int c2,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// The same into this CTA's shared memory, completing on a barrier of either
// CTA of the pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_3d_pair(const CUtensorMap* map, uint32_t bar, void* dst, int c0, int c1,
                                                 int c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(const CUtensorMap* map, uint32_t bar, void* dst, int c0, int c1,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
      : "memory");
}

// Store of a box from shared memory; what lies outside the tensor is dropped.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2,
                                             uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%2, %3, %4}], [%1], %5;" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until at most N of this thread's stores still read shared memory / are
// incomplete.
template <int N>
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void tma_store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Order this thread's writes to its shared memory before the asynchronous
// proxy's (TMA's, the tensor cores') accesses that follow.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// ---- operands -----------------------------------------------------------------
// Shared-memory descriptor of an operand whose M (or N) index is the
// contiguous one, as TMA writes it with 128-byte swizzle: boxes of 64
// 16-bit elements along M by `box_rows` contraction rows, each row a 128-byte
// line.  Eight lines form a 1024-byte core group (stride offset: the next
// eight contraction rows); the next 64 elements along M start one box later
// (leading offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t box_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(box_bytes >> 4) << 16;  // leading byte offset: next 64 elements along M
  d |= static_cast<uint64_t>(1024 >> 4) << 32;       // stride byte offset: next 8 contraction rows
  d |= static_cast<uint64_t>(1) << 46;               // descriptor version for sm_100
  d |= static_cast<uint64_t>(2) << 61;               // layout: 128-byte swizzle
  return d;
}

// Instruction descriptors.  kind::f16 with fp32 accumulation: both operands
// fp16 (fmt 0) or both bf16 (fmt 1); a_mn / b_mn: that operand's M / N index
// is contiguous.  kind::i8: signed bytes, int32 accumulation.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int fmt, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(fmt) << 7) | (static_cast<uint32_t>(fmt) << 10) |
         (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_s8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// The tensor cores truncate each addition to an accumulator, so that its error
// grows with their number.  An accumulator therefore takes a segment of the
// contraction, and the segments' sums are added with rounding.  Measured on
// B200 for terms of one sign, relative to the sum: 64 MMAs of 16 products lose
// 1.0e-6 (bf16) and 5.8e-6 (fp16, whose products are longer and cut as well),
// longer segments 1e-7 per MMA of either; with random signs 64 MMAs are off by
// 1.0e-6 and 1.3e-6 in the 2-norm.
//   fp32 outputs: segments of 16 stages, 64 MMAs.  With 32 stages twice the
//     error, for 1 % of the time of a product and 2 % of an input gradient.
//   fp16: 128 stages, 5e-5, a tenth of half a step (4.9e-4; one accumulator
//     over 2^18 elements is off by 1.7e-3).
//   bf16: 512 stages, 1.7e-4, 5 % of half a step (3.9e-3).
constexpr int kSegment = 16;
__host__ __device__ constexpr int segment_stages(int out_type) {
  return out_type == MOE_DT_FP32 ? kSegment : out_type == MOE_DT_FP16 ? 128 : 512;
}

// ---- issue ----------------------------------------------------------------------
// The issuing warps run their loops with all 32 lanes (so that addresses and
// descriptors stay in uniform registers) and let one elected lane issue.
// With the loop inside `if (lane == 0)` a pair's pipeline step of four MMAs
// took 680 cycles on B200 with nothing to load, and takes 620 this way (the
// MMAs alone need 512): a dense 8192 x 4096 x 7168 product 360 -> 327 us.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "elect.sync _|P, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, P;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// STEPS MMAs along the contraction, each `sa` / `sb` (descriptor units) after
// the last; the first one overwrites the accumulator unless `accumulate`.  CG
// = 1: of this CTA; CG = 2: of the pair (M / 2 rows of A and N / 2 rows of B
// in each CTA, M / 2 accumulator rows in each).  Called by a whole warp.
#define MOE_MMA_STEPS(GROUP, KIND)                                                                       \
  asm volatile(                                                                                          \
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"                                   \
      "elect.sync _|e, 0xFFFFFFFF;\n\t"                                                                  \
      "setp.ne.b32 p, %6, 0;\n\t"                                                                        \
      "add.u64 a1, %1, %3;\n\tadd.u64 a2, a1, %3;\n\tadd.u64 a3, a2, %3;\n\t"                            \
      "add.u64 b1, %2, %4;\n\tadd.u64 b2, b1, %4;\n\tadd.u64 b3, b2, %4;\n\t"                            \
      "@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %5, p;\n\t"                      \
      "@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], a1, b1, %5, 1;\n\t"                      \
      "@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], a2, b2, %5, 1;\n\t"                      \
      "@e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], a3, b3, %5, 1;\n\t}\n" ::"r"(d),         \
      "l"(a), "l"(b), "l"(sa), "l"(sb), "r"(idesc), "r"(accumulate)                                      \
      : "memory")
template <bool INT8, int CG>
__device__ __forceinline__ void mma_steps4(uint32_t d, uint64_t a, uint64_t b, uint64_t sa, uint64_t sb,
                                           uint32_t idesc, uint32_t accumulate) {
  if constexpr (INT8 && CG == 1) MOE_MMA_STEPS("1", "i8");
  if constexpr (INT8 && CG == 2) MOE_MMA_STEPS("2", "i8");
  if constexpr (!INT8 && CG == 1) MOE_MMA_STEPS("1", "f16");
  if constexpr (!INT8 && CG == 2) MOE_MMA_STEPS("2", "f16");
}
#undef MOE_MMA_STEPS
// One MMA of the pair on 16-bit operands, by a whole warp.
__device__ __forceinline__ void mma_f16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ---- CTA pairs ------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// shared::cluster address of the same shared-memory location in CTA `rank`
__device__ __forceinline__ uint32_t mapa_rank(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
// Bounded wait, acquire at cluster scope (for data another CTA wrote here).
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const long long t0 = clock64();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitCycles) {
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
// Arrive on a barrier (in both CTAs of a pair, at the same place) once the
// MMAs that this warp's elected lane issued so far completed.  Called by a
// whole warp.  One commit for both CTAs: a commit each costs the issuing warp
// another 50 cycles per step.  `both` names the pair's CTAs in their cluster.
template <int CG>
__device__ __forceinline__ void mma_commit_all(uint32_t bar, uint16_t both = 3) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}\n" ::"r"(
            bar),
        "h"(both)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_alloc_cg(uint32_t* dst, uint32_t ncols) {
  if constexpr (CG == 1) {
    tmem_alloc(dst, ncols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc_cg(uint32_t taddr, uint32_t ncols) {
  if constexpr (CG == 1)
    tmem_dealloc(taddr, ncols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// mbar_wait by a whole warp: false for every lane if it gave up for one.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort));
}
// Bounded wait of a whole warp for what lies any number of units of work away:
// the limit covers one unit, and starts anew whenever *moved, which the
// producer advances unit by unit, has changed.
__device__ __forceinline__ bool mbar_wait_moving(uint64_t* bar, uint32_t parity, volatile int* abort,
                                                 const volatile int* moved) {
  bool ok = mbar_try_wait(bar, parity);
  long long t0 = clock64();
  for (int seen = *moved; !ok && !*abort; ok = mbar_try_wait(bar, parity)) {
    const int now = *moved;
    if (now != seen) {
      seen = now;
      t0 = clock64();
    } else if (clock64() - t0 > kWaitCycles) {
      *abort = 1;
    }
  }
  return __all_sync(0xFFFFFFFFu, ok);
}
// Bounded wait used while draining: like mbar_wait, but blind to the abort word.
__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitCycles) break;
}

// Two fp32 values -> two bf16 or fp16 (lo in bits 0-15), each rounded to nearest even once.
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ---- accumulators out of tensor memory, turned -------------------------------
// 16 lanes by 8 * NG columns of 32 bits as matrix fragments: thread l gets, for
// each group of 8 columns, (lane l / 4, columns 2 (l % 4) and + 1) and the same
// columns of lane l / 4 + 8.
template <int NG>
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t* r) {
  static_assert(NG == 2 || NG == 4, "column groups");
  if constexpr (NG == 2)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// Four 8 x 8 matrices of 16-bit values, each stored transposed: column r of
// matrix i becomes the 16 bytes at the address that lane 8 i + r gives.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// Store 16 fp32 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}

// ---- work handed out by the hardware --------------------------------------------
// A grid larger than the machine has clusters that wait for room.  try_cancel
// takes the first of them off the grid; the taker does its work instead.  The
// answer (16 bytes) lands in shared memory and is counted on `bar`.
__device__ __forceinline__ void try_cancel(void* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
// First block of the cluster that was taken, or -1: none was left.
__device__ __forceinline__ int cancelled_block(const void* answer) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, h;\n\t}\n"
      : "=r"(got), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return got ? (int)x : -1;
}

// The next unit of work below `total`, or `total` when the grid has none left.
// ask(&v) takes one cluster off the grid (v: its unit), or returns false: none
// was left, and nothing may be asked again.  Clusters come in no promised
// order: those past the last unit are passed over, not taken for the end.
template <typename Ask>
__device__ __forceinline__ int next_handed(Ask&& ask, int total, bool& left) {
  while (left) {
    int v = total;
    left = ask(&v);
    if (left && v < total) return v;
  }
  return total;
}

// ---- groups --------------------------------------------------------------------
// Builds in shared memory the groups' offsets and the first row tile of each
// group (tiles of `tile_rows` rows).  All THREADS threads of the CTA call it;
// it ends with a barrier.  offsets == nullptr: one group of all P rows.
// Returns false when the offsets are unusable (negative, falling, or past P):
// the caller then computes nothing.
template <int THREADS>
__device__ __forceinline__ bool build_group_table(const int32_t* offsets, int E, int P, int tile_rows, int* s_off,
                                                  int* s_tile, int* s_scan) {
  static_assert(THREADS % 32 == 0 && THREADS <= 1024, "block");
  constexpr int NW = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (E + THREADS - 1) / THREADS;  // consecutive groups per thread
  const int e0 = tid * per;
  int sum = 0, bad = 0;
  for (int i = 0; i < per; ++i) {
    const int e = e0 + i;
    if (e >= E) break;
    const int lo = offsets ? offsets[e] : 0, hi = offsets ? offsets[e + 1] : P;
    bad |= (lo < 0) | (hi < lo) | (hi > P);
    s_off[e] = lo;
    if (e == E - 1) s_off[E] = hi;
    s_tile[e + 1] = bad ? 0 : (hi - lo) / tile_rows + ((hi - lo) % tile_rows != 0);
    sum += s_tile[e + 1];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_scan[warp] = incl;
  bad = __syncthreads_or(bad);
  int run = incl - sum;
#pragma unroll
  for (int w = 0; w < NW; ++w)
    if (w < warp) run += s_scan[w];
  for (int i = 0; i < per; ++i) {
    const int e = e0 + i;
    if (e >= E) break;
    run += s_tile[e + 1];
    s_tile[e + 1] = run;
  }
  if (tid == 0) s_tile[0] = 0;
  __syncthreads();
  return !bad;
}

}  // namespace moe
