// moe_grouped.cu -- ragged grouped products with the weights on the MMA's M
// side: y[p, :] = x[p, :] W_e^T (forward), dx[p, :] = dy[p, :] W_e (input
// gradient), and the 8-bit integer product y[p, n] = s[p] c[e, n]
// sum_k q[p, k] w[e, n, k], for the rows p of every group e.
#include "moe_grouped.cuh"

namespace moe {
namespace {

// One CTA computes tiles of 128 output features by BN rows.  Warp 0 loads
// both operands with TMA, warp 1 issues the MMAs, warps 4-7 read the
// accumulators (double-buffered in tensor memory) and store the result.
template <int KIND, int BN>
struct Cfg {
  static constexpr int THREADS = 256;
  static constexpr int CH = KIND == GG_INT8 ? 128 : 64;  // contraction elements per stage: 128 bytes
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int TABLE = (2 * (kMaxGroups + 3) + 32) * 4;
  static constexpr int BARS = 512;
  static constexpr int FIT = (232448 - 1024 - TABLE - BARS) / STAGE;
  static constexpr int STAGES = FIT < 12 ? FIT : 12;
  static constexpr int TMEM_COLS = 2 * BN < 32 ? 32 : 2 * BN;
  static constexpr int SMEM = 1024 + STAGES * STAGE + TABLE + BARS;
  static_assert((2 * STAGES + 5) * 8 + 8 <= BARS, "barriers");
  static_assert(BN % 16 == 0 && BN <= 256 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "tile");
};

// Row tiles of one group are taken in bands of this many, all features of a
// band before the next one, so that the CTAs running at one time share their
// rows and their weights in the L2.
constexpr int kBand = 8;

struct Tile {
  int e, m0, p0, rows;
};

// Tile number u -> group, first feature, first row, rows.  e walks upwards
// with u, which only grows.
template <int BN>
__device__ __forceinline__ Tile tile_of(int u, int NT, const int* s_off, const int* s_tile, int& e) {
  const int v = u / NT;
  while (s_tile[e + 1] <= v) ++e;
  const int local = u - s_tile[e] * NT, mt = s_tile[e + 1] - s_tile[e];
  const int band = local / (kBand * NT), in_band = local - band * kBand * NT;
  const int bw = min(kBand, mt - band * kBand);
  const int nt = in_band / bw, tt = band * kBand + in_band % bw;
  Tile t;
  t.e = e;
  t.m0 = nt * 128;
  t.p0 = s_off[e] + tt * BN;
  t.rows = min(BN, s_off[e + 1] - t.p0);
  return t;
}

template <int KIND, int BN>
__global__ void __launch_bounds__(Cfg<KIND, BN>::THREADS, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const GroupedParams p) {
  using C = Cfg<KIND, BN>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int* s_off = reinterpret_cast<int*>(smem + STAGES * C::STAGE);
  int* s_tile = s_off + kMaxGroups + 3;
  int* s_scan = s_tile + kMaxGroups + 3;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE + C::TABLE);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);
    }
    mbar_init(done, 1);
    *abort = 0;
    mbar_fence_init();
    tma_prefetch_map(&tmW);
    tma_prefetch_map(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  const bool good = build_group_table<C::THREADS>(p.offsets, p.E, p.P, BN, s_off, s_tile, s_scan);
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int NT = (p.M + 127) / 128;
  const int total = good ? s_tile[p.E] * NT : 0;
  const int KB = (p.R + C::CH - 1) / C::CH;

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_w = p.stream_w ? policy_evict_first() : policy_evict_normal();
      const uint64_t pol_x = policy_evict_normal();
      uint32_t armed = 0, parity = 0;
      bool ok = true;
      int it = 0, e = 0;
      for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
        const Tile t = tile_of<BN>(u, NT, s_off, s_tile, e);
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const int st = it % STAGES;
          const uint32_t ph = (uint32_t)(it / STAGES) & 1u;
          if (!mbar_wait(&empty[st], ph ^ 1u, abort)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[st], C::STAGE);
          armed |= 1u << st;
          parity = (parity & ~(1u << st)) | (ph << st);
          uint8_t* a = smem + st * C::STAGE;
          if (KIND == GG_DGRAD) {
            tma_load_3d(&tmW, &full[st], a, t.m0, kb * C::CH, t.e, pol_w);
            tma_load_3d(&tmW, &full[st], a + C::A_BYTES / 2, t.m0 + 64, kb * C::CH, t.e, pol_w);
          } else {
            tma_load_3d(&tmW, &full[st], a, kb * C::CH, t.m0, t.e, pol_w);
          }
          tma_load_2d(&tmX, &full[st], a + C::A_BYTES, kb * C::CH, t.p0, pol_x);
        }
      }
      // after an abort: every copy in flight lands before the CTA leaves
      if (*abort)
        for (int s = 0; s < STAGES; ++s)
          if (armed & (1u << s)) mbar_drain(&full[s], (parity >> s) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = p.idesc;
      bool ok = true;
      int it = 0, j = 0;
      for (int u = blockIdx.x; u < total && ok; u += gridDim.x, ++j) {
        const int buf = j & 1;
        ok = mbar_wait(&tempty[buf], ((uint32_t)(j >> 1) & 1u) ^ 1u, abort);
        if (!ok) break;
        tc_fence_after();
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const int st = it % STAGES;
          if (!mbar_wait(&full[st], (uint32_t)(it / STAGES) & 1u, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(smem + st * C::STAGE);
          const uint64_t ad = KIND == GG_DGRAD ? sdesc_mn_sw128(a, C::A_BYTES / 2) : sdesc_k_sw128(a);
          const uint64_t bd = sdesc_k_sw128(a + C::A_BYTES);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            // 32 bytes of the contraction per instruction, or 16 rows of 128 bytes
            const uint64_t da = ad + (KIND == GG_DGRAD ? 128 * kk : 2 * kk);
            if (KIND == GG_INT8)
              mma_s8(tmem + buf * BN, da, bd + 2 * kk, idesc, (kb | kk) != 0);
            else
              mma_f16(tmem + buf * BN, da, bd + 2 * kk, idesc, (kb | kk) != 0);
          }
          mma_commit(&empty[st]);
        }
        if (ok) mma_commit(&tfull[buf]);
      }
      mma_commit(done);
      mbar_drain(done, 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int q = warp & 3;
    bool ok = true;
    int j = 0, e = 0;
    for (int u = blockIdx.x; u < total && ok; u += gridDim.x, ++j) {
      const Tile t = tile_of<BN>(u, NT, s_off, s_tile, e);
      const int buf = j & 1;
      ok = mbar_wait(&tfull[buf], (uint32_t)(j >> 1) & 1u, abort);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc_fence_after();
      const int m = t.m0 + q * 32 + lane;
      const bool in = m < p.M;
      const float cs = (KIND == GG_INT8 && in) ? p.col_scale[(size_t)t.e * p.M + m] : 1.0f;
#pragma unroll 1
      for (int c0 = 0; c0 < BN; c0 += 16) {
        if (c0 >= t.rows) break;
        float v[16];
        tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + buf * BN + c0, v);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          if (c0 + c < t.rows && in) {
            const size_t row = (size_t)(t.p0 + c0 + c);
            float r = v[c];
            if (KIND == GG_INT8) r = __fmul_rn(__fmul_rn((float)__float_as_int(r), p.row_scale[row]), cs);
            const size_t at = row * p.ldy + m;
            if (p.out_type == MOE_DT_FP32) static_cast<float*>(p.y)[at] = r;
            else if (p.out_type == MOE_DT_BF16) static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(r);
            else static_cast<__half*>(p.y)[at] = __float2half_rn(r);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[buf]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
  if (threadIdx.x == 0 && p.status) {
    if (*abort) atomicOr(p.status, DEV_TIMEOUT);
    if (!good) atomicOr(p.status, DEV_BAD_ROUTING);
  }
}

template <int KIND, int BN>
cudaError_t launch(const CUtensorMap& tw, const CUtensorMap& tx, const GroupedParams& p, int grid, cudaStream_t s) {
  using C = Cfg<KIND, BN>;
  // per device: the attribute belongs to the current device's context
  const cudaError_t e = cudaFuncSetAttribute(grouped_kernel<KIND, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  grouped_kernel<KIND, BN><<<grid, C::THREADS, C::SMEM, s>>>(tw, tx, p);
  return cudaGetLastError();
}

}  // namespace

int grouped_tile_rows(const GroupedParams& p) {
  const long long avg = ((long long)p.P + p.E - 1) / p.E;
  return avg <= 16 ? 16 : avg <= 64 ? 64 : 256;
}

template <int KIND>
static cudaError_t launch_kind(int bn, const CUtensorMap& tw, const CUtensorMap& tx, const GroupedParams& p, int grid,
                               cudaStream_t s) {
  switch (bn) {
    case 16: return launch<KIND, 16>(tw, tx, p, grid, s);
    case 64: return launch<KIND, 64>(tw, tx, p, grid, s);
    case 256: return launch<KIND, 256>(tw, tx, p, grid, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_grouped(int kind, int bn, const CUtensorMap& tw, const CUtensorMap& tx, const GroupedParams& p0,
                           int sms, cudaStream_t s) {
  GroupedParams p = p0;
  p.idesc = kind == GG_INT8 ? idesc_s8(128, bn) : idesc_f16(128, bn, p.fmt, kind == GG_DGRAD, 0);
  if (kind == GG_FWD) return launch_kind<GG_FWD>(bn, tw, tx, p, sms, s);
  if (kind == GG_DGRAD) return launch_kind<GG_DGRAD>(bn, tw, tx, p, sms, s);
  return launch_kind<GG_INT8>(bn, tw, tx, p, sms, s);
}

}  // namespace moe
