// moe_wgrad.cu -- weight gradients of the ragged grouped product:
// dW_e[n, k] = sum over the rows p of group e of dy[p, n] x[p, k].
#include "moe_grouped.cuh"

namespace moe {
namespace {

// The contraction runs over rows, so both operands have their output index
// contiguous (MN-major).  A stage holds 64 rows of 128 dy columns (two boxes
// of 64) and of BN x columns (BN / 64 boxes).
struct WCfg {
  static constexpr int THREADS = 256;
  static constexpr int BN = 256;
  static constexpr int CH = 64;
  static constexpr int BOX = 64 * 128;
  static constexpr int NA = 2, NB = BN / 64;
  static constexpr int STAGE = (NA + NB) * BOX;
  static constexpr int STAGES = 4;
  static constexpr int TMEM_COLS = 512;
  static constexpr int BARS = 512;
  static constexpr int SMEM = 1024 + STAGES * STAGE + BARS;
};

__global__ void __launch_bounds__(WCfg::THREADS, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmX,
                 const WgradParams p) {
  using C = WCfg;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE);
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
    tma_prefetch_map(&tmY);
    tma_prefetch_map(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  // everything above ran while the kernel before this one could still be
  // running; nothing of its results is read before this point
  griddep_wait();
  // unusable offsets (negative, falling, past P): nothing is computed
  int bad = 0;
  for (int e = threadIdx.x; e < p.E; e += C::THREADS) {
    const int lo = p.offsets[e], hi = p.offsets[e + 1];
    bad |= (lo < 0) | (hi < lo) | (hi > p.P);
  }
  tc_fence_before();
  bad = __syncthreads_or(bad);
  tc_fence_after();
  griddep_launch_dependents();  // (tensor memory is held: no later kernel can take it first)
  const uint32_t tmem = *tmem_holder;
  const int TN = (p.N + 127) / 128, TK = (p.K + C::BN - 1) / C::BN;
  const long long total = bad ? 0 : (long long)p.E * TN * TK;

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = policy_evict_normal();
      uint32_t armed = 0, parity = 0;
      bool ok = true;
      int it = 0;
      for (long long u = blockIdx.x; u < total && ok; u += gridDim.x) {
        const int e = (int)(u / (TN * TK)), r = (int)(u % (TN * TK));
        const int n0 = (r % TN) * 128, k0 = (r / TN) * C::BN;
        const int lo = p.offsets[e], hi = p.offsets[e + 1];
        for (int row = lo; row < hi; row += C::CH, ++it) {
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
#pragma unroll
          for (int b = 0; b < C::NA; ++b) tma_load_2d(&tmY, &full[st], a + b * C::BOX, n0 + 64 * b, row, pol);
#pragma unroll
          for (int b = 0; b < C::NB; ++b)
            tma_load_2d(&tmX, &full[st], a + (C::NA + b) * C::BOX, k0 + 64 * b, row, pol);
        }
      }
      if (*abort)
        for (int s = 0; s < STAGES; ++s)
          if (armed & (1u << s)) mbar_drain(&full[s], (parity >> s) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    bool ok = true;
    int it = 0, j = 0;
    for (long long u = blockIdx.x; u < total && ok; u += gridDim.x) {
      const int e = (int)(u / (TN * TK));
      const int lo = p.offsets[e], hi = p.offsets[e + 1];
      if (hi == lo) continue;
      const int buf = j & 1;
      ok = mbar_wait(&tempty[buf], ((uint32_t)(j >> 1) & 1u) ^ 1u, abort);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc_fence_after();
      for (int row = lo; row < hi; row += C::CH, ++it) {
        const int st = it % STAGES;
        ok = mbar_wait(&full[st], (uint32_t)(it / STAGES) & 1u, abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        uint8_t* a = smem + st * C::STAGE;
        const int held = min(C::CH, hi - row), steps = (held + 15) / 16;
        if (held & 15) {
          // The last step's rows past the group's end belong to the next
          // group (or to no one) and may hold anything, NaN too: zeros in
          // both operands.  A row is one 128-byte line of each box, whatever
          // the swizzle does inside it.
          const int lines = steps * 16 - held;
          for (int i = lane; i < lines * 8 * (C::NA + C::NB); i += 32) {
            const int b = i / (lines * 8), in = i % (lines * 8);
            *reinterpret_cast<uint4*>(a + b * C::BOX + held * 128 + in * 16) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        tc_fence_after();
        if (lane == 0) {
          const uint64_t ad = sdesc_mn_sw128(smem_u32(a), C::BOX);
          const uint64_t bd = sdesc_mn_sw128(smem_u32(a + C::NA * C::BOX), C::BOX);
          for (int kk = 0; kk < steps; ++kk)
            mma_f16<1>(tmem + buf * C::BN, ad + 128 * kk, bd + 128 * kk, p.idesc, (row != lo) | (kk != 0));
          mma_commit(&empty[st]);
        }
        __syncwarp();
      }
      if (ok && lane == 0) mma_commit(&tfull[buf]);
      __syncwarp();
      ++j;
    }
    if (lane == 0) mma_commit(done);
    __syncwarp();
    mbar_drain(done, 0);
  } else if (warp >= 4) {
    const int q = warp & 3;
    bool ok = true;
    int j = 0;
    for (long long u = blockIdx.x; u < total && ok; u += gridDim.x) {
      const int e = (int)(u / (TN * TK)), r = (int)(u % (TN * TK));
      const int n = (r % TN) * 128 + q * 32 + lane, k0 = (r / TN) * C::BN;
      const bool empty_group = p.offsets[e + 1] == p.offsets[e];
      const int buf = j & 1;
      if (!empty_group) {
        ok = mbar_wait(&tfull[buf], (uint32_t)(j >> 1) & 1u, abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
      }
      const size_t at = ((size_t)e * p.N + n) * p.K + k0;
#pragma unroll 1
      for (int c0 = 0; c0 < C::BN; c0 += 16) {
        float v[16];
        if (empty_group) {
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] = 0.0f;
        } else {
          tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + buf * C::BN + c0, v);
          tmem_wait_ld();
        }
        if (n >= p.N) continue;
#pragma unroll
        for (int g = 0; g < 16; g += 8) {
          // K is a multiple of 8 (16-bit) or of 4 (fp32): no partial vector
          if (p.out_type == MOE_DT_FP32) {
#pragma unroll
            for (int h = 0; h < 8; h += 4)
              if (k0 + c0 + g + h < p.K)
                *reinterpret_cast<float4*>(static_cast<float*>(p.dw) + at + c0 + g + h) =
                    make_float4(v[g + h], v[g + h + 1], v[g + h + 2], v[g + h + 3]);
          } else if (k0 + c0 + g < p.K) {
            uint32_t w[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) w[h] = pack16(v[g + 2 * h], v[g + 2 * h + 1], p.out_type == MOE_DT_BF16);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dw) + at + c0 + g) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (!empty_group) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[buf]);
        ++j;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
  if (threadIdx.x == 0 && p.status) {
    if (*abort) atomicOr(p.status, DEV_TIMEOUT);
    if (bad) atomicOr(p.status, DEV_BAD_ROUTING);
  }
}

}  // namespace

cudaError_t launch_wgrad(const CUtensorMap& ty, const CUtensorMap& tx, const WgradParams& p0, int sms,
                         cudaStream_t s) {
  WgradParams p = p0;
  p.idesc = idesc_f16(128, WCfg::BN, p.fmt, 1, 1);
  return launch_cluster(wgrad_kernel, sms, WCfg::THREADS, WCfg::SMEM, 1, s, ty, tx, p);
}

}  // namespace moe
