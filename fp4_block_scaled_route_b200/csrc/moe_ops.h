// moe_ops.h -- parameter blocks and launchers of the expert operators
// (ragged grouped products, int8 products, row movement), shared by their
// translation units (not part of the public C ABI).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "moe.h"

namespace moe {

constexpr int kMaxCombine = 33;  // largest top-k plus a shared expert

enum { GG_FWD = 0, GG_DGRAD = 1, GG_INT8 = 2 };

struct GroupedParams {
  int E, P;                 // groups, rows
  int M, R;                 // output features, contraction length
  const int32_t* offsets;   // [E + 1] (null: one group of all rows)
  void* y;                  // [P, M] row stride ldy
  long long ldy;
  int out_type;             // MOE_DT_*
  int fmt;                  // 16-bit operands: 0 fp16, 1 bf16
  const float* row_scale;   // int8: [P]
  const float* col_scale;   // int8: [E, M]
  int32_t* status;
  int stream_w;             // weights are read about once: leave the L2 to the rows
  uint32_t idesc;
  int split;                // CTAs that share a tile's contraction
  int hand_out, teams;      // pairs: units are handed out at run time to so many pairs
};

struct WgradParams {
  int E, P, N, K;
  const int32_t* offsets;
  const uint16_t* dy;       // [P, N], row stride lddy
  const uint16_t* x;        // [P, K], row stride ldx
  long long lddy, ldx;
  void* dw;                 // [E, N, K]
  int out_type, fmt;
  int32_t* status;
  uint32_t idesc;
  int split;                // pairs that share a tile's rows
};

// Token of a routing slot: t * k + j for routed slots, T * k + t for the
// shared expert's; -1 outside.
struct SlotMap {
  const int32_t* perm;      // position -> slot (null: position = token)
  int T, k;
};

struct QuantInt8Params {
  int rows, K;
  const void* x;            // [T, K], row stride ldx
  long long ldx;
  int8_t* q;                // [rows, K], row stride ldq
  long long ldq;
  float* s;                 // [rows]
  SlotMap map;
};

struct PermuteParams {
  int rows;
  long long row_bytes, ldx, ldy;  // bytes
  const void* x;
  void* y;
  SlotMap map;
};

struct RowCombineParams {
  int T, k, n_shared, H, rows;
  const void* y;            // [rows, H], row stride ldy
  long long ldy;
  const int32_t* inv;       // [T*k + n_shared*T]
  const float* g;           // [T, k] (null: ones)
  void* out;                // [T, H], row stride ldo
  long long ldo;
};

struct RowCombineBwdParams {
  int T, k, n_shared, H, rows;
  const void* dout;         // [T, H], row stride ldd
  long long ldd;
  const void* y;            // [rows, H], row stride ldy
  long long ldy;
  const int32_t* inv;
  const float* g;
  void* dy;                 // [rows, H], row stride lddy
  long long lddy;
  float* dg;                // [T, k]
};

// How a call is tiled: rows of one tile (the rows side of the MMA), CTAs of
// one MMA, CTAs that share a tile's contraction, CTAs in all and at one time.  tx has boxes
// of rows / ctas rows; txs, of 32, is used by pairs only.
struct GroupedTile {
  int rows, ctas, split, grid, running;
};
GroupedTile grouped_tile(const GroupedParams& p, int kind, int sms);
cudaError_t launch_grouped(int kind, GroupedTile t, const CUtensorMap& tw, const CUtensorMap& tx,
                           const CUtensorMap& txs, const GroupedParams& p, cudaStream_t s);
// ty, tx: boxes of 64 rows; ty16, tx16: of 16; to: dw [E][N][K] with boxes of 32.
cudaError_t launch_wgrad(const CUtensorMap& ty, const CUtensorMap& tx, const CUtensorMap& to, const CUtensorMap& ty16,
                         const CUtensorMap& tx16, const WgradParams& p, int sms, cudaStream_t s);
cudaError_t launch_quant_int8(const QuantInt8Params& p, int dtype, cudaStream_t s);
cudaError_t launch_permute(const PermuteParams& p, cudaStream_t s);
cudaError_t launch_row_combine(const RowCombineParams& p, int dtype, cudaStream_t s);
cudaError_t launch_row_combine_bwd(const RowCombineBwdParams& p, int dtype, cudaStream_t s);

// Clusters of `size` CTAs, one CTA per SM, that are resident at once: the SMs
// of a GPC do not all fit clusters of 4 and 8 (B200, 148 SMs, as the occupancy
// query gives it: 74 of 2, 33 of 4, 15 of 8).
inline int resident_clusters(int size, int sms) {
  return size <= 2 ? sms / size : size <= 4 ? sms * 33 / 148 : sms * 15 / 148;
}

// Launch as a programmatic dependent of the kernel before it in the stream
// (the kernels wait, before they read anything, until that one is complete),
// in clusters of `cluster` CTAs.
template <auto Kernel, typename... Args>
cudaError_t launch_cluster(dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s, const Args&... args) {
  if (smem > 48 * 1024) {
    // once per kernel and device: the attribute belongs to the device's context
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(done.load(std::memory_order_relaxed) & bit)) {
      e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
      if (e != cudaSuccess) return e;
      done.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, Kernel, args...);
}

}  // namespace moe
