// moe_ops.h -- parameter blocks and launchers of the expert operators
// (ragged grouped products, int8 products, row movement), shared by their
// translation units (not part of the public C ABI).
#pragma once

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
};

struct WgradParams {
  int E, P, N, K;
  const int32_t* offsets;
  void* dw;                 // [E, N, K]
  int out_type, fmt;
  int32_t* status;
  uint32_t idesc;
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

// How a call is tiled: rows of one tile (the rows side of the MMA), and CTAs
// that work on a tile together.  tx has boxes of rows / ctas rows, txs of 32.
struct GroupedTile {
  int rows, ctas;
};
GroupedTile grouped_tile(const GroupedParams& p);
cudaError_t launch_grouped(int kind, GroupedTile t, const CUtensorMap& tw, const CUtensorMap& tx,
                           const CUtensorMap& txs, const GroupedParams& p, int sms, cudaStream_t s);
cudaError_t launch_wgrad(const CUtensorMap& ty, const CUtensorMap& tx, const WgradParams& p, int sms, cudaStream_t s);
cudaError_t launch_quant_int8(const QuantInt8Params& p, int dtype, cudaStream_t s);
cudaError_t launch_permute(const PermuteParams& p, cudaStream_t s);
cudaError_t launch_row_combine(const RowCombineParams& p, int dtype, cudaStream_t s);
cudaError_t launch_row_combine_bwd(const RowCombineBwdParams& p, int dtype, cudaStream_t s);

}  // namespace moe
