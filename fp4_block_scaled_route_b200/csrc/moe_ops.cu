// moe_ops.cu -- C ABI of the expert operators (include/moe.h): argument
// checks, tensor maps and launches.  None of them keeps state: no workspace,
// no allocation, nothing cached between calls, but for a word per device that
// collects the errors of calls without a status word of their own.
#include <cuda.h>
#include <cuda_runtime.h>

#include "moe.h"
#include "moe_internal.h"
#include "moe_ops.h"
#include "moe_ptx.cuh"

namespace {

__device__ int32_t g_status, g_taken;  // errors since they were last taken; what was taken

__global__ void take_status_kernel() { g_taken = atomicExch(&g_status, 0); }

using moe::GroupedParams;

constexpr long long kMaxRows = 1LL << 24;  // a weight-gradient tile walks all rows within a bounded wait
constexpr int kMaxDim = 1 << 20;
constexpr long long kMaxStrideBytes = 1LL << 40;  // TMA's limit

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Map with 128-byte swizzle over [planes][rows][inner] (planes = 0: two
// dimensions), boxes of 128 bytes by box_rows rows; what lies outside reads
// as zero.
bool make_map(CUtensorMap* m, CUtensorMapDataType dt, int es, const void* base, uint64_t inner, uint64_t rows,
              uint64_t row_stride, uint64_t planes, uint64_t plane_stride, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dim[3] = {inner, rows, planes};
  cuuint64_t stride[2] = {row_stride * es, plane_stride * es};
  cuuint32_t box[3] = {(cuuint32_t)(128 / es), box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, dt, planes ? 3 : 2, const_cast<void*>(base), dim, stride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int elem_size(int dtype) {
  return dtype == MOE_DT_BF16 || dtype == MOE_DT_FP16 ? 2 : dtype == MOE_DT_FP32 ? 4 : 0;
}

bool is16(int dtype) { return dtype == MOE_DT_BF16 || dtype == MOE_DT_FP16; }

CUtensorMapDataType map_type(int dtype) {
  return dtype == MOE_DT_BF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
         : dtype == MOE_DT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
}

// A row stride in elements: at least the row, a multiple of 16 bytes, within TMA's limit.
bool row_stride_ok(long long ld, long long n, int es) {
  return ld >= n && ld < kMaxStrideBytes / es && ld * es % 16 == 0;
}

// The current device's SM count; MOE_ERR_UNSUPPORTED when it is no sm_100.
moe_status device_sms(int* sms) {
  static std::atomic<int> known[64];  // SM count of a usable device, 0: not asked yet
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) != 0) return MOE_OK;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (major != 10) return MOE_ERR_UNSUPPORTED;
  if (dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return MOE_OK;
}

// Where a call's kernels report: the caller's word, or that of the current
// device's context (35 ns to find, so it is not kept).
moe_status status_word(int32_t** d_status) {
  if (*d_status) return MOE_OK;
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess) return MOE_ERR_CUDA;
  *d_status = static_cast<int32_t*>(p);
  return MOE_OK;
}

moe_status sizes_ok(int E, int P, int N, int K) {
  if (E < 1 || P < 0 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  if (E > 1024 || P > kMaxRows || N > kMaxDim || K > kMaxDim) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Weights [E, N, K]: rows ldw elements apart, groups stride_w apart.
moe_status weights_ok(int E, int N, int K, const void* w, long long ldw, long long stride_w, int es) {
  if (!w || !aligned(w, 16) || !row_stride_ok(ldw, K, es)) return MOE_ERR_INVALID_ARG;
  if (E > 1 && (!row_stride_ok(stride_w, (long long)(N - 1) * ldw + K, es))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status run_grouped(int kind, int dtype, int out_dtype, int E, int P, int N, int K, const int32_t* offsets,
                       const void* x, long long ldx, const float* row_scale, const void* w, long long ldw,
                       long long stride_w, const float* col_scale, void* y, long long ldy, int32_t* d_status,
                       void* stream) {
  const bool i8 = kind == moe::GG_INT8;
  const int es = i8 ? 1 : 2;
  const int M = kind == moe::GG_DGRAD ? K : N, R = kind == moe::GG_DGRAD ? N : K;
  const moe_status st = sizes_ok(E, P, N, K);
  if (st != MOE_OK) return st;
  if (P == 0) return MOE_OK;
  if (!x || !y || !aligned(x, 16) || !aligned(y, 16) || !row_stride_ok(ldx, R, es) ||
      !row_stride_ok(ldy, M, elem_size(out_dtype)))
    return MOE_ERR_INVALID_ARG;
  const moe_status ws = weights_ok(E, N, K, w, ldw, stride_w, es);
  if (ws != MOE_OK) return ws;
  if ((!offsets && !(i8 && E == 1)) || !aligned(offsets, 4) || !aligned(d_status, 4)) return MOE_ERR_INVALID_ARG;
  int sms = 0;
  const moe_status ds = device_sms(&sms);
  if (ds != MOE_OK) return ds;
  const moe_status sw = status_word(&d_status);
  if (sw != MOE_OK) return sw;
  GroupedParams p{};
  p.E = E; p.P = P; p.M = M; p.R = R;
  p.offsets = offsets;
  p.y = y; p.ldy = ldy; p.out_type = out_dtype;
  p.fmt = dtype == MOE_DT_BF16 ? 1 : 0;
  p.row_scale = row_scale; p.col_scale = col_scale;
  p.status = d_status;
  const moe::GroupedTile t = moe::grouped_tile(p, kind, sms);
  p.stream_w = t.rows < 256;
  CUtensorMap tw, tx, txs{};
  const CUtensorMapDataType dt = i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : map_type(dtype);
  if (!make_map(&tw, dt, es, w, K, N, ldw, E, E > 1 ? stride_w : (long long)N * ldw, kind == moe::GG_DGRAD ? 64 : 128) ||
      !make_map(&tx, dt, es, x, R, P, ldx, 0, 0, t.rows / t.ctas) ||
      (t.ctas > 1 && !make_map(&txs, dt, es, x, R, P, ldx, 0, 0, 32)))
    return MOE_ERR_CUDA;
  return moe::launch_grouped(kind, t, tw, tx, txs, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                                      : MOE_ERR_CUDA;
}

}  // namespace

extern "C" {

moe_status moe_grouped_gemm(int dtype, int out_dtype, int E, int P, int N, int K, const int32_t* offsets,
                            const void* x, long long ldx, const void* w, long long ldw, long long stride_w, void* y,
                            long long ldy, int32_t* d_status, void* stream) {
  if (!is16(dtype) || (out_dtype != dtype && out_dtype != MOE_DT_FP32)) return MOE_ERR_UNSUPPORTED;
  return run_grouped(moe::GG_FWD, dtype, out_dtype, E, P, N, K, offsets, x, ldx, nullptr, w, ldw, stride_w, nullptr, y,
                     ldy, d_status, stream);
}

moe_status moe_grouped_gemm_dgrad(int dtype, int out_dtype, int E, int P, int N, int K, const int32_t* offsets,
                                  const void* dy, long long lddy, const void* w, long long ldw, long long stride_w,
                                  void* dx, long long lddx, int32_t* d_status, void* stream) {
  if (!is16(dtype) || (out_dtype != dtype && out_dtype != MOE_DT_FP32)) return MOE_ERR_UNSUPPORTED;
  return run_grouped(moe::GG_DGRAD, dtype, out_dtype, E, P, N, K, offsets, dy, lddy, nullptr, w, ldw, stride_w, nullptr,
                     dx, lddx, d_status, stream);
}

moe_status moe_grouped_gemm_wgrad(int dtype, int out_dtype, int E, int P, int N, int K, const int32_t* offsets,
                                  const void* dy, long long lddy, const void* x, long long ldx, void* dw,
                                  int32_t* d_status, void* stream) {
  if (!is16(dtype) || (out_dtype != dtype && out_dtype != MOE_DT_FP32)) return MOE_ERR_UNSUPPORTED;
  const moe_status st = sizes_ok(E, P, N, K);
  if (st != MOE_OK) return st;
  const int oes = elem_size(out_dtype);
  if (!dw || !aligned(dw, 16) || !row_stride_ok(K, K, oes)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (P == 0)  // every sum is empty
    return cudaMemsetAsync(dw, 0, (size_t)E * N * K * oes, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  if (!offsets || !dy || !x || !aligned(offsets, 4) || !aligned(dy, 16) || !aligned(x, 16) ||
      !row_stride_ok(lddy, N, 2) || !row_stride_ok(ldx, K, 2) || !aligned(d_status, 4))
    return MOE_ERR_INVALID_ARG;
  int sms = 0;
  const moe_status ds = device_sms(&sms);
  if (ds != MOE_OK) return ds;
  if ((long long)E * ((N + 255) / 256) * ((K + 255) / 256) > (1LL << 30)) return MOE_ERR_UNSUPPORTED;
  const moe_status sw = status_word(&d_status);
  if (sw != MOE_OK) return sw;
  moe::WgradParams p{};
  p.E = E; p.P = P; p.N = N; p.K = K;
  p.offsets = offsets;
  p.dw = dw; p.out_type = out_dtype;
  p.fmt = dtype == MOE_DT_BF16 ? 1 : 0;
  p.status = d_status;
  p.dy = static_cast<const uint16_t*>(dy); p.lddy = lddy;
  p.x = static_cast<const uint16_t*>(x); p.ldx = ldx;
  CUtensorMap ty, tx, to, ty16, tx16;
  if (!make_map(&ty, map_type(dtype), 2, dy, N, P, lddy, 0, 0, 64) ||
      !make_map(&tx, map_type(dtype), 2, x, K, P, ldx, 0, 0, 64) ||
      !make_map(&ty16, map_type(dtype), 2, dy, N, P, lddy, 0, 0, 16) ||
      !make_map(&tx16, map_type(dtype), 2, x, K, P, ldx, 0, 0, 16) ||
      !make_map(&to, map_type(out_dtype), oes, dw, K, N, K, E, (long long)N * K, 32))
    return MOE_ERR_CUDA;
  return moe::launch_wgrad(ty, tx, to, ty16, tx16, p, sms, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_ops_status(void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  take_status_kernel<<<1, 1, 0, s>>>();
  int32_t v = 0;
  if (cudaGetLastError() != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess ||
      cudaMemcpyFromSymbol(&v, g_taken, sizeof(v)) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (v & moe::DEV_TIMEOUT) return MOE_ERR_TIMEOUT;
  return v & moe::DEV_BAD_ROUTING ? MOE_ERR_BAD_ROUTING : MOE_OK;
}

moe_status moe_int8_gemm(int out_dtype, int E, int P, int N, int K, const int32_t* offsets, const int8_t* q,
                         long long ldq, const float* q_scale, const int8_t* w, long long ldw, long long stride_w,
                         const float* w_scale, void* y, long long ldy, int32_t* d_status, void* stream) {
  if (!elem_size(out_dtype)) return MOE_ERR_UNSUPPORTED;
  // |sum| <= 128 * 128 * K stays below 2^31
  if (K > 131071) return MOE_ERR_UNSUPPORTED;
  if (P > 0 && (!q_scale || !w_scale || !aligned(q_scale, 4) || !aligned(w_scale, 4))) return MOE_ERR_INVALID_ARG;
  return run_grouped(moe::GG_INT8, 0, out_dtype, E, P, N, K, offsets, q, ldq, q_scale, w, ldw, stride_w, w_scale, y,
                     ldy, d_status, stream);
}

moe_status moe_quant_int8(int dtype, int rows, int K, int T, int k, const void* x, long long ldx, const int32_t* perm,
                          int8_t* q, long long ldq, float* scale, void* stream) {
  if (!is16(dtype)) return MOE_ERR_UNSUPPORTED;
  if (rows < 0 || T < 0 || k < 1 || K < 1 || (!perm && rows > T)) return MOE_ERR_INVALID_ARG;
  if (rows > kMaxRows || T > kMaxRows || k > moe::kMaxK || K > kMaxDim) return MOE_ERR_UNSUPPORTED;
  if (rows == 0 || T == 0) return MOE_OK;
  if (!x || !q || !scale || !aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4) || !aligned(perm, 4) ||
      !row_stride_ok(ldx, K, 2) || !row_stride_ok(ldq, K, 1))
    return MOE_ERR_INVALID_ARG;
  moe::QuantInt8Params p{rows, K, x, ldx, q, ldq, scale, {perm, T, k}};
  return moe::launch_quant_int8(p, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_permute(int dtype, int rows, int H, int T, int k, const void* x, long long ldx, const int32_t* perm,
                       void* y, long long ldy, void* stream) {
  const int es = elem_size(dtype);
  if (!es) return MOE_ERR_UNSUPPORTED;
  if (rows < 0 || T < 0 || k < 1 || H < 1) return MOE_ERR_INVALID_ARG;
  if (rows > kMaxRows || T > kMaxRows || k > moe::kMaxK || H > kMaxDim) return MOE_ERR_UNSUPPORTED;
  if (rows == 0 || T == 0) return MOE_OK;
  if (!x || !perm || !y || !aligned(x, 16) || !aligned(perm, 4) || !aligned(y, 16) || !row_stride_ok(ldx, H, es) ||
      !row_stride_ok(ldy, H, es))
    return MOE_ERR_INVALID_ARG;
  moe::PermuteParams p{rows, (long long)H * es, ldx * es, ldy * es, x, y, {perm, T, k}};
  return moe::launch_permute(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_combine(int dtype, int rows, int H, int T, int k, int n_shared, const void* y, long long ldy,
                       const int32_t* inv, const float* topk_w, void* out, long long ldo, void* stream) {
  const int es = elem_size(dtype);
  if (!es) return MOE_ERR_UNSUPPORTED;
  if (rows < 0 || T < 0 || k < 1 || H < 1 || n_shared < 0) return MOE_ERR_INVALID_ARG;
  if (rows > kMaxRows || T > kMaxRows || k > moe::kMaxK || H > kMaxDim || n_shared > 1) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if ((rows > 0 && !y) || !inv || !out || !aligned(y, 16) || !aligned(inv, 4) || !aligned(topk_w, 4) ||
      !aligned(out, 16) || (rows > 0 && !row_stride_ok(ldy, H, es)) || !row_stride_ok(ldo, H, es))
    return MOE_ERR_INVALID_ARG;
  moe::RowCombineParams p{T, k, n_shared, H, rows, y, ldy, inv, topk_w, out, ldo};
  return moe::launch_row_combine(p, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_combine_backward(int dtype, int rows, int H, int T, int k, int n_shared, const void* dout,
                                long long lddout, const void* y, long long ldy, const int32_t* inv,
                                const float* topk_w, void* dy, long long lddy, float* dtopk_w, void* stream) {
  const int es = elem_size(dtype);
  if (!es) return MOE_ERR_UNSUPPORTED;
  if (rows < 0 || T < 0 || k < 1 || H < 1 || n_shared < 0) return MOE_ERR_INVALID_ARG;
  if (rows > kMaxRows || T > kMaxRows || k > moe::kMaxK || H > kMaxDim || n_shared > 1) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!dout || !inv || !topk_w || !dtopk_w || !aligned(dout, 16) || !aligned(inv, 4) || !aligned(topk_w, 4) ||
      !aligned(dtopk_w, 4) || !row_stride_ok(lddout, H, es))
    return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!y || !dy || !aligned(y, 16) || !aligned(dy, 16) || !row_stride_ok(ldy, H, es) ||
                   !row_stride_ok(lddy, H, es)))
    return MOE_ERR_INVALID_ARG;
  moe::RowCombineBwdParams p{T, k, n_shared, H, rows, dout, lddout, y, ldy, inv, topk_w, dy, lddy, dtopk_w};
  return moe::launch_row_combine_bwd(p, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                               : MOE_ERR_CUDA;
}

}  // extern "C"
