// moe_rows.cu -- rows between token order and expert order: copies, the
// weighted combination with its gradients, and 8-bit quantisation of rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_ops.h"

namespace moe {
namespace {

__device__ __forceinline__ long long slot_token(const SlotMap& m, int pos) {
  if (!m.perm) return pos < m.T ? pos : -1;
  const long long s = m.perm[pos], S = (long long)m.T * m.k;
  if (s < 0) return -1;
  if (s < S) return s / m.k;
  return s - S < m.T ? s - S : -1;
}

template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<__half> {
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <> struct Elem<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};

// 16 bytes of a row starting at element c, as floats; elements past n are
// zero and never read.  Rows are 16-byte aligned and c a multiple of VN.
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  float v[N];
  __device__ __forceinline__ void load(const T* row, int c, int n) {
    if (c + N <= n) {
      const uint4 raw = *reinterpret_cast<const uint4*>(row + c);
      const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = Elem<T>::get(e[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = c + i < n ? Elem<T>::get(row[c + i]) : 0.0f;
    }
  }
  __device__ __forceinline__ void store(T* row, int c, int n) const {
    if (c + N <= n) {
      uint4 raw;
      T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = Elem<T>::put(v[i]);
      *reinterpret_cast<uint4*>(row + c) = raw;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c + i < n) row[c + i] = Elem<T>::put(v[i]);
    }
  }
};

// ---- permute: y[p] = x[token(p)] ------------------------------------------------
constexpr int kPermThreads = 256;
__global__ void __launch_bounds__(kPermThreads) permute_kernel(const PermuteParams p) {
  for (int pos = blockIdx.x; pos < p.rows; pos += gridDim.x) {
    const long long t = slot_token(p.map, pos);
    if (t < 0) continue;
    const char* src = static_cast<const char*>(p.x) + t * p.ldx;
    char* dst = static_cast<char*>(p.y) + (long long)pos * p.ldy;
    const long long whole = p.row_bytes & ~15LL;
    for (long long i = threadIdx.x * 16LL; i < whole; i += kPermThreads * 16LL)
      *reinterpret_cast<uint4*>(dst + i) = *reinterpret_cast<const uint4*>(src + i);
    for (long long i = whole + threadIdx.x; i < p.row_bytes; i += kPermThreads) dst[i] = src[i];
  }
}

// ---- combine: out[t] = sum_j g[t, j] y[inv[t, j]] (+ the shared expert's row) --
constexpr int kCombThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kCombThreads) combine_kernel(const RowCombineParams p) {
  __shared__ int pos[kMaxCombine];
  __shared__ float wt[kMaxCombine];
  const int t = blockIdx.x;
  const int n = p.k + p.n_shared;
  if (threadIdx.x < n) {
    const int j = threadIdx.x;
    const bool routed = j < p.k;
    pos[j] = p.inv[routed ? (size_t)t * p.k + j : (size_t)p.T * p.k + t];
    wt[j] = routed && p.g ? p.g[(size_t)t * p.k + j] : 1.0f;
  }
  __syncthreads();
  T* out = static_cast<T*>(p.out) + t * p.ldo;
  for (int c = threadIdx.x * Vec<T>::N; c < p.H; c += kCombThreads * Vec<T>::N) {
    Vec<T> acc;
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) acc.v[i] = 0.0f;
    for (int j = 0; j < n; ++j) {
      if (pos[j] < 0 || pos[j] >= p.rows) continue;
      Vec<T> y;
      y.load(static_cast<const T*>(p.y) + pos[j] * p.ldy, c, p.H);
#pragma unroll
      for (int i = 0; i < Vec<T>::N; ++i) acc.v[i] = fmaf(wt[j], y.v[i], acc.v[i]);
    }
    acc.store(out, c, p.H);
  }
}

// ---- its gradients: a warp per slot ----------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kCombThreads) combine_bwd_kernel(const RowCombineBwdParams p) {
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = p.k + p.n_shared;
  const T* dout = static_cast<const T*>(p.dout) + t * p.ldd;
  for (int j = warp; j < n; j += kCombThreads / 32) {
    const bool routed = j < p.k;
    const size_t slot = routed ? (size_t)t * p.k + j : (size_t)p.T * p.k + t;
    const int pos = p.inv[slot];
    const bool held = pos >= 0 && pos < p.rows;
    float dot = 0.0f;
    if (held) {
      const float g = routed ? p.g[slot] : 1.0f;
      const T* y = static_cast<const T*>(p.y) + pos * p.ldy;
      T* dy = static_cast<T*>(p.dy) + pos * p.lddy;
      for (int c = lane * Vec<T>::N; c < p.H; c += 32 * Vec<T>::N) {
        Vec<T> d, v;
        d.load(dout, c, p.H);
        if (routed) v.load(y, c, p.H);
#pragma unroll
        for (int i = 0; i < Vec<T>::N; ++i) {
          if (routed) dot = fmaf(d.v[i], v.v[i], dot);
          d.v[i] *= g;
        }
        d.store(dy, c, p.H);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
    if (routed && lane == 0) p.dg[slot] = dot;
  }
}

// ---- row quantisation ---------------------------------------------------------------
constexpr int kQ8Threads = 256;
template <typename T>
__global__ void __launch_bounds__(kQ8Threads) quant_int8_kernel(const QuantInt8Params p) {
  __shared__ float red[kQ8Threads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int pos = blockIdx.x; pos < p.rows; pos += gridDim.x) {
    const long long t = slot_token(p.map, pos);
    if (t < 0) continue;
    const T* x = static_cast<const T*>(p.x) + t * p.ldx;
    int8_t* q = p.q + (long long)pos * p.ldq;
    float amax = 0.0f;
    for (int c = threadIdx.x; c < p.K; c += kQ8Threads) {
      const float a = fabsf(Elem<T>::get(x[c]));
      amax = a <= 3.402823466e38f ? fmaxf(amax, a) : __int_as_float(0x7F800000);  // NaN counts as infinite
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if (lane == 0) red[warp] = amax;
    __syncthreads();
    for (int w = 0; w < kQ8Threads / 32; ++w) amax = fmaxf(amax, red[w]);
    __syncthreads();
    const bool finite = amax <= 3.402823466e38f;
    const float pre = amax > 1e30f ? 5.421010862e-20f : 1.0f;  // 2^-64: 127 times the largest bf16 overflows
    for (int c = threadIdx.x; c < p.K; c += kQ8Threads) {
      const float v = Elem<T>::get(x[c]);
      q[c] = (finite && amax > 0.0f) ? (int8_t)__float2int_rn(__fdiv_rn(v * pre * 127.0f, amax * pre)) : (int8_t)0;
    }
    if (threadIdx.x == 0)
      p.s[pos] = !finite ? __int_as_float(0x7FC00000) : amax == 0.0f ? 1.0f : __fdiv_rn(amax, 127.0f);
  }
}

}  // namespace

cudaError_t launch_permute(const PermuteParams& p, cudaStream_t s) {
  permute_kernel<<<p.rows, kPermThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_row_combine(const RowCombineParams& p, int dtype, cudaStream_t s) {
  if (dtype == MOE_DT_BF16) combine_kernel<__nv_bfloat16><<<p.T, kCombThreads, 0, s>>>(p);
  else if (dtype == MOE_DT_FP16) combine_kernel<__half><<<p.T, kCombThreads, 0, s>>>(p);
  else combine_kernel<float><<<p.T, kCombThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_row_combine_bwd(const RowCombineBwdParams& p, int dtype, cudaStream_t s) {
  if (dtype == MOE_DT_BF16) combine_bwd_kernel<__nv_bfloat16><<<p.T, kCombThreads, 0, s>>>(p);
  else if (dtype == MOE_DT_FP16) combine_bwd_kernel<__half><<<p.T, kCombThreads, 0, s>>>(p);
  else combine_bwd_kernel<float><<<p.T, kCombThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_quant_int8(const QuantInt8Params& p, int dtype, cudaStream_t s) {
  if (dtype == MOE_DT_BF16) quant_int8_kernel<__nv_bfloat16><<<p.rows, kQ8Threads, 0, s>>>(p);
  else quant_int8_kernel<__half><<<p.rows, kQ8Threads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
