// moe_rows.cu -- rows between token order and expert order: copies, the
// weighted combination with its gradients, and 8-bit quantisation of rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "moe_ops.h"
#include "moe_ptx.cuh"

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
      __stcs(reinterpret_cast<uint4*>(row + c), raw);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c + i < n) row[c + i] = Elem<T>::put(v[i]);
    }
  }
};

constexpr int kThreads = 256;

// ---- permute: y[p] = x[token(p)] ------------------------------------------------
// W warps copy a row, each thread up to kCopies pieces of 16 bytes that are
// all loaded before the first is stored.  4096 tokens of 7168 bf16 to 32768
// rows take 104 (in token order) to 116 us on B200, 4.1 to 4.5 TB/s written,
// with DRAM 68 % busy and the L2 47 %; a fill of as many bytes takes 66.
constexpr int kCopies = 4;
template <int W>
__global__ void __launch_bounds__(kThreads) permute_kernel(const PermuteParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int sub = threadIdx.x / (32 * W), i0 = threadIdx.x % (32 * W);
  const long long pos = (long long)blockIdx.x * (kThreads / 32 / W) + sub;
  if (pos >= p.rows) return;
  const long long t = slot_token(p.map, (int)pos);
  if (t < 0) return;
  const char* src = static_cast<const char*>(p.x) + t * p.ldx;
  char* dst = static_cast<char*>(p.y) + pos * p.ldy;
  const long long whole = p.row_bytes & ~15LL;
  for (long long base = (long long)blockIdx.y * (512 * W * kCopies); base < whole;
       base += (long long)gridDim.y * (512 * W * kCopies)) {
    uint4 v[kCopies];
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const long long at = base + (c * 32 * W + i0) * 16LL;
      if (at < whole) v[c] = __ldg(reinterpret_cast<const uint4*>(src + at));
    }
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const long long at = base + (c * 32 * W + i0) * 16LL;
      if (at < whole) __stcs(reinterpret_cast<uint4*>(dst + at), v[c]);
    }
  }
  if (blockIdx.y == 0)
    for (long long i = whole + i0; i < p.row_bytes; i += 32 * W) dst[i] = src[i];
}

// 16 bytes of a row as loaded, to be unpacked later: several of them can be
// in flight at a small cost in registers.
template <typename T>
struct Raw {
  uint4 u;
  __device__ __forceinline__ void load(const T* row, int c, int n) {
    if (c + Vec<T>::N <= n) {
      u = __ldcs(reinterpret_cast<const uint4*>(row + c));
    } else {
      T e[Vec<T>::N];
#pragma unroll
      for (int i = 0; i < Vec<T>::N; ++i) e[i] = c + i < n ? row[c + i] : Elem<T>::put(0.0f);
      u = *reinterpret_cast<const uint4*>(e);
    }
  }
  __device__ __forceinline__ float get(int i) const { return Elem<T>::get(reinterpret_cast<const T*>(&u)[i]); }
};

// ---- combine: out[t] = sum_j g[t, j] y[inv[t, j]] (+ the shared expert's row) --
// One block per token and 256 pieces of 16 bytes of its columns; the rows of
// J slots are loaded together, all of them up to 4 (4096 tokens of 7168 bf16 on
// B200, 8 slots: one by one 95 us, 2 together 93, 4 together 88, 6.0 TB/s, 8
// together 97; 2 slots: 36 with J = 2, 40 with 4; 1 slot: 24 with 1, 33 with 4).
template <typename T, int J>
__global__ void __launch_bounds__(kThreads) combine_kernel(const RowCombineParams p) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int pos[kMaxCombine];
  __shared__ float wt[kMaxCombine];
  __shared__ int s_n;
  const int t = blockIdx.x;
  if (threadIdx.x < 32) {
    // the held slots in ascending order, closed up; lane 0 adds the shared expert's row
    const int j = threadIdx.x;
    int at = j < p.k ? p.inv[(size_t)t * p.k + j] : -1;
    const float g = j < p.k && p.g ? p.g[(size_t)t * p.k + j] : 1.0f;
    if (at >= p.rows) at = -1;
    const unsigned held = __ballot_sync(0xFFFFFFFFu, at >= 0);
    if (at >= 0) {
      const int i = __popc(held & ((1u << j) - 1u));
      pos[i] = at;
      wt[i] = g;
    }
    if (j == 0) {
      int n = __popc(held);
      if (p.n_shared) {
        const int sh = p.inv[(size_t)p.T * p.k + t];
        if (sh >= 0 && sh < p.rows) {
          pos[n] = sh;
          wt[n++] = 1.0f;
        }
      }
      s_n = n;
    }
  }
  __syncthreads();
  const int n = s_n;
  T* out = static_cast<T*>(p.out) + t * p.ldo;
  const T* y = static_cast<const T*>(p.y);
  for (int c = (blockIdx.y * kThreads + threadIdx.x) * Vec<T>::N; c < p.H; c += gridDim.y * kThreads * Vec<T>::N) {
    Vec<T> acc;
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) acc.v[i] = 0.0f;
    for (int j = 0; j < n; j += J) {
      Raw<T> r[J];
#pragma unroll
      for (int q = 0; q < J; ++q)
        if (j + q < n) r[q].load(y + pos[j + q] * p.ldy, c, p.H);
#pragma unroll
      for (int q = 0; q < J; ++q)
        if (j + q < n) {
          const float g = wt[j + q];
#pragma unroll
          for (int i = 0; i < Vec<T>::N; ++i) acc.v[i] = fmaf(g, r[q].get(i), acc.v[i]);
        }
    }
    acc.store(out, c, p.H);
  }
}

// ---- its gradients: W warps per slot ----------------------------------------------
// One piece of 16 bytes per thread and pass: with four in flight (and a
// quarter of the warps) 32768 slots of 7168 values took 260 us on B200, with
// two 224, with one 184 (5.4 TB/s).
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) combine_bwd_kernel(const RowCombineBwdParams p) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float part[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long S = (long long)p.T * p.k, slots = S + (long long)p.n_shared * p.T;
  const long long slot = (long long)blockIdx.x * (kThreads / 32 / W) + warp / W;
  const bool routed = slot < S;
  float dot = 0.0f;
  if (slot < slots) {
    const int pos = p.inv[slot];
    if (pos >= 0 && pos < p.rows) {
      const long long t = routed ? slot / p.k : slot - S;
      const T* dout = static_cast<const T*>(p.dout) + t * p.ldd;
      const float g = routed ? p.g[slot] : 1.0f;
      const T* y = static_cast<const T*>(p.y) + pos * p.ldy;
      T* dy = static_cast<T*>(p.dy) + pos * p.lddy;
      constexpr int N = Vec<T>::N;
      for (int c = ((warp % W) * 32 + lane) * N; c < p.H; c += 32 * W * N) {
        Vec<T> d;
        Raw<T> v;
        if (routed) v.load(y, c, p.H);
        d.load(dout, c, p.H);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (routed) dot = fmaf(d.v[i], v.get(i), dot);
          d.v[i] *= g;
        }
        d.store(dy, c, p.H);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
  if (W > 1) {
    if (lane == 0) part[warp] = dot;
    __syncthreads();
    dot = 0.0f;
    for (int w = 0; w < W; ++w) dot += part[warp / W * W + w];
  }
  if (slot < slots && routed && lane == 0 && warp % W == 0) p.dg[slot] = dot;
}

// ---- row quantisation ---------------------------------------------------------------
// 8 consecutive 16-bit values of a row, zeros past its end.
constexpr int kChunk = 8;
struct Chunk {
  uint32_t w[4];
  __device__ __forceinline__ void load(const uint16_t* row, int c, int n) {
    if (c + kChunk <= n) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(row + c));
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = c + 2 * i < n ? row[c + 2 * i] : 0, hi = c + 2 * i + 1 < n ? row[c + 2 * i + 1] : 0;
        w[i] = lo | hi << 16;
      }
    }
  }
};

// Codes of a chunk's values v of a row with maximum amax: rint(127 v / amax),
// ties to even.  All of it is moved by a power of two, pre, where 127 v or 1 /
// amax would leave fp32's range: scale = 127 pre, top = amax pre, rcp = 1 / top.
// 127 v is exact for a 16-bit type; the first quotient is off by at most 2
// units in the last place, and its remainder brings it to within one.  A tie n + 1/2 is
// a float, so a quotient that is one comes out exactly and rounds to even; any
// other is at least 16 times that error away from one (a maximum of 11 bits).
// Dividing value by value made the kernel twice as slow as its traffic (B200,
// 8192 x 7168 bf16: 54 us).
template <typename T>
__device__ __forceinline__ void codes_int8(const Chunk& v, float scale, float top, float rcp, uint32_t (&o)[2]) {
  uint32_t t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint16_t raw = (uint16_t)(v.w[i / 2] >> (16 * (i & 1)));
    const float f = Elem<T>::get(*reinterpret_cast<const T*>(&raw)) * scale;
    const float q = f * rcp;
    // adding 1.5 * 2^23 rounds to an integer and leaves it in the low byte
    t[i] = __float_as_uint(__fadd_rn(__fmaf_rn(__fmaf_rn(-q, top, f), rcp, q), 12582912.0f));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    o[i] = __byte_perm(__byte_perm(t[4 * i], t[4 * i + 1], 0x0040), __byte_perm(t[4 * i + 2], t[4 * i + 3], 0x0040),
                       0x5410);
}

// W warps per row; a thread keeps its first kKeep chunks between the two
// passes (maximum, codes) and reads the others again.  8192 rows of 7168 bf16:
// 37 to 45 us on B200, 4.8 to 3.9 TB/s.
constexpr int kKeep = 4;
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) quant_int8_kernel(const QuantInt8Params p) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ uint32_t red[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i0 = threadIdx.x % (32 * W);
  const long long pos = (long long)blockIdx.x * (kThreads / 32 / W) + warp / W;
  const long long t = pos < p.rows ? slot_token(p.map, (int)pos) : -1;
  const uint16_t* x = static_cast<const uint16_t*>(p.x) + (t < 0 ? 0 : t) * p.ldx;
  const int K = t < 0 ? 0 : p.K;
  // magnitudes compare as their bits; an infinity or a NaN is above every finite value
  Chunk keep[kKeep];
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if ((i0 + k * 32 * W) * kChunk < K) keep[k].load(x, (i0 + k * 32 * W) * kChunk, K);
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if ((i0 + k * 32 * W) * kChunk < K)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = __vmaxu2(top, keep[k].w[i] & 0x7FFF7FFFu);
  for (int c = (i0 + kKeep * 32 * W) * kChunk; c < K; c += 32 * W * kChunk) {
    Chunk v;
    v.load(x, c, K);
#pragma unroll
    for (int i = 0; i < 4; ++i) top = __vmaxu2(top, v.w[i] & 0x7FFF7FFFu);
  }
  top = max(top & 0xFFFFu, top >> 16);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (W > 1) {
    if (lane == 0) red[warp] = top;
    __syncthreads();
    for (int w = 0; w < W; ++w) top = max(top, red[warp / W * W + w]);
  }
  if (t < 0) return;
  constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
  const bool finite = top < (bf ? 0x7F80u : 0x7C00u);
  const uint16_t top16 = (uint16_t)top;
  const float amax = Elem<T>::get(*reinterpret_cast<const T*>(&top16));
  // near the ends of bf16's range 127 v leaves fp32's: such rows are moved by 2^64
  const float pre = amax > 1e30f ? 0x1p-64f : amax < 1e-30f ? 0x1p64f : 1.0f;
  const bool zero = !finite || amax == 0.0f;
  const float rcp = zero ? 0.0f : __fdiv_rn(1.0f, amax * pre);
  int8_t* q = p.q + pos * p.ldq;
  auto put = [&](const Chunk& v, int c) {
    uint32_t o[2] = {0, 0};
    if (!zero) codes_int8<T>(v, 127.0f * pre, amax * pre, rcp, o);
    if (c + kChunk <= K) {
      *reinterpret_cast<uint2*>(q + c) = make_uint2(o[0], o[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (c + i < K) q[c + i] = (int8_t)(o[i / 4] >> (8 * (i & 3)));
    }
  };
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if ((i0 + k * 32 * W) * kChunk < K) put(keep[k], (i0 + k * 32 * W) * kChunk);
  for (int c = (i0 + kKeep * 32 * W) * kChunk; c < K; c += 32 * W * kChunk) {
    Chunk v;
    v.load(x, c, K);
    put(v, c);
  }
  if (i0 == 0) p.s[pos] = !finite ? __int_as_float(0x7FC00000) : amax == 0.0f ? 1.0f : __fdiv_rn(amax, 127.0f);
}

}  // namespace

namespace {
unsigned blocks(long long n, int per) { return (unsigned)((n + per - 1) / per); }

template <typename T>
cudaError_t quant_int8(const QuantInt8Params& p, cudaStream_t s) {
  // the fewest warps that keep a row in registers
  if (p.K <= 32 * kChunk * kKeep) return launch_cluster<quant_int8_kernel<T, 1>>(blocks(p.rows, 8), kThreads, 0, 1, s, p);
  else if (p.K <= 2 * 32 * kChunk * kKeep) return launch_cluster<quant_int8_kernel<T, 2>>(blocks(p.rows, 4), kThreads, 0, 1, s, p);
  else if (p.K <= 4 * 32 * kChunk * kKeep) return launch_cluster<quant_int8_kernel<T, 4>>(blocks(p.rows, 2), kThreads, 0, 1, s, p);
  else return launch_cluster<quant_int8_kernel<T, 8>>(p.rows, kThreads, 0, 1, s, p);
}

template <typename T>
cudaError_t row_combine(const RowCombineParams& p, cudaStream_t s) {
  const dim3 grid(p.T, blocks(p.H, kThreads * Vec<T>::N));
  switch (p.k + p.n_shared) {
    case 1: return launch_cluster<combine_kernel<T, 1>>(grid, kThreads, 0, 1, s, p);
    case 2: return launch_cluster<combine_kernel<T, 2>>(grid, kThreads, 0, 1, s, p);
    case 3: return launch_cluster<combine_kernel<T, 3>>(grid, kThreads, 0, 1, s, p);
  }
  return launch_cluster<combine_kernel<T, 4>>(grid, kThreads, 0, 1, s, p);
}

template <typename T>
cudaError_t row_combine_bwd(const RowCombineBwdParams& p, cudaStream_t s) {
  const long long slots = (long long)p.T * (p.k + p.n_shared);
  // the fewest warps that take a row in one pass
  constexpr int piece = 32 * Vec<T>::N;
  if (p.H <= piece) return launch_cluster<combine_bwd_kernel<T, 1>>(blocks(slots, 8), kThreads, 0, 1, s, p);
  if (p.H <= 2 * piece) return launch_cluster<combine_bwd_kernel<T, 2>>(blocks(slots, 4), kThreads, 0, 1, s, p);
  if (p.H <= 4 * piece) return launch_cluster<combine_bwd_kernel<T, 4>>(blocks(slots, 2), kThreads, 0, 1, s, p);
  return launch_cluster<combine_bwd_kernel<T, 8>>(blocks(slots, 1), kThreads, 0, 1, s, p);
}
}  // namespace

cudaError_t launch_permute(const PermuteParams& p, cudaStream_t s) {
  if (p.row_bytes <= 512 * kCopies) {
    return launch_cluster<permute_kernel<1>>(blocks(p.rows, 8), kThreads, 0, 1, s, p);
  } else {
    const unsigned chunks = blocks(p.row_bytes, 512 * 8 * kCopies);
    return launch_cluster<permute_kernel<8>>(dim3(p.rows, chunks < 64 ? chunks : 64), kThreads, 0, 1, s, p);
  }
}

cudaError_t launch_row_combine(const RowCombineParams& p, int dtype, cudaStream_t s) {
  if (dtype == MOE_DT_BF16) return row_combine<__nv_bfloat16>(p, s);
  if (dtype == MOE_DT_FP16) return row_combine<__half>(p, s);
  return row_combine<float>(p, s);
}

cudaError_t launch_row_combine_bwd(const RowCombineBwdParams& p, int dtype, cudaStream_t s) {
  if (dtype == MOE_DT_BF16) return row_combine_bwd<__nv_bfloat16>(p, s);
  if (dtype == MOE_DT_FP16) return row_combine_bwd<__half>(p, s);
  return row_combine_bwd<float>(p, s);
}

cudaError_t launch_quant_int8(const QuantInt8Params& p, int dtype, cudaStream_t s) {
  return dtype == MOE_DT_BF16 ? quant_int8<__nv_bfloat16>(p, s) : quant_int8<__half>(p, s);
}

}  // namespace moe
