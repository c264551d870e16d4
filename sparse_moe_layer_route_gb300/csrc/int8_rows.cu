// Symmetric 8-bit quantization: rows of activations (one scale per token) and, once per model, the
// output channels of bf16 weights.
//
//   scale = max|x| * fl(1 / 127),  q = clamp(rint(x / scale), -127, 127)   (fp32, rint to even)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "int8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

// Eight consecutive elements of a row, loaded as 16-byte pieces.
template <typename XT>
struct Vec8 {
  uint4 p;
  __device__ __forceinline__ void load(const XT* at) { p = *reinterpret_cast<const uint4*>(at); }
  __device__ __forceinline__ void get(float (&v)[8]) const;
  // Largest magnitudes so far, one per half of a word (16-bit magnitudes order as their bits do).
  __device__ __forceinline__ void top(uint32_t& pair) const {
    pair = __vimax3_u16x2(pair, p.x & 0x7fff7fffu, p.y & 0x7fff7fffu);
    pair = __vimax3_u16x2(pair, p.z & 0x7fff7fffu, p.w & 0x7fff7fffu);
  }
  // The larger of the two as fp32 bits.
  static __device__ __forceinline__ uint32_t top_bits(uint32_t pair) {
    const uint32_t m = max(pair & 0xffffu, pair >> 16);
    if (std::is_same<XT, __half>::value) return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
    return m << 16;
  }
};
template <>
__device__ __forceinline__ void Vec8<__nv_bfloat16>::get(float (&v)[8]) const {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void Vec8<__half>::get(float (&v)[8]) const {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <>
struct Vec8<float> {
  float4 p, q;
  __device__ __forceinline__ void load(const float* at) {
    p = reinterpret_cast<const float4*>(at)[0];
    q = reinterpret_cast<const float4*>(at)[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w;
    v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
  }
  __device__ __forceinline__ void top(uint32_t& t) const {
    float v[8];
    get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) t = max(t, __float_as_uint(v[j]) & 0x7fffffffu);
  }
  static __device__ __forceinline__ uint32_t top_bits(uint32_t t) { return t; }
};

// Where the codes go: 8-bit, or 16-bit for the tensor cores (whole numbers up to 127 are exact in
// fp16). m: the codes plus kMagic, 1.5 * 2^23, whose fp32 neighbours are one apart: adding it rounds to the
// nearest whole number, and the sum's low byte is the code.
constexpr float kMagic = 12582912.0f;
__device__ __forceinline__ void store_codes8(int8_t* at, const float (&m)[8]) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(m[i]);
  uint2 o;
  o.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  o.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  *reinterpret_cast<uint2*>(at) = o;
}
__device__ __forceinline__ void store_codes8(uint16_t* at, const float (&m)[8]) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(m[2 * i] - kMagic, m[2 * i + 1] - kMagic);
    o[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(at) = make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void store_code(int8_t* at, int c) { *at = (int8_t)c; }
__device__ __forceinline__ void store_code(uint16_t* at, int c) {
  *at = __half_as_ushort(__int2half_rn(c));
}

// The largest magnitude bits over the threads of a row: a warp (W = 32) or a CTA of W threads.
template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t top, uint32_t* warp_top) {
  top = __reduce_max_sync(kFull, top);
  if (W > 32) {
    if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W / 32; ++w) top = max(top, warp_top[w]);
  }
  return top;
}

// One row by W threads, thread t of them. VEC: rows in 16-byte pieces, d a multiple of 8 and at most
// 64 W; the row stays in registers between its two passes. x / scale is q = x r with r the correctly rounded
// 1 / scale, then q + (x - q scale) r: the correctly rounded quotient (Markstein 1990) in three
// instructions without a branch, so the codes are the division's. (Halfway values are common among bf16
// ones: dividing the near-halfway values alone took 15 of 66 us for 16384 rows of 7168.)
template <int W, bool VEC, typename XT, typename QT>
__device__ __forceinline__ void quantize_row(const XT* __restrict__ row, int d,
                                             QT* __restrict__ out, float* __restrict__ scale,
                                             int t, uint32_t* warp_top) {
  uint32_t top = 0u;
  if constexpr (VEC) {
    constexpr int NV = 8;
    Vec8<XT> x[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * W + t) * 8 < d) x[i].load(row + (i * W + t) * 8);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * W + t) * 8 < d) x[i].top(top);
    const float s = int8_scale(row_max<W>(Vec8<XT>::top_bits(top), warp_top));
    if (t == 0) *scale = s;
    const bool plain = s > 1e-30f && s < 1e30f;  // 1 / s is a normal number
    const float r = plain ? __frcp_rn(s) : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * W + t) * 8 < d) {
        float v[8], m[8];
        x[i].get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y = __fmul_rn(v[j], r);
          m[j] = __fadd_rn(__fmaf_rn(__fmaf_rn(-y, s, v[j]), r, y), kMagic);
        }
        if (!plain) {
#pragma unroll
          for (int j = 0; j < 8; ++j) m[j] = (float)int8_code(v[j], s) + kMagic;
        }
        store_codes8(out + (i * W + t) * 8, m);
      }
  } else {
    for (int j = t; j < d; j += W)
      top = max(top, __float_as_uint(to_f32(row[j])) & 0x7fffffffu);
    const float s = int8_scale(row_max<W>(top, warp_top));
    if (t == 0) *scale = s;
    for (int j = t; j < d; j += W) store_code(out + j, int8_code(to_f32(row[j]), s));
  }
}

// Rows of x to 8-bit codes. W = 32: a warp per row, else a CTA of W threads.
template <int W, bool VEC, typename XT>
__global__ void __launch_bounds__(W == 32 ? kThreads : W)
    quantize_rows_kernel(const XT* __restrict__ x, long long ld, int T, int d,
                         int8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ uint32_t warp_top[W / 32];
  griddep_wait();
  const long long p = W == 32 ? (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)
                              : (long long)blockIdx.x;
  if (p >= T) return;
  quantize_row<W, VEC>(x + p * ld, d, q + p * d, scale + p, W == 32 ? threadIdx.x & 31 : threadIdx.x,
                       warp_top);
}

template <int W, bool VEC, typename QT>
__global__ void __launch_bounds__(W == 32 ? kThreads : W) quantize_gather_kernel(
    const __nv_bfloat16* __restrict__ x, const int32_t* __restrict__ perm_slot,
    const int32_t* __restrict__ offsets, int E, int k, int d, int TK, int rows,
    QT* __restrict__ xq, float* __restrict__ sx, int* status) {
  __shared__ uint32_t warp_top[W / 32];
  griddep_wait();
  const long long p = W == 32 ? (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)
                              : (long long)blockIdx.x;
  const int t = W == 32 ? threadIdx.x & 31 : threadIdx.x;
  if (p >= rows) return;
  long long token = p - TK;  // shared experts: every token
  if (p < TK) {
    const int n_kept = offsets[E], slot = perm_slot[p];  // both loads in flight
    if (p >= n_kept) return;
    token = slot / k;
    if (slot < 0 || slot >= TK) {
      for (int j = t; j < d; j += W) xq[p * d + j] = 0;
      if (t == 0) {
        sx[p] = 0.0f;
        atomicOr(status, MOE_DEVFAULT_BAD_TILE);
      }
      return;
    }
  }
  quantize_row<W, VEC>(x + token * d, d, xq + p * d, sx + p, t, warp_top);
}

template <int W, bool VEC, typename QT>
__global__ void __launch_bounds__(W == 32 ? kThreads : W)
    quantize_hidden_kernel(const float* __restrict__ h, const int32_t* __restrict__ offsets, int E,
                           int f, int TK, long long rows, QT* __restrict__ hq,
                           float* __restrict__ sh) {
  __shared__ uint32_t warp_top[W / 32];
  griddep_wait();
  const long long p = W == 32 ? (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)
                              : (long long)blockIdx.x;
  if (p >= rows || (p < TK && p >= offsets[E])) return;
  quantize_row<W, VEC>(h + p * f, f, hq + p * f, sh + p, W == 32 ? threadIdx.x & 31 : threadIdx.x,
                       warp_top);
}

__global__ void __launch_bounds__(kThreads) widen_codes_kernel(const int4* __restrict__ q,
                                                               uint4* __restrict__ xq,
                                                               long long n16) {
  griddep_wait();
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n16) return;
  const int4 v = q[i];
  uint4 a, b;
  widen4(v.x, a.x, a.y);
  widen4(v.y, a.z, a.w);
  widen4(v.z, b.x, b.y);
  widen4(v.w, b.z, b.w);
  xq[2 * i] = a;
  xq[2 * i + 1] = b;
}

// W [K, N] bf16 to q [N, K], scale [N]; one CTA per 32 output channels of one matrix.
__global__ void __launch_bounds__(kThreads) quantize_channels_kernel(
    const uint16_t* __restrict__ W, int K, int N, int8_t* __restrict__ q,
    float* __restrict__ scale) {
  __shared__ uint32_t top[8][33];
  __shared__ float sc[32];
  __shared__ int8_t tile[32][33];
  griddep_wait();
  const long long m = blockIdx.y;
  const int n0 = blockIdx.x * 32, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const __nv_bfloat16* w = reinterpret_cast<const __nv_bfloat16*>(W) + m * K * N;
  const bool in = n0 + tx < N;
  uint32_t t = 0u;
  for (int k = ty; in && k < K; k += 8)
    t = max(t, __float_as_uint(__bfloat162float(w[(long long)k * N + n0 + tx])) & 0x7fffffffu);
  top[ty][tx] = t;
  __syncthreads();
  if (ty == 0) {
    for (int i = 1; i < 8; ++i) t = max(t, top[i][tx]);
    sc[tx] = int8_scale(t);
    if (in) scale[m * N + n0 + tx] = sc[tx];
  }
  __syncthreads();
  for (int k0 = 0; k0 < K; k0 += 32) {
    for (int i = ty; i < 32; i += 8)
      if (in && k0 + i < K)
        tile[tx][i] =
            (int8_t)int8_code(__bfloat162float(w[(long long)(k0 + i) * N + n0 + tx]), sc[tx]);
    __syncthreads();
    for (int i = ty; i < 32; i += 8)
      if (n0 + i < N && k0 + tx < K) q[(m * N + n0 + i) * K + k0 + tx] = tile[i][tx];
    __syncthreads();
  }
}

}  // namespace

namespace {

// Calls f(W, VEC) for rows of d elements: a warp per row up to 2048 elements, else a CTA, with the row in
// registers up to 8192 (128 threads) or 16384 (256); vec: rows are in 16-byte pieces of eight elements.
// At most as many rows as GB300 has SMs (152) take 512 threads each: then one row's time is the kernel's.
template <int N>
using Int = std::integral_constant<int, N>;
template <typename F>
cudaError_t by_row(long long rows, int d, bool vec, F f) {
  if (vec && rows <= 152 && d > 512 && d <= 16384) return f(Int<512>{}, std::true_type{});
  if (d <= 2048) return vec ? f(Int<32>{}, std::true_type{}) : f(Int<32>{}, std::false_type{});
  if (vec && d <= 8192) return f(Int<128>{}, std::true_type{});
  if (vec && d <= 16384) return f(Int<256>{}, std::true_type{});
  return f(Int<256>{}, std::false_type{});
}
template <int W>
dim3 row_grid(long long rows) {
  return dim3((unsigned)(W == 32 ? (rows + kThreads / 32 - 1) / (kThreads / 32) : rows));
}
template <int W>
dim3 row_block() {
  return dim3(W == 32 ? kThreads : W);
}

template <typename XT>
cudaError_t quantize_rows_as(int T, int d, const XT* x, long long ld, int8_t* q, float* scale,
                             cudaStream_t st) {
  const bool vec = d % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                   (T == 1 || ld * sizeof(XT) % 16 == 0) &&
                   reinterpret_cast<uintptr_t>(q) % 8 == 0;
  return by_row(T, d, vec, [&](auto w, auto v) {
    constexpr int W = decltype(w)::value;
    return launch_k(quantize_rows_kernel<W, decltype(v)::value, XT>, row_grid<W>(T),
                    row_block<W>(), 0, st, x, ld, T, d, q, scale);
  });
}

}  // namespace

cudaError_t launch_quantize_rows(int T, int d, int dtype, const void* x, long long ld, int8_t* q,
                                 float* scale, cudaStream_t st) {
  switch (dtype) {
    case MOE_DTYPE_BF16:
      return quantize_rows_as(T, d, static_cast<const __nv_bfloat16*>(x), ld, q, scale, st);
    case MOE_DTYPE_F16:
      return quantize_rows_as(T, d, static_cast<const __half*>(x), ld, q, scale, st);
    default:
      return quantize_rows_as(T, d, static_cast<const float*>(x), ld, q, scale, st);
  }
}

cudaError_t launch_quantize_channels(int n_mat, int K, int N, const uint16_t* W, int8_t* q,
                                     float* scale, cudaStream_t st) {
  return launch_k(quantize_channels_kernel, dim3((N + 31) / 32, n_mat), dim3(kThreads), 0, st, W,
                  K, N, q, scale);
}

cudaError_t launch_widen_codes(const int8_t* q, uint16_t* xq, long long n, cudaStream_t st) {
  const long long n16 = n / 16;
  return launch_k(widen_codes_kernel, dim3((unsigned)((n16 + kThreads - 1) / kThreads)),
                  dim3(kThreads), 0, st, reinterpret_cast<const int4*>(q),
                  reinterpret_cast<uint4*>(xq), n16);
}

template <typename QT>
cudaError_t launch_quantize_gather(const Shape& s, const uint16_t* x, const int32_t* perm_slot,
                                   const int32_t* offsets, QT* xq, float* sx, int* status,
                                   cudaStream_t st) {
  const long long rows = s.TK + (s.S > 0 ? s.T : 0);
  return by_row(rows, s.d, true, [&](auto w, auto v) {  // d is a multiple of 64, x 16-byte aligned
    constexpr int W = decltype(w)::value;
    return launch_k(quantize_gather_kernel<W, decltype(v)::value, QT>, row_grid<W>(rows),
                    row_block<W>(), 0, st, reinterpret_cast<const __nv_bfloat16*>(x), perm_slot,
                    offsets, s.E, s.k, s.d, (int)s.TK, (int)rows, xq, sx, status);
  });
}

template <typename QT>
cudaError_t launch_quantize_hidden(const Shape& s, const float* h, const int32_t* offsets, QT* hq,
                                   float* sh, cudaStream_t st) {
  return by_row(s.rows, s.f, true, [&](auto w, auto v) {
    constexpr int W = decltype(w)::value;
    return launch_k(quantize_hidden_kernel<W, decltype(v)::value, QT>, row_grid<W>(s.rows),
                    row_block<W>(), 0, st, h, offsets, s.E, s.f, (int)s.TK, (long long)s.rows, hq,
                    sh);
  });
}

template cudaError_t launch_quantize_gather<uint16_t>(const Shape&, const uint16_t*, const int32_t*,
                                                     const int32_t*, uint16_t*, float*, int*,
                                                     cudaStream_t);
template cudaError_t launch_quantize_gather<int8_t>(const Shape&, const uint16_t*, const int32_t*,
                                                   const int32_t*, int8_t*, float*, int*,
                                                   cudaStream_t);
template cudaError_t launch_quantize_hidden<uint16_t>(const Shape&, const float*, const int32_t*,
                                                     uint16_t*, float*, cudaStream_t);
template cudaError_t launch_quantize_hidden<int8_t>(const Shape&, const float*, const int32_t*,
                                                   int8_t*, float*, cudaStream_t);

}  // namespace moe
