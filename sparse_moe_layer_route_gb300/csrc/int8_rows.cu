// Symmetric 8-bit quantization: rows of activations (one scale per token) and, once per model, the
// output channels of bf16 weights.
//
//   scale = max|x| * fl(1 / 127),  q = clamp(rint(x / scale), -127, 127)   (fp32, rint to even)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "internal.h"
#include "int8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

// One CTA per row.
template <typename XT>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const XT* __restrict__ x,
                                                                 long long ld, int d,
                                                                 int8_t* __restrict__ q,
                                                                 float* __restrict__ scale) {
  __shared__ uint32_t warp_top[kThreads / 32];
  griddep_wait();
  const XT* row = x + (long long)blockIdx.x * ld;
  uint32_t top = 0u;
  for (int j = threadIdx.x; j < d; j += kThreads)
    top = max(top, __float_as_uint(to_f32(row[j])) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) top = max(top, warp_top[w]);
  const float s = int8_scale(top);
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
  for (int j = threadIdx.x; j < d; j += kThreads)
    q[(long long)blockIdx.x * d + j] = (int8_t)int8_code(to_f32(row[j]), s);
}

// Codes of one row in fp16, for the tensor cores (whole numbers up to 127 are exact there).
template <typename XT>
__device__ __forceinline__ void code_row(const XT* __restrict__ row, int d,
                                         uint16_t* __restrict__ out, float* __restrict__ scale,
                                         uint32_t* warp_top) {
  uint32_t top = 0u;
  for (int j = threadIdx.x; j < d; j += kThreads)
    top = max(top, __float_as_uint(to_f32(row[j])) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) top = max(top, warp_top[w]);
  const float s = int8_scale(top);
  if (threadIdx.x == 0) *scale = s;
  for (int j = threadIdx.x; j < d; j += kThreads)
    out[j] = __half_as_ushort(__int2half_rn(int8_code(to_f32(row[j]), s)));
}

__global__ void __launch_bounds__(kThreads) quantize_gather_kernel(
    const __nv_bfloat16* __restrict__ x, const int32_t* __restrict__ perm_slot,
    const int32_t* __restrict__ offsets, int E, int k, int d, int TK, uint16_t* __restrict__ xq,
    float* __restrict__ sx, int* status) {
  __shared__ uint32_t warp_top[kThreads / 32];
  griddep_wait();
  const int p = blockIdx.x;
  long long t = p - TK;  // shared experts: every token
  if (p < TK) {
    if (p >= offsets[E]) return;
    const int slot = perm_slot[p];
    t = slot / k;
    if (slot < 0 || slot >= TK) {
      for (int j = threadIdx.x; j < d; j += kThreads) xq[(long long)p * d + j] = 0;
      if (threadIdx.x == 0) {
        sx[p] = 0.0f;
        atomicOr(status, MOE_DEVFAULT_BAD_TILE);
      }
      return;
    }
  }
  code_row(x + t * d, d, xq + (long long)p * d, sx + p, warp_top);
}

__global__ void __launch_bounds__(kThreads) quantize_hidden_kernel(
    const float* __restrict__ h, const int32_t* __restrict__ offsets, int E, int f, int TK,
    uint16_t* __restrict__ hq, float* __restrict__ sh) {
  __shared__ uint32_t warp_top[kThreads / 32];
  griddep_wait();
  const long long p = blockIdx.x;
  if (p < TK && p >= offsets[E]) return;
  code_row(h + p * f, f, hq + p * f, sh + p, warp_top);
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

cudaError_t launch_quantize_rows(int T, int d, int dtype, const void* x, long long ld, int8_t* q,
                                 float* scale, cudaStream_t st) {
  const dim3 grid(T), block(kThreads);
  switch (dtype) {
    case MOE_DTYPE_BF16:
      return launch_k(quantize_rows_kernel<__nv_bfloat16>, grid, block, 0, st,
                      static_cast<const __nv_bfloat16*>(x), ld, d, q, scale);
    case MOE_DTYPE_F16:
      return launch_k(quantize_rows_kernel<__half>, grid, block, 0, st,
                      static_cast<const __half*>(x), ld, d, q, scale);
    default:
      return launch_k(quantize_rows_kernel<float>, grid, block, 0, st,
                      static_cast<const float*>(x), ld, d, q, scale);
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

cudaError_t launch_quantize_gather(const Shape& s, const uint16_t* x, const int32_t* perm_slot,
                                   const int32_t* offsets, uint16_t* xq, float* sx, int* status,
                                   cudaStream_t st) {
  const long long rows = s.TK + (s.S > 0 ? s.T : 0);
  return launch_k(quantize_gather_kernel, dim3((unsigned)rows), dim3(kThreads), 0, st,
                  reinterpret_cast<const __nv_bfloat16*>(x), perm_slot, offsets, s.E, s.k, s.d,
                  (int)s.TK, xq, sx, status);
}

cudaError_t launch_quantize_hidden(const Shape& s, const float* h, const int32_t* offsets,
                                   uint16_t* hq, float* sh, cudaStream_t st) {
  return launch_k(quantize_hidden_kernel, dim3((unsigned)s.rows), dim3(kThreads), 0, st, h,
                  offsets, s.E, s.f, (int)s.TK, hq, sh);
}

}  // namespace moe
