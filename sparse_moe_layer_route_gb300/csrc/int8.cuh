// 8-bit expert products: the quantization rule and the launch interface between the entry points
// (int8_api.cu) and the kernels (int8_rows.cu, int8_gemm.cu).
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "internal.h"

namespace moe {

// Scale of a row from the largest magnitude bits among its values (sign cleared; in this order
// infinity follows every number and NaN follows infinity, so either becomes the scale).
__device__ __forceinline__ float int8_scale(uint32_t top_bits) {
  return __fmul_rn(__uint_as_float(top_bits), 1.0f / 127.0f);
}

// Code of one value: rint(x / scale) to nearest even. The clamp acts where the scale is subnormal
// (its rounding may leave x / scale past 127); a zero or non-finite scale gives 0.
__device__ __forceinline__ int int8_code(float x, float scale) {
  if (scale == 0.0f) return 0;
  const int v = __float2int_rn(__fdiv_rn(x, scale));  // NaN converts to 0
  return max(-127, min(127, v));
}

// One grouped product. Segment e < n_mat holds rows [offsets[e], offsets[e + 1]) (offsets NULL: all
// rows); with shared experts, segment n_mat + s is rows [rows + s * T, rows + (s + 1) * T).
struct Int8Gemm {
  const int8_t* qx;        // A rows [.., K]
  const float* sx;
  const int8_t *qw, *qw2;  // [n_mat, N, K]; qw2: the up projection of the SwiGLU pass
  const float *sw, *sw2;
  const int8_t *sh_qw, *sh_qw2;  // shared experts [S, N, K]
  const float *sh_sw, *sh_sw2;
  const int32_t* offsets;
  const int32_t* perm_slot;  // SwiGLU and slot passes: position -> slot (slot / k is the token)
  const float* topk_w;       // slot pass: gate per slot (NULL: 1)
  void* out;
  int* status;
  int rows, K, N, n_mat, S, T, k;
  int out_dtype;             // matrix pass
};

enum Int8Pass {
  kInt8Matrix = 0,  // out [rows, N] = product
  kInt8SwiGLU = 1,  // out [rows + S T, N] fp32 = silu(gate product) * (up product)
  kInt8Slot = 2     // out [slot, N] fp16 = gate weight * product
};

cudaError_t launch_int8_gemm(Int8Pass pass, const Int8Gemm& g, cudaStream_t st);
cudaError_t launch_quantize_rows(int T, int d, int dtype, const void* x, long long ld, int8_t* q,
                                 float* scale, cudaStream_t st);
cudaError_t launch_quantize_channels(int n_mat, int K, int N, const uint16_t* W, int8_t* q,
                                     float* scale, cudaStream_t st);

}  // namespace moe
