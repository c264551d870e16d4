// Products of few work units, done in pieces of K: partial sums from the tensor cores, and their join.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "int8.cuh"
#include "internal.h"

namespace moe {
namespace {

// y = (sum of the pieces, in their order) * row scale * channel scale; rows past the last segment are left.
template <typename YT>
__global__ void __launch_bounds__(256) join_splits_kernel(const float* __restrict__ part,
                                                          const Int8Gemm g) {
  griddep_wait();
  const int row = blockIdx.x;
  int seg = 0;
  if (g.offsets != nullptr) {
    // the last segment that begins at or before the row and reaches it (bad offsets were reported by
    // the product, which left their rows out)
    int lo = 0, hi = g.n_mat;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (g.offsets[mid] <= row)
        lo = mid;
      else
        hi = mid;
    }
    seg = lo;
    const int r0 = g.offsets[seg], r1 = g.offsets[seg + 1];
    if (r0 < 0 || r1 > g.rows || row < r0 || row >= r1) return;
  }
  const int n = blockIdx.y * 256 + threadIdx.x;
  if (n >= g.N) return;
  const long long at = (long long)row * g.N + n, cols = int8_part_cols(g.N);
  const long long from = row * cols + n, plane = g.rows * cols;
  const float scale = g.sx[row] * g.sw[(long long)seg * g.N + n];
  float sum = 0.0f;
  for (int i = 0; i < g.splits; i += 8) {  // eight loads in flight, added in the pieces' order
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j < g.splits ? part[(i + j) * plane + from] : 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += v[j];
  }
  sum *= scale;
  if constexpr (sizeof(YT) == 4)
    static_cast<float*>(g.out)[at] = sum;
  else if constexpr (std::is_same<YT, __nv_bfloat16>::value)
    static_cast<__nv_bfloat16*>(g.out)[at] = __float2bfloat16(sum);
  else
    static_cast<__half*>(g.out)[at] = __float2half(sum);
}

}  // namespace

int int8_splits(long long rows, int K, int N, int n_mat) {
  const long long mean = rows / n_mat;
  const long long at_once = 76;  // units that run at the same time, one on each pair of CTAs
  const long long tile = mean <= kInt8Mean64 ? 64 : mean <= kInt8Mean128 ? 128 : 192;
  const long long units = std::max(1ll, (mean + tile - 1) / tile) * n_mat * ((N + 255) / 256);
  if (units * 2 > at_once || N > 65535 * 256) return 1;
  // at least four 128-k steps a piece: shorter ones spend their time on filling the pipeline
  return (int)std::max(1ll, std::min(at_once / units, (long long)(K / kInt8StageK / 4)));
}

cudaError_t launch_int8_split(const Int8Gemm& g, float* part, cudaStream_t st) {
  Int8Gemm p = g;
  p.splits = int8_splits(g.rows, g.K, g.N, g.n_mat);
  p.out = part;
  const cudaError_t e = launch_int8_gemm(kInt8Partial, p, st);
  if (e != cudaSuccess) return e;
  p.out = g.out;
  const dim3 grid(g.rows, (g.N + 255) / 256), block(256);
  switch (g.out_dtype) {
    case MOE_DTYPE_F32: return launch_k(join_splits_kernel<float>, grid, block, 0, st, part, p);
    case MOE_DTYPE_BF16:
      return launch_k(join_splits_kernel<__nv_bfloat16>, grid, block, 0, st, part, p);
    default: return launch_k(join_splits_kernel<__half>, grid, block, 0, st, part, p);
  }
}

}  // namespace moe
