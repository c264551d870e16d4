// Products of few work units, done in pieces of K: partial sums from the tensor cores, and their join.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "int8.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kJoinThreads = 128;

// y = (sum of the pieces, in their order) * row scale * channel scale; rows past the last segment are left.
// Four channels a thread (one each, 300 rows of 4096 channels in two pieces took 9.3 us of this kernel, not 3.6;
// eight loads in flight 4.6). vec: y's rows and the scales begin on four elements.
template <typename YT>
__global__ void __launch_bounds__(kJoinThreads) join_splits_kernel(const float* __restrict__ part,
                                                                   const Int8Gemm g, bool vec) {
  griddep_wait();
  const int row = blockIdx.x;
  int seg = 0;
  if (g.offsets != nullptr) {
    // the first sound segment that holds the row; offsets may not ascend, so every one is looked at
    __shared__ int first;
    if (threadIdx.x == 0) first = INT_MAX;
    __syncthreads();
    for (int e = threadIdx.x; e < g.n_mat; e += kJoinThreads) {
      const int r0 = g.offsets[e], r1 = g.offsets[e + 1];
      if (segment_ok(r0, r1, g.rows) && row >= r0 && row < r1) atomicMin(&first, e);
    }
    __syncthreads();
    seg = first;
    if (seg == INT_MAX) return;
  }
  const int n = (blockIdx.y * kJoinThreads + threadIdx.x) * 4;
  if (n >= g.N) return;
  const long long cols = int8_part_cols(g.N), plane = g.rows * cols;
  const float* from = part + row * cols + n;
  const float* sw = g.sw + (long long)seg * g.N + n;
  const float sx = g.sx[row];
  float scale[4];
  if (vec) {
    *reinterpret_cast<float4*>(scale) = *reinterpret_cast<const float4*>(sw);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) scale[c] = n + c < g.N ? sw[c] : 0.0f;
  }
  float sum[4] = {};
  for (int i = 0; i < g.splits; i += 4) {  // four loads in flight, added in the pieces' order
    float4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = i + j < g.splits ? *reinterpret_cast<const float4*>(from + (i + j) * plane)
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sum[0] += v[j].x;
      sum[1] += v[j].y;
      sum[2] += v[j].z;
      sum[3] += v[j].w;
    }
  }
  YT y[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float f = sum[c] * sx * scale[c];
    if constexpr (sizeof(YT) == 4)
      y[c] = f;
    else if constexpr (std::is_same<YT, __nv_bfloat16>::value)
      y[c] = __float2bfloat16(f);
    else
      y[c] = __float2half(f);
  }
  YT* to = static_cast<YT*>(g.out) + (long long)row * g.N + n;
  if (vec) {
    using V = std::conditional_t<sizeof(YT) == 4, uint4, uint2>;
    V out;
    memcpy(&out, y, sizeof(out));
    *reinterpret_cast<V*>(to) = out;
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (n + c < g.N) to[c] = y[c];
  }
}

template <typename YT>
cudaError_t launch_join(const float* part, const Int8Gemm& g, cudaStream_t st) {
  const dim3 grid(g.rows, (g.N + 4 * kJoinThreads - 1) / (4 * kJoinThreads));
  const bool vec = g.N % 4 == 0 && reinterpret_cast<uintptr_t>(g.out) % (4 * sizeof(YT)) == 0 &&
                   reinterpret_cast<uintptr_t>(g.sw) % 16 == 0;
  return launch_k(join_splits_kernel<YT>, grid, dim3(kJoinThreads), 0, st, part, g, vec);
}

}  // namespace

namespace {
long long tile_rows(long long mean) { return mean <= kInt8Mean64 ? 64 : mean <= kInt8Mean128 ? 128 : 192; }
}  // namespace

int int8_splits(long long rows, int K, int N, int n_mat) {
  const long long mean = rows / n_mat, tile = tile_rows(mean);
  // units that run at the same time, one on each pair of GB300's 152 SMs: a constant, as the size of a workspace
  // depends on it and may be asked for where there is no GPU
  const long long at_once = 76;
  const long long units = std::max(1ll, (mean + tile - 1) / tile) * n_mat * ((N + 255) / 256);
  if (units * 2 > at_once || N > 65535 * 4 * kJoinThreads) return 1;
  // at least four 128-k steps a piece: shorter ones spend their time on filling the pipeline
  return (int)std::max(1ll, std::min(at_once / units, (long long)(K / kInt8StageK / 4)));
}

long long int8_splits_end(long long rows, int n_mat) {
  const long long mean = rows / n_mat, tile = tile_rows(mean);
  const long long end = tile == 64 ? kInt8Mean64 : tile == 128 ? kInt8Mean128 : (mean + 191) / 192 * 192;
  return (end + 1) * n_mat - 1;
}

cudaError_t launch_int8_split(const Int8Gemm& g, float* part, cudaStream_t st) {
  Int8Gemm p = g;
  p.splits = int8_splits(g.rows, g.K, g.N, g.n_mat);
  p.out = part;
  const cudaError_t e = launch_int8_gemm(kInt8Partial, p, st);
  if (e != cudaSuccess) return e;
  p.out = g.out;
  switch (g.out_dtype) {
    case MOE_DTYPE_F32: return launch_join<float>(part, p, st);
    case MOE_DTYPE_BF16: return launch_join<__nv_bfloat16>(part, p, st);
    default: return launch_join<__half>(part, p, st);
  }
}

}  // namespace moe
