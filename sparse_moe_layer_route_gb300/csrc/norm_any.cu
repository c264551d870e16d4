// Norms around a block for rows of any alignment and types looked up, and the sum over the CTAs' partial
// sums of the gradient.
#include "norm_backward.cuh"
#include "norm_forward.cuh"

namespace moe {
namespace {

// Adds the CTAs' partial sums in order: blockIdx.y 0-3 a parameter, then the rows of gates that CTAs share
// (row y - 4, or the row at the boundary of CTAs y - 4 and y - 3 where there are fewer of those).
// A thread has V columns (4, or 1 where rows do not start on 16 bytes) of every 32nd CTA.
constexpr int kJoinLanes = 16, kJoinSlices = 32;
template <int V>
__global__ void __launch_bounds__(kJoinLanes* kJoinSlices)
    norm_join_kernel(const __grid_constant__ NormGradArgs a, int ctas) {
  __shared__ float s[kJoinSlices / 2][kJoinLanes * V];
  const int x = threadIdx.x % kJoinLanes * V, slice = threadIdx.x / kJoinLanes;
  const int c = blockIdx.x * kJoinLanes * V + x, y = blockIdx.y;
  const int per = norm_rows_per_cta(a.T, ctas);
  float* dst = y == 0 ? a.d_w_after : y == 1 ? a.d_b_after : y == 2 ? a.d_w_before
                                                         : y == 3 ? a.d_b_before : a.d_gate;
  griddep_wait();
  if (dst == nullptr) return;
  int first = 0, last = ctas - 1;
  if (y >= 4) {
    const long long rows = a.gate_rows, groups = (a.T + rows - 1) / rows;
    long long j = y - 4;
    if (groups > ctas - 1) {
      const long long edge = (long long)(y - 3) * per;  // first token of the second CTA
      if (edge >= a.T || edge % rows == 0) return;
      j = edge / rows;
      if (j * rows < edge - per) return;  // an earlier boundary's
    }
    const long long start = j * rows;
    const long long end = start + rows < a.T ? start + rows : a.T;
    first = (int)(start / per);
    last = (int)((end - 1) / per);
    if (first == last) return;  // complete
    dst += j * a.d;
  }
  float v[V] = {};
  if (c < a.d) {
    // of a row of gates the first CTA has the sum that it shares with the next, the others the one with the CTA before
    const float* p = a.part + ((size_t)(first + slice) * kNormParts + (y < 4 ? y : 4)) * a.d + c;
    int ahead = y >= 4 && slice == 0 ? a.d : 0;
#pragma unroll 4
    for (int i = first + slice; i <= last; i += kJoinSlices) {
      if constexpr (V == 4) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(p + ahead));
        v[0] += q.x, v[1] += q.y, v[2] += q.z, v[3] += q.w;
      } else {
        v[0] += __ldg(p + ahead);
      }
      ahead = 0;
      p += (size_t)kJoinSlices * kNormParts * a.d;
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    v[k] += __shfl_xor_sync(0xffffffffu, v[k], 16);
    if (slice % 2 == 0) s[slice / 2][x + k] = v[k];
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < kJoinLanes * V && blockIdx.x * kJoinLanes * V + t < a.d) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinSlices / 2; ++i) sum += s[i][t];
    dst[blockIdx.x * kJoinLanes * V + t] = sum;
  }
}

}  // namespace

cudaError_t launch_norm_any(const NormArgs& a, cudaStream_t st) { return launch_forward<Any, Any>(a, st); }
cudaError_t launch_norm_grad_any(const NormGradArgs& a, int* ctas, cudaStream_t st) {
  return launch_backward<Any, Any>(a, ctas, st);
}

cudaError_t launch_norm_join(const NormGradArgs& a, int ctas, cudaStream_t st) {
  int shared = 0;  // rows of gates that CTAs may share
  if (a.d_gate != nullptr && a.gate_rows > 1) {
    const long long rows = ((long long)a.T + a.gate_rows - 1) / a.gate_rows;
    shared = (int)(rows < ctas - 1 ? rows : ctas - 1);
  }
  if (!a.d_w_after && !a.d_b_after && !a.d_w_before && !a.d_b_before && shared == 0)
    return cudaSuccess;
  const auto launch = [&](auto kernel, int cols) {
    return launch_k(kernel, dim3((a.d + cols - 1) / cols, 4 + shared), dim3(kJoinLanes * kJoinSlices), 0, st, a, ctas);
  };
  return a.d % 4 == 0 ? launch(norm_join_kernel<4>, 4 * kJoinLanes) : launch(norm_join_kernel<1>, kJoinLanes);
}

}  // namespace moe
