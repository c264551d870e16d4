// Norms around a block for rows of any alignment and types looked up, and the sum over the CTAs' partial
// sums of the gradient.
#include "norm_backward.cuh"
#include "norm_forward.cuh"

namespace moe {
namespace {

// Adds the CTAs' partial sums in order: blockIdx.y 0-3 a parameter, then the rows of gates that CTAs share
// (row y - 4, or the row at the boundary of CTAs y - 4 and y - 3 where there are fewer of those).
constexpr int kJoinCols = 32, kJoinSlices = 16;
__global__ void __launch_bounds__(kJoinCols* kJoinSlices)
    norm_join_kernel(const __grid_constant__ NormGradArgs a, int ctas) {
  __shared__ float s[kJoinSlices][kJoinCols];
  const int x = threadIdx.x % kJoinCols, slice = threadIdx.x / kJoinCols;
  const int c = blockIdx.x * kJoinCols + x, y = blockIdx.y;
  const int per = norm_rows_per_cta(a.T, ctas);
  float* dst = y == 0 ? a.d_w_after : y == 1 ? a.d_b_after : y == 2 ? a.d_w_before
                                                         : y == 3 ? a.d_b_before : a.d_gate;
  griddep_wait();
  if (dst == nullptr) return;
  int first = 0, last = ctas - 1, part = y;
  long long start = 0;
  if (y >= 4) {
    const long long rows = a.gate_rows, groups = (a.T + rows - 1) / rows;
    long long j = y - 4;
    if (groups > ctas - 1) {
      const long long edge = (long long)(y - 3) * per;  // first token of the second CTA
      if (edge >= a.T || edge % rows == 0) return;
      j = edge / rows;
      if (j * rows < edge - per) return;  // an earlier boundary's
    }
    start = j * rows;
    const long long end = start + rows < a.T ? start + rows : a.T;
    first = (int)(start / per);
    last = (int)((end - 1) / per);
    if (first == last) return;  // complete
    dst += j * a.d;
  }
  float v = 0.f;
  if (c < a.d)
    for (int i = first + slice; i <= last; i += kJoinSlices) {
      if (y >= 4) part = start < (long long)i * per ? 4 : 5;
      v += a.part[((size_t)i * kNormParts + part) * a.d + c];
    }
  s[slice][x] = v;
  __syncthreads();
  if (slice == 0 && c < a.d) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinSlices; ++i) v += s[i][x];
    dst[c] = v;
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
  return launch_k(norm_join_kernel, dim3((a.d + kJoinCols - 1) / kJoinCols, 4 + shared),
                  dim3(kJoinCols * kJoinSlices), 0, st, a, ctas);
}

}  // namespace moe
