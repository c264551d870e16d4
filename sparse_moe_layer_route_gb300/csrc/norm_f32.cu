// Norms around a block for a stream in f32, rows that start on 16 bytes.
#include "norm_backward.cuh"
#include "norm_forward.cuh"

namespace moe {

cudaError_t launch_norm_f32(const NormArgs& a, cudaStream_t st) {
  return a.y.dtype == MOE_DTYPE_F32    ? launch_forward<F32, F32>(a, st)
         : a.y.dtype == MOE_DTYPE_BF16 ? launch_forward<F32, BF16>(a, st)
                                       : launch_forward<F32, F16>(a, st);
}
cudaError_t launch_norm_grad_f32(const NormGradArgs& a, int* ctas, cudaStream_t st) {
  return a.y.dtype == MOE_DTYPE_F32    ? launch_backward<F32, F32>(a, ctas, st)
         : a.y.dtype == MOE_DTYPE_BF16 ? launch_backward<F32, BF16>(a, ctas, st)
                                       : launch_backward<F32, F16>(a, ctas, st);
}

}  // namespace moe
