// Norms around a block for a stream in bf16, rows that start on 16 bytes.
#include "norm_backward.cuh"
#include "norm_forward.cuh"

namespace moe {

cudaError_t launch_norm_bf16(const NormArgs& a, cudaStream_t st) {
  return a.y.dtype == MOE_DTYPE_F32    ? launch_forward<BF16, F32>(a, st)
         : a.y.dtype == MOE_DTYPE_BF16 ? launch_forward<BF16, BF16>(a, st)
                                       : launch_forward<BF16, F16>(a, st);
}
cudaError_t launch_norm_grad_bf16(const NormGradArgs& a, int* ctas, cudaStream_t st) {
  return a.y.dtype == MOE_DTYPE_F32    ? launch_backward<BF16, F32>(a, ctas, st)
         : a.y.dtype == MOE_DTYPE_BF16 ? launch_backward<BF16, BF16>(a, ctas, st)
                                       : launch_backward<BF16, F16>(a, ctas, st);
}

}  // namespace moe
