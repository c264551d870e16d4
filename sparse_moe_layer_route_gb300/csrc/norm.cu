// Norms before and after a block with residual, gate and dropout (forward), and dropout alone.
//
//   h' = alpha h + beta gate * drop(norm_after(y)),   n = norm_before(h')
//
// One pass: a row is read into registers once (by a warp up to 512 channels, by 128 to 512 threads up to
// 8192, by a cluster of CTAs above), its sums are taken there, and h' and n are written. The bytes of h, y,
// h' and n bound it. Layer norm takes its variance in a second sum over the registers, around the mean.
#include "norm.cuh"

namespace moe {
namespace {

template <int R>
constexpr int cta_threads() {
  return R < 256 ? 256 : R;
}

template <int R, int NC, int CL>
__global__ void __launch_bounds__(cta_threads<R>()) norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kRows = cta_threads<R>() / R;
  __shared__ float red[kRows][2][(R / 32 + CL) * 2];
  const int group = threadIdx.x / R, tid = threadIdx.x % R;
  const long long row = (long long)(blockIdx.x / CL) * kRows + group;
  griddep_wait();
  if (row >= a.T) return;
  RowSum<R, CL> sum(&red[group][0][0], group);
  const int base = CL > 1 ? (int)(blockIdx.x % CL) * (R * NC * 8) : 0;
  int col[NC];
  float h[NC][8], y[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    col[c] = base + (c * R + tid) * 8;
    load8(a.h, row, col[c], a.d, h[c]);
    if (a.y.p != nullptr) load8(a.y, row, col[c], a.d, y[c]);
  }
  if (a.y.p != nullptr) {
    const DropState ds(a.drop);
    float mean = 0.f, rstd = 1.f;
    if (a.after != MOE_NORM_NONE) row_stats<NC>(sum, a.after, y, col, a.d, a.eps, mean, rstd);
    const long long gate_row = a.gate.p != nullptr ? row / a.gate_rows : 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float v[8];
      if (a.after != MOE_NORM_NONE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[c][i] = (y[c][i] - mean) * rstd;
        if (a.w_after.p != nullptr) {
          load8(a.w_after, 0, col[c], a.d, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[c][i] *= v[i];
        }
        if (a.b_after.p != nullptr) {
          load8(a.b_after, 0, col[c], a.d, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[c][i] += v[i];
        }
      }
      if (a.drop.rng != nullptr) {
        drop8(a.drop, ds, (uint32_t)row, (uint32_t)col[c], v);
        // a dropped element is 0 whatever it was
#pragma unroll
        for (int i = 0; i < 8; ++i) y[c][i] = v[i] != 0.f ? y[c][i] * v[i] : 0.f;
      }
      if (a.gate.p != nullptr) {
        load8(a.gate, gate_row, col[c], a.d, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[c][i] *= v[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = fmaf(a.alpha, h[c][i], a.beta * y[c][i]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] *= a.alpha;
  }
  if (a.h_out.p != nullptr) {
#pragma unroll
    for (int c = 0; c < NC; ++c) store8(a.h_out, row, col[c], a.d, h[c]);
  }
  if (a.before != MOE_NORM_NONE) {
    float mean, rstd;
      row_stats<NC>(sum, a.before, h, col, a.d, a.eps, mean, rstd);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = (h[c][i] - mean) * rstd;
      if (a.w_before.p != nullptr) {
        load8(a.w_before, 0, col[c], a.d, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] *= v[i];
      }
      if (a.b_before.p != nullptr) {
        load8(a.b_before, 0, col[c], a.d, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] += v[i];
      }
      store8(a.n, row, col[c], a.d, h[c]);
    }
  }
}

// y = residual + x * factor, eight channels a thread; columns of threads are as wide as a row asks.
constexpr int kDropThreads = 256;
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const __grid_constant__ DropoutArgs a,
                                                               int wide) {
  const int tx = threadIdx.x & (wide - 1), ty = threadIdx.x / wide, rows = kDropThreads / wide;
  griddep_wait();
  const DropState ds(a.drop);
  for (long long row = (long long)blockIdx.x * rows + ty; row < a.T; row += (long long)gridDim.x * rows)
    for (int c = tx * 8; c < a.d; c += wide * 8) {
      float v[8], r[8];
      load8(a.x, row, c, a.d, v);
      if (a.residual.p != nullptr) load8(a.residual, row, c, a.d, r);
      if (a.drop.rng != nullptr) {
        float m[8];
        drop8(a.drop, ds, (uint32_t)row, (uint32_t)c, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = m[i] != 0.f ? v[i] * m[i] : 0.f;
      }
      if (a.residual.p != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
      }
      store8(a.y, row, c, a.d, v);
    }
}

template <int R, int NC, int CL>
cudaError_t launch_form(const NormArgs& a, cudaStream_t st) {
  constexpr int rows = cta_threads<R>() / R;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)a.T + rows - 1) / rows * CL));
  cfg.blockDim = dim3(cta_threads<R>());
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, norm_kernel<R, NC, CL>, a);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  return MOE_NORM_FORMS(launch_form, a.d, a, st);
}

cudaError_t launch_dropout(const DropoutArgs& a, cudaStream_t st) {
  int wide = 1;
  while (wide < kDropThreads && wide * 8 < a.d) wide *= 2;
  const int rows = kDropThreads / wide;
  const long long need = ((long long)a.T + rows - 1) / rows, most = 8ll * num_sms();
  return launch_k(dropout_kernel, dim3((unsigned)(need < most ? need : most)), dim3(kDropThreads), 0, st,
                  a, wide);
}

}  // namespace moe
