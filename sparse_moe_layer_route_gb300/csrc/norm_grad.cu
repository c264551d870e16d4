// Gradients of the norms around a block (forward: norm.cu). With hats for normed values before w and b,
// D = d_h_out, N = d_n:
//   G  = D + r_b (N w_b - h^ mean(N w_b h^) - mean(N w_b))      gradient to h' (last mean: layer norm)
//   d_h = alpha G
//   E  = beta G m gate                                          to u, m: dropout's factor
//   d_y = r_a (E w_a - y^ mean(E w_a y^) - mean(E w_a))
// and over the tokens d_gate = sum beta G m u, d_w_a = sum E y^, d_b_a = sum E, d_w_b = sum N h^, d_b_b = sum N.
//
// One pass as in norm.cu: h', y, D and N are read once, the statistics are taken again from them (cheaper than
// keeping them), d_h and d_y written. Every CTA has a run of consecutive tokens and adds up the
// parameters' gradients in registers, a thread its own channels; the CTAs' sums go to the workspace and
// are added there in order by a second, small kernel. A row of gates whose tokens are all in one CTA's run is
// complete there; one that is shared leaves a partial sum in each.
#include "norm.cuh"

namespace moe {
namespace {

template <int R>
constexpr int grad_threads() {
  return R < 256 ? 256 : R;
}

// Tokens of a CTA (a cluster).
__host__ __device__ __forceinline__ int rows_per_cta(int T, int ctas) {
  return (int)(((long long)T + ctas - 1) / ctas);
}

// Sums of the CTA's row groups for their channels, in order, to dst [d] (fp32).
template <int R, int NC>
__device__ __forceinline__ void flush(const float (&acc)[NC][8], float* stage, int group, int tid,
                                      const int (&col)[NC], int d, float* dst) {
  constexpr int kGroups = grad_threads<R>() / R;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col[c] + i < d) dst[col[c] + i] = acc[c][i];
  } else {
    constexpr int kWidth = R * NC * 8;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) stage[group * kWidth + col[c] + i] = acc[c][i];
    __syncthreads();
    for (int k = threadIdx.x; k < d; k += blockDim.x) {
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) s += stage[g * kWidth + k];
      dst[k] = s;
    }
  }
}

// BIAS: a bias has a gradient (its sums cost 16 registers a chunk).
template <int R, int NC, int CL, bool BIAS>
__global__ void __launch_bounds__(grad_threads<R>()) norm_grad_kernel(const __grid_constant__ NormGradArgs a) {
  constexpr int kGroups = grad_threads<R>() / R;
  __shared__ float red[kGroups][2][(R / 32 + CL) * 2];
  __shared__ float stage[kGroups > 1 ? kGroups * R * NC * 8 : 1];
  const int group = threadIdx.x / R, tid = threadIdx.x % R;
  const int cta = blockIdx.x / CL, ctas = gridDim.x / CL;
  const int per = rows_per_cta(a.T, ctas);
  const long long r0 = (long long)cta * per, r1 = r0 + per < a.T ? r0 + per : a.T;
  RowSum<R, CL> sum(&red[group][0][0], group);
  const int base = CL > 1 ? (int)(blockIdx.x % CL) * (R * NC * 8) : 0;
  const float inv = 1.f / (float)a.d;
  int col[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) col[c] = base + (c * R + tid) * 8;
  griddep_wait();
  const DropState ds(a.drop);
  float* part = a.part + (size_t)cta * kNormParts * a.d;
  const bool normed = a.d_n.p != nullptr;  // the norm before the next block has a gradient
  // the tokens are taken in the same order whether or not the gates' gradient is wanted, so that the others
  // do not depend on it
  const bool sum_gates = a.gate.p != nullptr && a.gate_rows > 1;
  float wa[NC][8] = {}, wb[NC][8] = {}, ga[NC][8] = {};
  float ba[BIAS ? NC : 1][8] = {}, bb[BIAS ? NC : 1][8] = {};
  for (long long s0 = r0; s0 < r1;) {
    // tokens with the same row of gates
    long long s1 = r1;
    if (sum_gates) {
      const long long end = (s0 / a.gate_rows + 1) * a.gate_rows;
      s1 = end < r1 ? end : r1;
    }
    for (long long row = s0 + group; row < s1; row += kGroups) {
      float g[NC][8], y[NC][8], v[8];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (a.d_h_out.p != nullptr) {
          load8(a.d_h_out, row, col[c], a.d, g[c]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) g[c][i] = 0.f;
        }
        if (a.y.p != nullptr) load8(a.y, row, col[c], a.d, y[c]);
      }
      if (normed) {
        float h[NC][8], n[NC][8];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          load8(a.h, row, col[c], a.d, h[c]);
          load8(a.d_n, row, col[c], a.d, n[c]);
        }
        float mean, rstd;
        row_stats<NC>(sum, a.before, h, col, a.d, a.eps, mean, rstd);
        float m[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (a.w_before.p != nullptr) load8(a.w_before, 0, col[c], a.d, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            h[c][i] = (h[c][i] - mean) * rstd;
            wb[c][i] = fmaf(n[c][i], h[c][i], wb[c][i]);
            if constexpr (BIAS) bb[c][i] += n[c][i];
            if (a.w_before.p != nullptr) n[c][i] *= v[i];
            m[0] = fmaf(n[c][i], h[c][i], m[0]);
            m[1] += n[c][i];
          }
        }
        sum(m);
        m[0] *= inv;
        m[1] = a.before == MOE_NORM_LAYER ? m[1] * inv : 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            g[c][i] = fmaf(rstd, n[c][i] - fmaf(h[c][i], m[0], m[1]), g[c][i]);
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = a.alpha * g[c][i];
        store8(a.d_h, row, col[c], a.d, v);
      }
      if (a.y.p == nullptr) continue;
      float mean = 0.f, rstd = 1.f;
      if (a.after != MOE_NORM_NONE) row_stats<NC>(sum, a.after, y, col, a.d, a.eps, mean, rstd);
      const long long gate_row = a.gate.p != nullptr ? row / a.gate_rows : 0;
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[c][i] = (y[c][i] - mean) * rstd;
          g[c][i] *= a.beta;
        }
        if (a.drop.rng != nullptr) {
          drop8(a.drop, ds, (uint32_t)row, (uint32_t)col[c], v);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[c][i] = v[i] != 0.f ? g[c][i] * v[i] : 0.f;
        }
        float w[8], b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w[i] = col[c] + i < a.d ? 1.f : 0.f;  // what is past the row's end adds nothing to its means
          b[i] = 0.f;
        }
        if (a.w_after.p != nullptr) load8(a.w_after, 0, col[c], a.d, w);
        if (a.b_after.p != nullptr) load8(a.b_after, 0, col[c], a.d, b);
        if (a.gate.p != nullptr) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            // a dropped element is 0 whatever u is
            const float u = fmaf(y[c][i], w[i], b[i]);
            v[i] = g[c][i] != 0.f ? g[c][i] * u : 0.f;
          }
          if (sum_gates) {
#pragma unroll
            for (int i = 0; i < 8; ++i) ga[c][i] += v[i];
          } else if (a.d_gate != nullptr) {
            const RowsOut out{a.d_gate, a.d, MOE_DTYPE_F32, a.d % 8 == 0};
            store8(out, row, col[c], a.d, v);
          }
          load8(a.gate, gate_row, col[c], a.d, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[c][i] *= v[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          wa[c][i] = fmaf(g[c][i], y[c][i], wa[c][i]);
          if constexpr (BIAS) ba[c][i] += g[c][i];
          g[c][i] *= w[i];
          m[0] = fmaf(g[c][i], y[c][i], m[0]);
          m[1] += g[c][i];
        }
      }
      if (a.after != MOE_NORM_NONE) {
        sum(m);
        m[0] *= inv;
        m[1] = a.after == MOE_NORM_LAYER ? m[1] * inv : 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            g[c][i] = rstd * (g[c][i] - fmaf(y[c][i], m[0], m[1]));
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) store8(a.d_y, row, col[c], a.d, g[c]);
    }
    if (sum_gates && a.d_gate != nullptr) {
      const long long first = s0 / a.gate_rows * a.gate_rows;
      const bool whole = first >= r0 && (s1 < r1 || s1 == a.T || s1 % a.gate_rows == 0);
      float* dst = whole ? a.d_gate + s0 / a.gate_rows * a.d : part + (first < r0 ? 4 : 5) * a.d;
      flush<R, NC>(ga, stage, group, tid, col, a.d, dst);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) ga[c][i] = 0.f;
    }
    s0 = s1;
  }
  if (a.d_w_after != nullptr) flush<R, NC>(wa, stage, group, tid, col, a.d, part);
  if (a.d_w_before != nullptr) flush<R, NC>(wb, stage, group, tid, col, a.d, part + 2 * a.d);
  if constexpr (BIAS) {
    if (a.d_b_after != nullptr) flush<R, NC>(ba, stage, group, tid, col, a.d, part + a.d);
    if (a.d_b_before != nullptr) flush<R, NC>(bb, stage, group, tid, col, a.d, part + 3 * a.d);
  }
}

// Adds the CTAs' partial sums in order: blockIdx.y 0-3 a parameter, then the rows of gates that CTAs share
// (row y - 4, or the row at the boundary of CTAs y - 4 and y - 3 where there are fewer of those).
constexpr int kJoinCols = 32, kJoinSlices = 16;
__global__ void __launch_bounds__(kJoinCols* kJoinSlices)
    norm_join_kernel(const __grid_constant__ NormGradArgs a, int ctas) {
  __shared__ float s[kJoinSlices][kJoinCols];
  const int x = threadIdx.x % kJoinCols, slice = threadIdx.x / kJoinCols;
  const int c = blockIdx.x * kJoinCols + x, y = blockIdx.y;
  const int per = rows_per_cta(a.T, ctas);
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

template <int R, int NC, int CL>
int ctas_form(int T) {
  constexpr int groups = grad_threads<R>() / R;
  const int most = R == 512 ? num_sms() / CL : 2 * num_sms();
  const int n = most < kNormMaxCtas ? most : kNormMaxCtas;
  const int need = (int)(((long long)T + groups - 1) / groups);
  const int ctas = need < n ? need : n;
  // no CTA without a token: the runs are equal, so fewer may do
  return (T + rows_per_cta(T, ctas) - 1) / rows_per_cta(T, ctas);
}

template <int R, int NC, int CL>
cudaError_t launch_form(const NormGradArgs& a, cudaStream_t st) {
  const int ctas = ctas_form<R, NC, CL>(a.T);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas * CL);
  cfg.blockDim = dim3(grad_threads<R>());
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL > 1 ? 2 : 1;
  const cudaError_t e =
      a.d_b_after != nullptr || a.d_b_before != nullptr
          ? cudaLaunchKernelEx(&cfg, norm_grad_kernel<R, NC, CL, true>, a)
          : cudaLaunchKernelEx(&cfg, norm_grad_kernel<R, NC, CL, false>, a);
  if (e != cudaSuccess) return e;
  int shared = 0;  // rows of gates that CTAs may share
  if (a.d_gate != nullptr && a.gate_rows > 1) {
    const long long groups = ((long long)a.T + a.gate_rows - 1) / a.gate_rows;
    shared = (int)(groups < ctas - 1 ? groups : ctas - 1);
  }
  if (!a.d_w_after && !a.d_b_after && !a.d_w_before && !a.d_b_before && shared == 0)
    return cudaSuccess;
  return launch_k(norm_join_kernel, dim3((a.d + kJoinCols - 1) / kJoinCols, 4 + shared),
                  dim3(kJoinCols * kJoinSlices), 0, st, a, ctas);
}

}  // namespace

cudaError_t launch_norm_grad(const NormGradArgs& a, cudaStream_t st) {
  return MOE_NORM_FORMS(launch_form, a.d, a, st);
}

}  // namespace moe
