// Gradients of the norms around a block (forward: norm_forward.cuh). With hats for normed values before w and
// b, D = d_h_out, N = d_n:
//   G  = D + r_b (N w_b - h^ mean(N w_b h^) - mean(N w_b))      gradient to h' (last mean: layer norm)
//   d_h = alpha G
//   E  = beta G m gate                                          to u, m: dropout's factor
//   d_y = r_a (E w_a - y^ mean(E w_a y^) - mean(E w_a))
// and over the tokens d_gate = sum beta G m u, d_w_a = sum E y^, d_b_a = sum E, d_w_b = sum N h^, d_b_b = sum N.
//
// One pass as in the forward direction: h', y, D and N are read once, the statistics are taken again from them
// (cheaper than keeping them), d_h and d_y written. Every CTA has a run of consecutive tokens and adds up the
// parameters' gradients, a thread its own channels (those of w and the gates in registers, the biases',
// which few have, in shared memory); the CTAs' sums go to the workspace and are added there in order by a
// second, small kernel. A row of gates whose tokens are all in one CTA's run is complete there; one that
// is shared leaves a partial sum in each.
#pragma once
#include "norm_rows.cuh"

namespace moe {
namespace {

// Sums of the CTA's row groups for their channels [first, d), in order, to dst (fp32). Where there are several,
// `stage` has room for all groups' channels.
template <int R, int NC>
constexpr int stage_bytes() {
  return norm_threads<R>() == R ? 0 : norm_threads<R>() * NC * 8 * 4;
}
template <int R, int NC>
__device__ __forceinline__ void flush(const F2 (&acc)[NC][4], float* stage, int group, int w0, int lane,
                                      int first, int d, float* dst) {
  constexpr int kGroups = norm_threads<R>() / R, kWidth = R * NC * 8;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = w0 + c * R * 8 + lane * 8 + 2 * i;
        const float2 v = both(acc[c][i]);
        if (k < d) dst[k] = v.x;
        if (k + 1 < d) dst[k + 1] = v.y;
      }
    return;
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    F2* to = reinterpret_cast<F2*>(stage + group * kWidth + w0 - first + c * R * 8 + lane * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = acc[c][i];
  }
  __syncthreads();
  for (int k = threadIdx.x; first + k < d && k < kWidth; k += norm_threads<R>()) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) s += stage[g * kWidth + k];
    dst[first + k] = s;
  }
}

// v added to a lane's eight sums in shared memory, 16 bytes of every lane side by side.
__device__ __forceinline__ void add_shared(float* sums, int lane, const F2 (&v)[4]) {
  ulonglong2* at = reinterpret_cast<ulonglong2*>(sums) + lane;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    ulonglong2 s = at[32 * k];
    s.x = add2(s.x, v[2 * k]);
    s.y = add2(s.y, v[2 * k + 1]);
    at[32 * k] = s;
  }
}
__device__ __forceinline__ void get_shared(const float* sums, int lane, F2 (&v)[4]) {
  const ulonglong2* at = reinterpret_cast<const ulonglong2*>(sums) + lane;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const ulonglong2 s = at[32 * k];
    v[2 * k] = s.x;
    v[2 * k + 1] = s.y;
  }
}

// A thread's share of sum(g x) and, for a layer norm, sum(g).
template <int NC>
__device__ __forceinline__ void sums_of(const F2 (&g)[NC][4], const F2 (&x)[NC][4], bool layer, float (&m)[2]) {
  F2 s[2] = {0, 0}, t[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i & 1] = fma2(g[c][i], x[c][i], s[i & 1]);
  if (layer) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i & 1] = add2(g[c][i], t[i & 1]);
  }
  const float2 a = both(add2(s[0], s[1])), b = both(add2(t[0], t[1]));
  m[0] = a.x + a.y;
  m[1] = b.x + b.y;
}
// g = r (g - x p - q): a gradient to normed values x becomes one to what was normed.
template <int NC>
__device__ __forceinline__ void through_norm(F2 (&g)[NC][4], const F2 (&x)[NC][4], float p, float q, float r) {
  const F2 np = twice(-p), nq = twice(-q), rr = twice(r);
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) g[c][i] = mul2(rr, add2(g[c][i], fma2(x[c][i], np, nq)));
}

// Shared memory of a CTA: what flush needs, and for each warp the biases' sums, `stages` rows of its inputs and
// what turns rows round.
template <int NC, class H, class Y>
__host__ __device__ __forceinline__ int grad_pitch(const NormGradArgs& a) {
  const int h = NC * kWarpCols * bytes_of<H>(a.d_h.dtype), y = NC * kWarpCols * bytes_of<Y>(a.y.dtype);
  return (a.d_h_out.p != nullptr ? h : 0) + (a.d_n.p != nullptr ? h + y : 0) + (a.y.p != nullptr ? y : 0);
}
template <int NC>
__host__ __device__ __forceinline__ int bias_bytes(const NormGradArgs& a) {
  return ((a.d_b_after != nullptr) + (a.d_b_before != nullptr)) * NC * kWarpCols * 4;  // of a warp
}

template <int R, int NC, bool CLUSTER, class H, class Y>
__global__ void __launch_bounds__(norm_threads<R>(), R == 512 ? 1 : 2)
    norm_grad_kernel(const __grid_constant__ NormGradArgs a, int cl, int stages) {
  constexpr int kGroups = norm_threads<R>() / R;
  constexpr bool kAny = std::is_same_v<H, Any>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float red[kGroups][RowSum<R, CLUSTER>::kFloats];
  const int group = kGroups == 1 ? 0 : threadIdx.x / R, tid = threadIdx.x % R, lane = tid % 32;
  const int cta = blockIdx.x / cl, ctas = gridDim.x / cl;
  const int rank = CLUSTER ? (int)blockIdx.x % cl : 0;
  const int base = CLUSTER ? rank * norm_width(a.d, cl) : 0;
  const int d = CLUSTER ? min(a.d, base + norm_width(a.d, cl)) : a.d;  // this CTA's channels end there
  const int per = norm_rows_per_cta(a.T, ctas);
  const long long r0 = (long long)cta * per, r1 = r0 + per < a.T ? r0 + per : a.T;
  RowSum<R, CLUSTER> sum(red[group], group, cl);
  const int w0 = base + tid / 32 * kWarpCols;  // channels of chunk c: w0 + c * R * 8 + lane * 8 + 0..7
  const float inv = 1.f / (float)a.d;
  const bool normed = a.d_n.p != nullptr;  // the norm before the next block has a gradient
  const bool block = a.y.p != nullptr, direct = a.d_h_out.p != nullptr;
  float* stage_s = reinterpret_cast<float*>(smem);
  // the warp's memory: sums of the biases, [stage] of h, d_n, d_h_out and y, then `turn`
  const uint32_t pitch = grad_pitch<NC, H, Y>(a);
  uint8_t* mine = smem + stage_bytes<R, NC>() +
                  threadIdx.x / 32 * (bias_bytes<NC>(a) + stages * pitch + (kAny ? kWarpCols * 4 : 0));
  float* sums_bb = reinterpret_cast<float*>(mine);
  float* sums_ba = sums_bb + (a.d_b_before != nullptr ? NC * kWarpCols : 0);
  mine += bias_bytes<NC>(a);
  float* turn = reinterpret_cast<float*>(mine + stages * pitch);
  Input<H, R, NC> h_in, g_in;
  Input<Y, R, NC> n_in, y_in;
  {
    uint32_t at = ptx::smem_u32(mine);
    if (normed) {
      h_in.init(a.h, w0, lane, at);
      at += h_in.bytes(a.h.dtype);
      n_in.init(a.d_n, w0, lane, at);
      at += n_in.bytes(a.d_n.dtype);
    }
    if (direct) {
      g_in.init(a.d_h_out, w0, lane, at);
      at += g_in.bytes(a.d_h_out.dtype);
    }
    if (block) y_in.init(a.y, w0, lane, at);
    for (int i = 0; i < stages; ++i) {
      if (normed) h_in.clear(w0, lane, d, i * pitch), n_in.clear(w0, lane, d, i * pitch);
      if (direct) g_in.clear(w0, lane, d, i * pitch);
      if (block) y_in.clear(w0, lane, d, i * pitch);
    }
    for (int i = lane; i < bias_bytes<NC>(a) / 4; i += 32) sums_bb[i] = 0.f;
    __syncwarp();
  }
  griddep_wait();
  const DropState ds(a.drop);
  float* part = a.part + (size_t)cta * kNormParts * a.d;
  // the tokens are taken in the same order whether or not the gates' gradient is wanted, so that the others
  // do not depend on it
  const bool sum_gates = a.gate.p != nullptr && a.gate_rows > 1;
  // a segment: tokens with the same row of gates, dealt out to the row groups
  auto segment_end = [&](long long s0) {
    if (!sum_gates) return r1;
    const long long end = (s0 / a.gate_rows + 1) * a.gate_rows;
    return end < r1 ? end : r1;
  };
  // this group's next token to bring and the end of its segment
  long long next = r0 + group, next_end = segment_end(r0);
  auto settle = [&] {
    while (next >= next_end && next_end < r1) {
      next = next_end + group;
      next_end = segment_end(next_end);
    }
  };
  settle();
  auto bring = [&](uint32_t stage) {
    if (next < next_end) {
      if (normed) {
        h_in.fetch(next, w0, lane, d, stage);
        n_in.fetch(next, w0, lane, d, stage);
      }
      if (direct) g_in.fetch(next, w0, lane, d, stage);
      if (block) y_in.fetch(next, w0, lane, d, stage);
      next += kGroups;
      if (next >= next_end) settle();
    }
    copies_commit();
  };
  for (int i = 0; i < stages; ++i) bring(i * pitch);
  uint32_t stage = 0;
  F2 wa[NC][4] = {}, wb[NC][4] = {}, ga[NC][4] = {};
  int col[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) col[c] = w0 + c * R * 8 + lane * 8;
  for (long long s0 = r0; s0 < r1;) {
    const long long s1 = segment_end(s0);
    for (long long row = s0 + group; row < s1; row += kGroups) {
      copies_wait_stage(stages);
      __syncwarp();
      F2 g[NC][4];
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) g[c][i] = 0;
      if (normed) {
        F2 h[NC][4];
#pragma unroll
        for (int c = 0; c < NC; ++c) h_in.read(c, lane, stage, h[c]);
        float mean, rstd;
        row_stats<NC, kAny>(sum, a.before, h, col, d, inv, a.eps, mean, rstd);
        scale_rows<NC>(h, a.before == MOE_NORM_LAYER, mean, rstd);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          n_in.read(c, lane, stage, g[c]);
#pragma unroll
          for (int i = 0; i < 4; ++i) wb[c][i] = fma2(g[c][i], h[c][i], wb[c][i]);
        }
        if (a.d_b_before != nullptr) {
#pragma unroll
          for (int c = 0; c < NC; ++c) add_shared(sums_bb + c * kWarpCols, lane, g[c]);
        }
        if (a.w_before.p != nullptr) times_params<kAny>(a.w_before, 0, col, d, g);
        float m[2];
        sums_of<NC>(g, h, a.before == MOE_NORM_LAYER, m);
        sum(m);
        through_norm<NC>(g, h, m[0] * inv, m[1] * inv, rstd);
      }
      if (direct) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          F2 v[4];
          g_in.read(c, lane, stage, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) g[c][i] = add2(g[c][i], v[i]);
        }
      }
      {
        const F2 alpha = twice(a.alpha);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          F2 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = mul2(alpha, g[c][i]);
          store<H>(a.d_h, row, w0 + c * R * 8, lane, d, v, turn);
        }
      }
      if (block) {
        F2 y[NC][4];
#pragma unroll
        for (int c = 0; c < NC; ++c) y_in.read(c, lane, stage, y[c]);
        float mean = 0.f, rstd = 1.f;
        if (a.after != MOE_NORM_NONE) {
          row_stats<NC, kAny>(sum, a.after, y, col, d, inv, a.eps, mean, rstd);
          scale_rows<NC>(y, a.after == MOE_NORM_LAYER, mean, rstd);
        }
        const F2 beta = twice(a.beta);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
#pragma unroll
          for (int i = 0; i < 4; ++i) g[c][i] = mul2(g[c][i], beta);
          if (a.drop.rng != nullptr) drop8(a.drop, ds, (uint32_t)row, (uint32_t)col[c], g[c]);
        }
        if (a.gate.p != nullptr) {
          const uint32_t gate_row = a.gate_rows < a.T ? (uint32_t)row / (uint32_t)a.gate_rows : 0;
          if (a.d_gate != nullptr) {
            F2 u[NC][4];
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
              for (int i = 0; i < 4; ++i) u[c][i] = y[c][i];
            if (a.w_after.p != nullptr) times_params<kAny>(a.w_after, 0, col, d, u);
            if (a.b_after.p != nullptr)
              with_params<kAny>(a.b_after, 0, col, d, [&](int c, const F2 (&w)[4]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) u[c][i] = add2(u[c][i], w[i]);
              });
            if (a.drop.rng != nullptr) {  // a dropped element is 0 whatever u is
#pragma unroll
              for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 e = both(g[c][i]), v = both(u[c][i]);
                  u[c][i] = pair(e.x != 0.f ? v.x : 0.f, e.y != 0.f ? v.y : 0.f);
                }
            }
            if (sum_gates) {
#pragma unroll
              for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) ga[c][i] = fma2(g[c][i], u[c][i], ga[c][i]);
            } else {
              const RowsOut out{a.d_gate, a.d, MOE_DTYPE_F32, true};
#pragma unroll
              for (int c = 0; c < NC; ++c) {
#pragma unroll
                for (int i = 0; i < 4; ++i) u[c][i] = mul2(g[c][i], u[c][i]);
                store<std::conditional_t<kAny, Any, F32>>(out, row, w0 + c * R * 8, lane, d, u[c], turn);
              }
            }
          }
          times_params<kAny>(a.gate, gate_row, col, d, g);
        }
        // what is past the row's end adds nothing to its means
        if (kAny || a.after == MOE_NORM_LAYER || a.before == MOE_NORM_LAYER) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (kAny || col[c] >= d) each(g[c], [&](int i, float v) { return col[c] + i < d ? v : 0.f; });
        }
        if (a.after != MOE_NORM_NONE) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) wa[c][i] = fma2(g[c][i], y[c][i], wa[c][i]);
          if (a.d_b_after != nullptr) {
#pragma unroll
            for (int c = 0; c < NC; ++c) add_shared(sums_ba + c * kWarpCols, lane, g[c]);
          }
          if (a.w_after.p != nullptr) times_params<kAny>(a.w_after, 0, col, d, g);
          float m[2];
          sums_of<NC>(g, y, a.after == MOE_NORM_LAYER, m);
          sum(m);
          through_norm<NC>(g, y, m[0] * inv, m[1] * inv, rstd);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
          store<Y>(a.d_y, row, w0 + c * R * 8, lane, d, g[c], turn);
      }
      __syncwarp();  // the stage is read; its next row may come
      bring(stage);
      stage = stage + pitch == stages * pitch ? 0 : stage + pitch;
    }
    if (sum_gates && a.d_gate != nullptr) {
      const long long first = s0 / a.gate_rows * a.gate_rows;
      const bool whole = first >= r0 && (s1 < r1 || s1 == a.T || s1 % a.gate_rows == 0);
      float* dst = whole ? a.d_gate + s0 / a.gate_rows * a.d : part + (first < r0 ? 4 : 5) * a.d;
      flush<R, NC>(ga, stage_s, group, w0, lane, base, d, dst);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) ga[c][i] = 0;
    }
    s0 = s1;
  }
  copies_wait<0>();
  if (a.d_w_after != nullptr) flush<R, NC>(wa, stage_s, group, w0, lane, base, d, part);
  if (a.d_w_before != nullptr) flush<R, NC>(wb, stage_s, group, w0, lane, base, d, part + 2 * a.d);
  if (a.d_b_after != nullptr) {
#pragma unroll
    for (int c = 0; c < NC; ++c) get_shared(sums_ba + c * kWarpCols, lane, wa[c]);
    flush<R, NC>(wa, stage_s, group, w0, lane, base, d, part + a.d);
  }
  if (a.d_b_before != nullptr) {
#pragma unroll
    for (int c = 0; c < NC; ++c) get_shared(sums_bb + c * kWarpCols, lane, wa[c]);
    flush<R, NC>(wa, stage_s, group, w0, lane, base, d, part + 3 * a.d);
  }
}

template <int R, int NC, bool CLUSTER, class H, class Y>
cudaError_t launch_grad_form(const NormGradArgs& a, int cl, int* ctas, cudaStream_t st) {
  constexpr int threads = norm_threads<R>(), groups = threads / R, per_sm = R == 512 ? 1 : 2;
  // one stage of four 32-bit inputs, both biases' sums and what turns rows round: 208 KB
  static_assert(16 * (2 * 2 * 1024 + 4 * 2 * 1024 + 1024) <= kNormSmem - 2048, "the widest form fits");
  const int pitch = grad_pitch<NC, H, Y>(a), turn = std::is_same_v<H, Any> ? kWarpCols * 4 : 0;
  // rows under way: as many as a CTA's share of shared memory holds, four at most
  int stages = 4;
  auto smem = [&] {
    return stage_bytes<R, NC>() + threads / 32 * (bias_bytes<NC>(a) + stages * pitch + turn);
  };
  while (stages > 1 && smem() > kNormSmem / per_sm - 2048) --stages;
  const int room = per_sm * num_sms() / cl;
  const int most = room < kNormMaxCtas ? room : kNormMaxCtas;
  const long long need = ((long long)a.T + groups - 1) / groups;
  *ctas = (int)(need < most ? need : most);
  const int per = norm_rows_per_cta(a.T, *ctas);
  *ctas = (int)(((long long)a.T + per - 1) / per);  // the runs are equal, so fewer may do
  return launch_rows<CLUSTER>(norm_grad_kernel<R, NC, CLUSTER, H, Y>, *ctas * cl, threads, smem(), cl, st, a,
                              cl, stages);
}

template <class H, class Y>
cudaError_t launch_backward(const NormGradArgs& a, int* ctas, cudaStream_t st) {
  const int d = a.d;
  if (d <= 512) return launch_grad_form<32, 2, false, H, Y>(a, 1, ctas, st);
  if (d <= 2048) return launch_grad_form<128, 2, false, H, Y>(a, 1, ctas, st);
  if (d <= 4096) return launch_grad_form<256, 2, false, H, Y>(a, 1, ctas, st);
  if (d <= 8192) return launch_grad_form<512, 2, false, H, Y>(a, 1, ctas, st);
  int cl = 2;
  while (norm_width(d, cl) > 8192) cl *= 2;
  return launch_grad_form<512, 2, true, H, Y>(a, cl, ctas, st);
}

}  // namespace
}  // namespace moe
