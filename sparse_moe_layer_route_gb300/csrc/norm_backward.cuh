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
//
// Measured: 8192 x 4096, rms norms, a 32-bit stream, gates per channel, dropout: 156 us (604 MB, 3.9 TB/s). A thread
// holds a row's values and the sums of its channels, up to 128 registers, so 16 warps an SM have to cover two sums
// over the row in a chain of some 95 instructions an element (issue 44 % of peak). 2051 x 2048, a layer norm before the next block
// only, gates per sequence: 27 us. 8192 x 7168, bf16, rms norms, gates per channel: 251 us (704 MB, 2.8 TB/s), without
// gates and a norm after 133: above 4096 channels a thread has two chunks, whose sums and values are more than its 128
// registers (128 to 152 bytes spilled, of a cluster's rows 164 to 216, of rows of any alignment 404 to 416; waits for
// memory are the first stall). All with the joining kernel.
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

// a + b, but not past the end (token numbers go up to 2^31 - 1).
__device__ __forceinline__ int at_most(int a, int b, int end) { return b < end - a ? a + b : end; }

// LAYER: a norm may be a layer norm, whose sums follow one another; others' are taken together.
template <int R, int NC, bool CLUSTER, class H, class Y, bool LAYER>
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
  const int r0 = (int)((long long)cta * per), r1 = at_most(r0, per, a.T);
  // where there are several groups, all their threads meet to write sums
  const int live = kGroups > 1 ? R / 32 : live_warps<R, CLUSTER>(d);
  RowSum<R, CLUSTER> sum(red[group], group, cl, live);
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
  using In = Input<H, R, NC>;
  using InY = Input<Y, R, NC>;
  const uint32_t sh = ptx::smem_u32(mine);
  const uint32_t sn = sh + (normed ? In::bytes(a.d_h.dtype) : 0);
  const uint32_t sg = sn + (normed ? InY::bytes(a.y.dtype) : 0);
  const uint32_t sy = sg + (direct ? In::bytes(a.d_h.dtype) : 0);
  {
    for (uint32_t i = 0; i < stages * pitch; i += pitch) {
      if (normed) In::clear(a.h, w0, lane, d, sh + i), InY::clear(a.d_n, w0, lane, d, sn + i);
      if (direct) In::clear(a.d_h_out, w0, lane, d, sg + i);
      if (block) InY::clear(a.y, w0, lane, d, sy + i);
    }
    for (int i = lane; i < bias_bytes<NC>(a) / 4; i += 32) sums_bb[i] = 0.f;
    __syncwarp();
  }
  griddep_wait();
  if (tid / 32 >= live) return;
  const DropState ds(a.drop);
  float* part = a.part + (size_t)cta * kNormParts * a.d;
  // the tokens are taken in the same order whether or not the gates' gradient is wanted, so that the others
  // do not depend on it
  const bool sum_gates = a.gate.p != nullptr && a.gate_rows > 1;
  // a segment: tokens with the same row of gates, dealt out to the row groups
  auto segment_end = [&](int s0) {
    if (!sum_gates) return r1;
    const uint32_t end = ((uint32_t)s0 / (uint32_t)a.gate_rows + 1) * (uint32_t)a.gate_rows;  // up to 2^32 - 2
    return end < (uint32_t)r1 ? (int)end : r1;
  };
  // this group's next token to bring and the end of its segment
  int next = at_most(r0, group, r1), next_end = segment_end(r0);
  auto settle = [&] {
    while (next >= next_end && next_end < r1) {
      next = at_most(next_end, group, r1);
      next_end = segment_end(next_end);
    }
  };
  settle();
  auto bring = [&](uint32_t stage) {
    if (next < next_end) {
      if (normed) {
        In::fetch(a.h, next, w0, lane, d, sh + stage);
        InY::fetch(a.d_n, next, w0, lane, d, sn + stage);
      }
      if (direct) In::fetch(a.d_h_out, next, w0, lane, d, sg + stage);
      if (block) InY::fetch(a.y, next, w0, lane, d, sy + stage);
      next = at_most(next, kGroups, r1);
      if (next >= next_end) settle();
    }
    copies_commit();
  };
  for (int i = 0; i < stages; ++i) bring(i * pitch);
  sum.all_started();
  uint32_t stage = 0;
  F2 wa[NC][4] = {}, wb[NC][4] = {}, ga[NC][4] = {};
  int col[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) col[c] = w0 + c * R * 8 + lane * 8;
  for (int s0 = r0; s0 < r1;) {
    const int s1 = segment_end(s0);
    for (int row = at_most(s0, group, s1); row < s1; row = at_most(row, kGroups, s1)) {
      copies_wait_stage(stages);
      __syncwarp();
      F2 g[NC][4];
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) g[c][i] = 0;
      // what needs no other sum is summed first, all at once: squares (a layer norm's follow its mean) and, with
      // an rms norm, the product that its gradient subtracts
      F2 h[NC][4], y[NC][4];
      float hm = 0.f, hr = 1.f, ym = 0.f, yr = 1.f;
      if (normed) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          In::read(a.h, c, lane, sh + stage, h[c]);
          InY::read(a.d_n, c, lane, sn + stage, g[c]);
        }
        if (a.d_b_before != nullptr) {
#pragma unroll
          for (int c = 0; c < NC; ++c) add_shared(sums_bb + c * kWarpCols, lane, g[c]);
        }
      }
      if (!LAYER && normed) {
        float t[4];
        t[0] = dot<NC>(h, h);
        if (a.w_before.p != nullptr) times_params<kAny>(a.w_before, 0, col, d, g);
        t[1] = dot<NC>(g, h);
        t[2] = t[3] = 0.f;
        if (block && a.after == MOE_NORM_RMS) {
          F2 s[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            F2 v[4];
            InY::read(a.y, c, lane, sy + stage, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = fma2(v[i], v[i], s[i]);
          }
          t[2] = total(s[0], s[1], s[2], s[3]);
        }
        sum(t);
        hr = deviation(t[0], inv, a.eps);
        if (block && a.after == MOE_NORM_RMS) yr = deviation(t[2], inv, a.eps);
        scale_rows<NC>(h, false, 0.f, hr);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          F2 v[4];
          InY::read(a.d_n, c, lane, sn + stage, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) wb[c][i] = fma2(v[i], h[c][i], wb[c][i]);
        }
        through_norm<NC>(g, h, t[1] * hr * inv, 0.f, hr);
      } else {
        if (LAYER && normed) {
          row_stats<NC, kAny>(sum, a.before, h, col, d, inv, a.eps, hm, hr);
          scale_rows<NC>(h, a.before == MOE_NORM_LAYER, hm, hr);
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) wb[c][i] = fma2(g[c][i], h[c][i], wb[c][i]);
          if (a.w_before.p != nullptr) times_params<kAny>(a.w_before, 0, col, d, g);
          float m[2] = {dot<NC>(g, h), a.before == MOE_NORM_LAYER ? plain_sum<NC>(g) : 0.f};
          sum(m);
          through_norm<NC>(g, h, m[0] * inv, m[1] * inv, hr);
        }
        if (block && a.after != MOE_NORM_NONE) {
#pragma unroll
          for (int c = 0; c < NC; ++c) InY::read(a.y, c, lane, sy + stage, y[c]);
          row_stats<NC, kAny>(sum, a.after, y, col, d, inv, a.eps, ym, yr);
        }
      }
      if (direct) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          F2 v[4];
          In::read(a.d_h_out, c, lane, sg + stage, v);
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
          store<H, R>(a.d_h, row, c, w0, lane, d, v, turn);
        }
      }
      if (block) {
        const uint32_t gate_row =
            a.gate.p != nullptr && a.gate_rows < a.T ? (uint32_t)row / (uint32_t)a.gate_rows : 0;
        const F2 beta = twice(a.beta), ymm = twice(-ym), yrr = twice(yr);
        // e: the gradient to u, without the gate. g becomes the normed values' gradient, e gate w
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (kAny && w0 + c * R * 8 >= d) {  // nothing of the warp's is there
#pragma unroll
            for (int i = 0; i < 4; ++i) g[c][i] = y[c][i] = 0;
            continue;
          }
          Raw rw, rg;
          if (a.w_after.p != nullptr) rw = param_raw<kAny>(a.w_after, 0, col[c], d);
          if (a.gate.p != nullptr) rg = param_raw<kAny>(a.gate, gate_row, col[c], d);
          F2 e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = mul2(g[c][i], beta);
          if (a.drop.rng != nullptr) drop8(a.drop, ds, row, col[c], e);
          InY::read(a.y, c, lane, sy + stage, y[c]);
          if (LAYER && a.after == MOE_NORM_LAYER) {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[c][i] = add2(y[c][i], ymm);
          }
          if (a.after != MOE_NORM_NONE) {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[c][i] = mul2(y[c][i], yrr);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) g[c][i] = e[i];
          if (a.w_after.p != nullptr) {
            F2 w[4];
            to_float<Any>(rw, a.w_after.dtype, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) g[c][i] = mul2(g[c][i], w[i]);
          }
          if (a.gate.p != nullptr) {
            if (a.d_gate != nullptr) {
              F2 u[4];  // e u = (e w) y^ + e b
#pragma unroll
              for (int i = 0; i < 4; ++i) u[i] = mul2(g[c][i], y[c][i]);
              if (a.drop.rng != nullptr) {  // a dropped element is 0 whatever u is
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 k = both(e[i]), v = both(u[i]);
                  u[i] = pair(k.x != 0.f ? v.x : 0.f, k.y != 0.f ? v.y : 0.f);
                }
              }
              if (a.b_after.p != nullptr) {
                F2 w[4];
                to_float<Any>(param_raw<kAny>(a.b_after, 0, col[c], d), a.b_after.dtype, w);
#pragma unroll
                for (int i = 0; i < 4; ++i) u[i] = fma2(e[i], w[i], u[i]);
              }
              if (sum_gates) {
#pragma unroll
                for (int i = 0; i < 4; ++i) ga[c][i] = add2(ga[c][i], u[i]);
              } else {
                const RowsOut out{a.d_gate, a.d, MOE_DTYPE_F32, true};
                store<std::conditional_t<kAny, Any, F32>, R>(out, row, c, w0, lane, d, u, turn);
              }
            }
            F2 w[4];
            to_float<Any>(rg, a.gate.dtype, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              e[i] = mul2(e[i], w[i]);
              g[c][i] = mul2(g[c][i], w[i]);
            }
          }
          if (a.after != MOE_NORM_NONE) {
#pragma unroll
            for (int i = 0; i < 4; ++i) wa[c][i] = fma2(e[i], y[c][i], wa[c][i]);
            if (a.d_b_after != nullptr) add_shared(sums_ba + c * kWarpCols, lane, e);
          }
        }
        if (a.after != MOE_NORM_NONE) {
          // what is past the row's end adds nothing to its means
          if (kAny || LAYER) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (kAny || col[c] >= d) each(g[c], [&](int i, float v) { return col[c] + i < d ? v : 0.f; });
          }
          if (LAYER && a.after == MOE_NORM_LAYER) {
            float m[2] = {dot<NC>(g, y), plain_sum<NC>(g)};
            sum(m);
            through_norm<NC>(g, y, m[0] * inv, m[1] * inv, yr);
          } else {
            float m[1] = {dot<NC>(g, y)};
            sum(m);
            through_norm<NC>(g, y, m[0] * inv, 0.f, yr);
          }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) store<Y, R>(a.d_y, row, c, w0, lane, d, g[c], turn);
      }
      __syncwarp();  // the stage is read; its next row may come
      bring(stage);
      stage = stage + pitch == stages * pitch ? 0 : stage + pitch;
    }
    if (sum_gates && a.d_gate != nullptr) {
      const int first = s0 / a.gate_rows * a.gate_rows;
      const bool whole = first >= r0 && (s1 < r1 || s1 == a.T || s1 % a.gate_rows == 0);
      float* dst = whole ? a.d_gate + (long long)(s0 / a.gate_rows) * a.d : part + (first < r0 ? 4 : 5) * a.d;
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
  constexpr int groups = norm_threads<R>() / R;
  const int threads = groups > 1 ? norm_threads<R>() : 32 * live_warps<R, CLUSTER>(a.d), per_sm = 512 / threads;
  // one stage of four 32-bit inputs, both biases' sums and what turns rows round: 208 KB
  static_assert(16 * (2 * 2 * 1024 + 4 * 2 * 1024 + 1024) <= kNormSmem - 2048, "the widest form fits");
  const int pitch = grad_pitch<NC, H, Y>(a), turn = std::is_same_v<H, Any> ? kWarpCols * 4 : 0;
  // rows under way: as many as a CTA's share of shared memory holds, four at most
  int stages = 4;
  auto smem = [&] {
    return stage_bytes<R, NC>() + threads / 32 * (bias_bytes<NC>(a) + stages * pitch + turn);
  };
  while (stages > 1 && smem() > kNormSmem / per_sm - 2048) --stages;
  if (threads != norm_grad_threads(a.d) || cl != norm_cluster(a.d)) return cudaErrorInvalidConfiguration;
  const int most = norm_grad_runs(a.d, num_sms() < kNormMaxSms ? num_sms() : kNormMaxSms);
  const long long need = ((long long)a.T + groups - 1) / groups;
  *ctas = (int)(need < most ? need : most);
  const int per = norm_rows_per_cta(a.T, *ctas);
  *ctas = (int)(((long long)a.T + per - 1) / per);  // the runs are equal, so fewer may do
  const bool layer = a.after == MOE_NORM_LAYER || a.before == MOE_NORM_LAYER;
  if (layer || std::is_same_v<H, Any>)
    return launch_rows<CLUSTER>(norm_grad_kernel<R, NC, CLUSTER, H, Y, true>, *ctas * cl, threads, smem(), cl,
                                st, a, cl, stages);
  if constexpr (!std::is_same_v<H, Any>)
    return launch_rows<CLUSTER>(norm_grad_kernel<R, NC, CLUSTER, H, Y, false>, *ctas * cl, threads, smem(), cl,
                                st, a, cl, stages);
  return cudaErrorInvalidValue;
}

// As in the forward direction, but one chunk is faster wherever it holds a row: two chunks' sums and values are more than
// a thread's registers (3001 rows with every gradient, one chunk and two: 1024 channels 29 us and 52, 1032 37 and 54,
// 2048 53 and 67, 2304 78 and 83, 4096 113 and 110, with rms norms 71 and 81; 50000 of 128 74 and 146, 20000 of 512 76
// and 80). From 2049 channels on an SM has one CTA, with as many warps as a row has pieces: 9 at 2304, 16 at 4096 (4096
// rows, rms norms: 2560 channels 51 us of a floor of 19, 3584 60 of 26).
template <class H, class Y>
cudaError_t launch_backward(const NormGradArgs& a, int* ctas, cudaStream_t st) {
  const int d = a.d;
  if (d <= 256) return launch_grad_form<32, 1, false, H, Y>(a, 1, ctas, st);
  if (d <= 512) return launch_grad_form<64, 1, false, H, Y>(a, 1, ctas, st);
  if (d <= 1024) return launch_grad_form<128, 1, false, H, Y>(a, 1, ctas, st);
  if (d <= 2048) return launch_grad_form<256, 1, false, H, Y>(a, 1, ctas, st);
  if (d <= 4096) return launch_grad_form<512, 1, false, H, Y>(a, 1, ctas, st);
  if (d <= 8192) return launch_grad_form<512, 2, false, H, Y>(a, 1, ctas, st);
  return launch_grad_form<512, 2, true, H, Y>(a, norm_cluster(d), ctas, st);
}

}  // namespace
}  // namespace moe
