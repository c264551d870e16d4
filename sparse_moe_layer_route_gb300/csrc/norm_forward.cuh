// Norms before and after a block with residual, gate and dropout (forward).
//
//   h' = alpha h + beta gate * drop(norm_after(y)),   n = norm_before(h')
//
// One pass: a row is read once, its sums are taken in registers (layer norm's variance in a second sum around
// the mean), and h' and n are written; the bytes of h, y, h' and n bound it. CTAs are persistent, and while
// a row is worked on, the next ones' copies are under way. Instructions are close behind the bytes (44 an
// element is what the SMs issue in the time of 8 bytes): types are the kernel's, not looked up, and a
// thread has up to 32 channels to pay for a row's sums and addresses.
//
// Measured: 16384 x 7168, rms norms, gates per channel, bf16: 150 us (940 MB, 6.3 TB/s); 3001 x 1027, layer norms with
// biases, gates per sequence, dropout (rows of any alignment, one element at a time): 26 us; 16 x 7168: 7.4 us, the
// call's.
#pragma once
#include "norm_rows.cuh"

namespace moe {
namespace {

template <int R, int NC>
constexpr int forward_ctas() {  // per SM: registers for the values of a row
  return NC == 4 ? 2 : 3;
}

template <int R, int NC, bool CLUSTER, class H, class Y>
__global__ void __launch_bounds__(norm_threads<R>(), forward_ctas<R, NC>())
    norm_kernel(const __grid_constant__ NormArgs a, int cl, int stages) {
  constexpr int kGroups = norm_threads<R>() / R;
  constexpr bool kAny = std::is_same_v<H, Any>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float red[kGroups][RowSum<R, CLUSTER>::kFloats];
  const int group = kGroups == 1 ? 0 : threadIdx.x / R, tid = threadIdx.x % R, lane = tid % 32;
  const int rank = CLUSTER ? (int)blockIdx.x % cl : 0;
  const int base = CLUSTER ? rank * norm_width(a.d, cl) : 0;
  const int d = CLUSTER ? min(a.d, base + norm_width(a.d, cl)) : a.d;  // this CTA's channels end there
  const int live = live_warps<R, CLUSTER>(d);
  RowSum<R, CLUSTER> sum(red[group], group, cl, live);
  const int w0 = base + tid / 32 * kWarpCols;  // channels of chunk c: w0 + c * R * 8 + lane * 8 + 0..7
  const bool block = a.y.p != nullptr;
  // the warp's memory: [stage] of h and y, then `turn`
  using In = Input<H, R, NC>;
  using InY = Input<Y, R, NC>;
  const uint32_t pitch = In::bytes(a.h.dtype) + (block ? InY::bytes(a.y.dtype) : 0);
  uint8_t* mine = smem + threadIdx.x / 32 * (stages * pitch + (kAny ? kWarpCols * 4 : 0));
  float* turn = reinterpret_cast<float*>(mine + stages * pitch);
  const uint32_t sh = ptx::smem_u32(mine), sy = sh + In::bytes(a.h.dtype);
  for (int i = 0; i < stages; ++i) {
    In::clear(a.h, w0, lane, d, sh + i * pitch);
    if (block) InY::clear(a.y, w0, lane, d, sy + i * pitch);
  }
  const int step = (int)(gridDim.x / cl) * kGroups;
  const long long first = (long long)(blockIdx.x / cl) * kGroups + group;
  const float inv = 1.f / (float)a.d;
  int col[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) col[c] = w0 + c * R * 8 + lane * 8;
  griddep_wait();
  if (tid / 32 >= live) return;
  const DropState ds(a.drop);
  int next = first < a.T ? (int)first : a.T;
  auto bring = [&](uint32_t stage) {
    if (next < a.T) {
      if (block) InY::fetch(a.y, next, w0, lane, d, sy + stage);
      In::fetch(a.h, next, w0, lane, d, sh + stage);
      next = step < a.T - next ? next + step : a.T;
    }
    copies_commit();
  };
  for (int i = 0; i < stages; ++i) bring(i * pitch);
  sum.all_started();
  uint32_t stage = 0;
  for (long long r = first; r < a.T; r += step) {
    const int row = (int)r;
    copies_wait_stage(stages);
    __syncwarp();
    F2 x[NC][4];  // y, then h'
    if (block) {
#pragma unroll
      for (int c = 0; c < NC; ++c) InY::read(a.y, c, lane, sy + stage, x[c]);
      float mean = 0.f, rstd = 1.f;
      if (a.after != MOE_NORM_NONE)
        row_stats<NC, kAny>(sum, a.after, x, col, d, inv, a.eps, mean, rstd);
      // beta goes with the deviation, and with the bias below
      scale_rows<NC>(x, a.after == MOE_NORM_LAYER, mean, rstd * a.beta);
      if (a.w_after.p != nullptr) times_params<kAny>(a.w_after, 0, col, d, x);
      if (a.b_after.p != nullptr) {
        const F2 beta = twice(a.beta);
        with_params<kAny>(a.b_after, 0, col, d, [&](int c, const F2 (&w)[4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[c][i] = fma2(w[i], beta, x[c][i]);
        });
      }
      if (a.drop.rng != nullptr) {
#pragma unroll
        for (int c = 0; c < NC; ++c) if (!kAny || w0 + c * R * 8 < d) drop8(a.drop, ds, row, col[c], x[c]);
      }
      if (a.gate.p != nullptr) {
        const uint32_t gate_row = a.gate_rows < a.T ? (uint32_t)row / (uint32_t)a.gate_rows : 0;
        times_params<kAny>(a.gate, gate_row, col, d, x);
      }
      const F2 alpha = twice(a.alpha);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        F2 v[4];
        In::read(a.h, c, lane, sh + stage, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[c][i] = fma2(alpha, v[i], x[c][i]);
      }
      if (kAny || a.after == MOE_NORM_LAYER) {
        // a layer norm leaves something of its mean past the row's end
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (kAny || col[c] >= d) each(x[c], [&](int i, float v) { return col[c] + i < d ? v : 0.f; });
      }
    } else {
      const F2 alpha = twice(a.alpha);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        In::read(a.h, c, lane, sh + stage, x[c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[c][i] = mul2(alpha, x[c][i]);
      }
    }
    __syncwarp();  // the stage is read; its next row may come
    bring(stage);
    stage = stage + pitch == stages * pitch ? 0 : stage + pitch;
    if (a.h_out.p != nullptr) {
#pragma unroll
      for (int c = 0; c < NC; ++c) store<H, R>(a.h_out, row, c, w0, lane, d, x[c], turn);
    }
    if (a.before != MOE_NORM_NONE) {
      float mean, rstd;
      row_stats<NC, kAny>(sum, a.before, x, col, d, inv, a.eps, mean, rstd);
      scale_rows<NC>(x, a.before == MOE_NORM_LAYER, mean, rstd);
      if (a.w_before.p != nullptr) times_params<kAny>(a.w_before, 0, col, d, x);
      if (a.b_before.p != nullptr)
        with_params<kAny>(a.b_before, 0, col, d, [&](int c, const F2 (&w)[4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[c][i] = add2(x[c][i], w[i]);
        });
#pragma unroll
      for (int c = 0; c < NC; ++c) store<Y, R>(a.n, row, c, w0, lane, d, x[c], turn);
    }
  }
  copies_wait<0>();
}

template <int R, int NC, bool CLUSTER, class H, class Y>
cudaError_t launch_form(const NormArgs& a, int cl, cudaStream_t st) {
  constexpr int groups = norm_threads<R>() / R;
  const int threads = groups > 1 ? norm_threads<R>() : 32 * live_warps<R, CLUSTER>(a.d);
  const int per_sm = forward_ctas<R, NC>() * norm_threads<R>() / threads;
  const int pitch = Input<H, R, NC>::bytes(a.h.dtype) +
                    (a.y.p != nullptr ? Input<Y, R, NC>::bytes(a.y.dtype) : 0);
  const int turn = std::is_same_v<H, Any> ? kWarpCols * 4 : 0;
  const long long need = ((long long)a.T + groups - 1) / groups, most = (long long)per_sm * num_sms() / cl;
  // rows under way: as many as a CTA has and its share of shared memory holds, four at most
  const long long rows = (need + most - 1) / most;
  int stages = rows < 4 ? (int)rows : 4;
  auto smem = [&] { return threads / 32 * (stages * pitch + turn); };
  while (stages > 1 && smem() > kNormSmem / per_sm - 2048) --stages;
  return launch_rows<CLUSTER>(norm_kernel<R, NC, CLUSTER, H, Y>, (int)(need < most ? need : most) * cl,
                              threads, smem(), cl, st, a, cl, stages);
}

// The narrowest form that holds a row, as what a form has past the row's end costs as much as channels do (3001 rows
// of 1024, layer norms, gates and dropout: 14 us with one chunk of 128 threads, 19 with two; 50000 of 128: 40 us with
// one chunk of a warp, 57 with two; but 20000 of 512 32 us so, 41 with one chunk of 64 threads). With one chunk of 256
// threads a CTA has as many warps as the row needs: up to six of the eight that is faster than two chunks of 128
// threads (1027 channels: 26 us instead of 31; 1800: 26 instead of 23).
template <class H, class Y>
cudaError_t launch_forward(const NormArgs& a, cudaStream_t st) {
  const int d = a.d;
  if (d <= 256) return launch_form<32, 1, false, H, Y>(a, 1, st);
  if (d <= 512) return launch_form<32, 2, false, H, Y>(a, 1, st);
  if (d <= 1024) return launch_form<128, 1, false, H, Y>(a, 1, st);
  if (d <= 1536) return launch_form<256, 1, false, H, Y>(a, 1, st);
  if (d <= 2048) return launch_form<128, 2, false, H, Y>(a, 1, st);
  if (d <= 4096) return launch_form<256, 2, false, H, Y>(a, 1, st);
  if (d <= 8192) return launch_form<256, 4, false, H, Y>(a, 1, st);
  return launch_form<256, 4, true, H, Y>(a, norm_cluster(d), st);
}

}  // namespace
}  // namespace moe
