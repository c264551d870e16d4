// Grouped products of 8-bit integers for a few rows: integer dot products of four (exact in 32 bits) that read
// a segment's weights once for each of its tiles of one to eight rows.
//
// Bound by the weight bytes. A warp takes kStreams output channels (SwiGLU pass: half as many channels of
// gate and of up) of one row tile of R rows and runs down K, 16 codes a lane and step: one 16-byte load per
// channel, past L1, two steps of each in flight (4 KB a warp), and one load per row, from L1, where the
// SM's warps share the rows. The lanes' sums meet in one reduction per channel and row. A tile of
// tensor-core units has 128 channels, so a single row of a [14336 x 4096] product would occupy 56 of the
// 152 SMs for 30 us; here its 3584 warps spread over all of them: 10.2 us, 5.8 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <climits>
#include <cstdint>

#include "int8.cuh"
#include "int8_units.cuh"
#include "internal.h"

namespace moe {
namespace {

// Small CTAs, two steps and at most 85 registers: 24 warps of 4 KB in flight each on an SM, and an even
// last wave (one [14336 x 4096] row 10.2 us; with 256 threads, four steps and 16 warps 14.6 us). Eight
// rows a tile hold 32 sums and the rows' codes besides: half as many warps, without spills (8 rows of
// that product 15.8 us, with four CTAs per SM 18.3).
constexpr int kThreads = 128;
constexpr int kCtasPerSm = 6;
constexpr int kCtasPerSm8 = 3;  // tiles of eight rows
constexpr int kStreams = 4;  // channels in flight per warp
constexpr int kSteps = 2;    // 512-byte steps of each in flight

// 16 weight codes, read once: not kept in L1.
__device__ __forceinline__ int4 load_once(const int8_t* p) {
  int4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int OUT, bool SLOT>
__device__ __forceinline__ void store_one(void* out, long long at, float y) {
  if (OUT == MOE_DTYPE_F32)
    static_cast<float*>(out)[at] = y;
  else if (OUT == MOE_DTYPE_BF16)
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16(y);
  else if (SLOT)
    static_cast<uint16_t*>(out)[at] = f16_sat(y);
  else
    static_cast<__half*>(out)[at] = __float2half(y);
}

// Row tile `tile` (R rows) of the segments, counted segment by segment: found by every warp, 32 segments at a
// time. seg -1: past the last tile. unsound: some segment up to the tile's is, or with `all` any of them (the
// search for a tile ends where it is found; only the last tile's CTAs look at every segment: when each CTA did,
// 84 rows of [1476 x 1056] took 9.9 us, not 8.3).
template <int PASS, int R>
__device__ __forceinline__ Unit find_tile(const Int8Gemm& g, int tile, int lane, bool all,
                                          bool& unsound) {
  constexpr bool X_SHARED = PASS == kInt8SwiGLU;  // all shared experts read the same rows
  constexpr int kParts = (kMaxSegs + 31) / 32;
  const int n = g.n_mat + g.S;
  const int end = rows_end<PASS>(g);
  int bound[kParts][2];  // every load in flight before the first is needed
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    const int s = p * 32 + lane;
    bound[p][0] = bound[p][1] = 0;
    if (g.offsets != nullptr && s < g.n_mat) {
      bound[p][0] = g.offsets[s];
      bound[p][1] = g.offsets[s + 1];
    }
  }
  bool bad = false;
  if (all) {
#pragma unroll
    for (int p = 0; p < kParts; ++p)
      bad |= p * 32 + lane < g.n_mat && !segment_ok(bound[p][0], bound[p][1], end);
  }
  int before = 0;
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    const int s0 = p * 32, s = s0 + lane;
    if (s0 >= n) break;
    int r0 = 0, nr = 0;
    if (s < g.n_mat) {
      int r1 = g.rows;
      if (g.offsets != nullptr) {
        r0 = bound[p][0];
        r1 = bound[p][1];
        if (!segment_ok(r0, r1, end)) {
          bad = true;
          r0 = r1 = 0;
        }
      }
      nr = r1 - r0;
    } else if (s < n) {
      r0 = g.rows + (s - g.n_mat) * g.T;
      nr = g.T;
    }
    const int nt = (nr + R - 1) / R;
    int v = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += w;
    }
    const int first = before + v - nt;
    const unsigned hit = __ballot_sync(0xffffffffu, tile >= first && tile < first + nt);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int off = (tile - __shfl_sync(0xffffffffu, first, src)) * R;
      Unit u;
      u.seg = s0 + src;
      u.ct = 0;
      u.row0 = __shfl_sync(0xffffffffu, r0, src) + off;
      u.rows = min(R, __shfl_sync(0xffffffffu, nr, src) - off);
      u.brow0 = X_SHARED && u.seg >= g.n_mat ? g.rows + off : u.row0;
      if (bad) atomicOr(g.status, MOE_DEVFAULT_BAD_TILE);
      unsound = __any_sync(0xffffffffu, bad);
      u.mixed = unsound;
      return u;
    }
    before += __shfl_sync(0xffffffffu, v, 31);
  }
  if (bad) atomicOr(g.status, MOE_DEVFAULT_BAD_TILE);
  unsound = false;
  Unit u = {};
  u.seg = -1;
  return u;
}

// Row r of a unit, channel ch, from its integer sums, unless either is past the end. Whether it was clamped.
template <int PASS, int OUT>
__device__ __forceinline__ bool finish(const Int8Gemm& g, const Unit& u, bool sh, long long ex, int r,
                                       int ch, float sum, float sum2) {
  bool clamped = false;
  if (r < u.rows && ch < g.N) {
    int orow;
    float sx;
    unit_row<PASS>(g, u, r, orow, sx);
    if (orow >= 0) {
      const long long at = (long long)orow * g.N + ch;
      float y = sum * sx * (sh ? g.sh_sw : g.sw)[ex * g.N + ch];
      if (PASS == kInt8SwiGLU) y = swiglu(y, sum2 * sx * (sh ? g.sh_sw2 : g.sw2)[ex * g.N + ch]);
      store_one<OUT, PASS == kInt8Slot>(g.out, at, y);
      clamped = PASS == kInt8Slot && mag_bits(y) >= kInt8F16Clamp;
    }
  }
  return clamped;
}

// The tiles after the grid's last one: where segments are unsound others may share rows, and then there can be
// more tiles than the grid holds. Sums one by one, and apart from the kernel, in which a loop over tiles cost
// every call 1.5 of 43 us (8 tokens, 104 + 1 experts of d 3392, d_ff 704; all tests of this kind 1.0).
template <int PASS, int OUT, int R>
__device__ __noinline__ void tiles_past_grid(const Int8Gemm& g, int tile, int ch0, int lane) {
  constexpr bool GLU = PASS == kInt8SwiGLU;
  bool unsound;
  for (;;) {
    const Unit u = find_tile<PASS, R>(g, ++tile, lane, true, unsound);
    if (u.seg < 0) return;
    const bool sh = u.seg >= g.n_mat;
    const long long ex = sh ? u.seg - g.n_mat : u.seg;
    const int8_t* wa = (sh ? g.sh_qw : g.qw) + ex * g.N * g.K;
    const int8_t* wb = GLU ? (sh ? g.sh_qw2 : g.qw2) + ex * g.N * g.K : wa;
    const int ch1 = min(ch0 + (GLU ? kStreams / 2 : kStreams), g.N);
    for (int r = 0; r < u.rows; ++r)
      for (int ch = ch0; ch < ch1; ++ch) {
        int sum = 0, sum2 = 0;
        for (int k = lane * 4; k < g.K; k += 128) {
          const int a = *reinterpret_cast<const int*>(g.x8 + (long long)(u.brow0 + r) * g.K + k);
          sum = __dp4a(*reinterpret_cast<const int*>(wa + (long long)ch * g.K + k), a, sum);
          if (GLU) sum2 = __dp4a(*reinterpret_cast<const int*>(wb + (long long)ch * g.K + k), a, sum2);
        }
        sum = __reduce_add_sync(0xffffffffu, sum);
        sum2 = __reduce_add_sync(0xffffffffu, sum2);
        if (lane == 0 && finish<PASS, OUT>(g, u, sh, ex, r, ch, (float)sum, (float)sum2))
          atomicOr(g.status, MOE_DEVFAULT_FP16_RANGE);
      }
  }
}

template <int PASS, int OUT, int R>
__global__ void __launch_bounds__(kThreads, R == 8 ? kCtasPerSm8 : kCtasPerSm)
    int8_gemv_kernel(const __grid_constant__ Int8Gemm g, int ctas_per_tile, int tiles) {
  constexpr bool GLU = PASS == kInt8SwiGLU;
  constexpr int CH = GLU ? kStreams / 2 : kStreams;  // channels per warp
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tile = blockIdx.x / ctas_per_tile, cta = blockIdx.x - tile * ctas_per_tile;
  // the last tile's CTAs look at every segment, and take the tiles past the grid where there are any
  const bool last = g.offsets != nullptr && tile == tiles - 1;
  bool unsound;
  const Unit u = find_tile<PASS, R>(g, tile, lane, last, unsound);  // every warp: no barrier
  if (u.seg < 0) return;
  const int ch0 = (cta * (kThreads / 32) + warp) * CH;
  if (ch0 >= g.N) return;
  const bool sh = u.seg >= g.n_mat;
  const long long ex = sh ? u.seg - g.n_mat : u.seg;
  const int8_t* wa = (sh ? g.sh_qw : g.qw) + ex * g.N * g.K;
  const int8_t* wb = GLU ? (sh ? g.sh_qw2 : g.qw2) + ex * g.N * g.K : wa;
  const int8_t* w[kStreams];
#pragma unroll
  for (int c = 0; c < kStreams; ++c) {
    const int ch = min(ch0 + (GLU ? c % CH : c), g.N - 1);  // past the end: the last channel again
    w[c] = (GLU && c >= CH ? wb : wa) + (long long)ch * g.K + lane * 16;
  }
  const int8_t* x[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    x[r] = g.x8 + (long long)(u.brow0 + min(r, u.rows - 1)) * g.K + lane * 16;
  int acc[kStreams][R];
#pragma unroll
  for (int c = 0; c < kStreams; ++c)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[c][r] = 0;
  for (int k0 = 0; k0 < g.K; k0 += 512 * kSteps) {
    int4 v[kSteps][kStreams];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int k = k0 + i * 512;
      if (k + lane * 16 < g.K) {
#pragma unroll
        for (int c = 0; c < kStreams; ++c) v[i][c] = load_once(w[c] + k);
      }
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int k = k0 + i * 512;
      if (k + lane * 16 < g.K) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int4 a = *reinterpret_cast<const int4*>(x[r] + k);
#pragma unroll
          for (int c = 0; c < kStreams; ++c) {
            acc[c][r] = __dp4a(v[i][c].x, a.x, acc[c][r]);
            acc[c][r] = __dp4a(v[i][c].y, a.y, acc[c][r]);
            acc[c][r] = __dp4a(v[i][c].z, a.z, acc[c][r]);
            acc[c][r] = __dp4a(v[i][c].w, a.w, acc[c][r]);
          }
        }
      }
    }
  }
  // lane r * CH + c finishes row r, channel ch0 + c
  float mine = 0.0f, mine2 = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int s = __reduce_add_sync(0xffffffffu, acc[c][r]);
      if (lane == r * CH + c) mine = (float)s;
      if (GLU) {
        const int s2 = __reduce_add_sync(0xffffffffu, acc[GLU ? CH + c : c][r]);
        if (lane == r * CH + c) mine2 = (float)s2;
      }
    }
  const int r = lane / CH, ch = ch0 + lane % CH;
  const bool clamped = r < R && finish<PASS, OUT>(g, u, sh, ex, r, ch, mine, mine2);
  if (PASS == kInt8Slot && clamped) atomicOr(g.status, MOE_DEVFAULT_FP16_RANGE);
  if (last && unsound) tiles_past_grid<PASS, OUT, R>(g, tile, ch0, lane);
}

template <int PASS, int OUT>
cudaError_t launch_out(const Int8Gemm& g, int most_rows, cudaStream_t st) {
  constexpr int kCta = kThreads / 32 * (PASS == kInt8SwiGLU ? kStreams / 2 : kStreams);
  const int gx = (g.N + kCta - 1) / kCta;
  auto go = [&](auto kern, int R) {
    // an upper bound of the row tiles: a segment's rows over R and one ragged tile each, and no more
    // than one tile per row
    const long long tiles =
        min((long long)g.rows, (long long)g.rows / R + g.n_mat) + (long long)g.S * ((g.T + R - 1) / R);
    if (tiles * gx > INT_MAX) return cudaErrorInvalidValue;
    return launch_k(kern, dim3((unsigned)(tiles * gx)), dim3(kThreads), 0, st, g, gx, (int)tiles);
  };
  // rows per tile: no more than any segment has, and no more than twice an even spread's (the rows that
  // a tile does not have are computed all the same)
  const long long want = std::min((long long)most_rows, 2 * ((g.rows + g.n_mat - 1ll) / g.n_mat));
  if (want <= 1) return go(int8_gemv_kernel<PASS, OUT, 1>, 1);
  if (want <= 2) return go(int8_gemv_kernel<PASS, OUT, 2>, 2);
  if (want <= 4) return go(int8_gemv_kernel<PASS, OUT, 4>, 4);
  return go(int8_gemv_kernel<PASS, OUT, 8>, 8);
}

}  // namespace

cudaError_t launch_int8_gemv(Int8Pass pass, const Int8Gemm& g, int most_rows, cudaStream_t st) {
  switch (pass) {
    case kInt8SwiGLU: return launch_out<kInt8SwiGLU, MOE_DTYPE_F32>(g, most_rows, st);
    case kInt8Slot: return launch_out<kInt8Slot, MOE_DTYPE_F16>(g, most_rows, st);
    default: break;
  }
  switch (g.out_dtype) {
    case MOE_DTYPE_F32: return launch_out<kInt8Matrix, MOE_DTYPE_F32>(g, most_rows, st);
    case MOE_DTYPE_BF16: return launch_out<kInt8Matrix, MOE_DTYPE_BF16>(g, most_rows, st);
    default: return launch_out<kInt8Matrix, MOE_DTYPE_F16>(g, most_rows, st);
  }
}

}  // namespace moe
