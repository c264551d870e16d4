// Grouped products of 8-bit integers over row segments, with a scale per row and per output channel.
//
// A CTA computes 64 rows x 64 channels with 4-way integer dot products, exact in 32-bit integers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "int8.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTM = 64, kTN = 64, kTK = 64;  // rows, channels, codes per step
constexpr int kLd = kTK / 4 + 1;             // words per staged row (odd: no bank conflicts)

__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
constexpr uint32_t kF16Clamp = 0x477FF000u;  // 65520.0f: the first value past fp16's range

__device__ __forceinline__ uint16_t f16_sat(float v) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.0f), "f"(v));
  return (uint16_t)r;
}

template <int PASS>
__global__ void __launch_bounds__(kThreads) int8_gemm_kernel(const Int8Gemm g) {
  constexpr bool PAIR = PASS == kInt8SwiGLU;
  __shared__ int xs[kTM][kLd], ws[PAIR ? 2 : 1][kTN][kLd];
  __shared__ int seg_expert, seg_row0, seg_rows;
  griddep_wait();
  // which segment the row tile blockIdx.y belongs to
  if (threadIdx.x == 0) {
    int tile = blockIdx.y, e = 0;
    seg_expert = -1;
    for (; e < g.n_mat + g.S; ++e) {
      int r0 = 0, r1 = g.rows;
      if (e >= g.n_mat) {
        r0 = g.rows + (e - g.n_mat) * g.T;
        r1 = r0 + g.T;
      } else if (g.offsets != nullptr) {
        r0 = g.offsets[e];
        r1 = g.offsets[e + 1];
        if (r0 < 0 || r1 < r0 || r1 > g.rows) {
          atomicOr(g.status, MOE_DEVFAULT_BAD_TILE);
          r1 = r0 = 0;
        }
      }
      const int nt = (r1 - r0 + kTM - 1) / kTM;
      if (tile < nt) {
        seg_expert = e;
        seg_row0 = r0 + tile * kTM;
        seg_rows = min(kTM, r1 - seg_row0);
        break;
      }
      tile -= nt;
    }
  }
  __syncthreads();
  if (seg_expert < 0) return;
  const bool sh = seg_expert >= g.n_mat;
  const long long ex = sh ? seg_expert - g.n_mat : seg_expert;
  const int n0 = blockIdx.x * kTN;
  const int8_t* w1 = (sh ? g.sh_qw : g.qw) + ex * g.N * g.K;
  const int8_t* w2 = PAIR ? (sh ? g.sh_qw2 : g.qw2) + ex * g.N * g.K : nullptr;
  // this thread stages 16 codes of one row per step: row threadIdx.x / 4, piece threadIdx.x % 4
  const int lr = threadIdx.x >> 2, lc = threadIdx.x & 3;
  long long xrow = -1;
  if (lr < seg_rows) {
    xrow = seg_row0 + lr;
    if (PASS == kInt8SwiGLU) {
      if (sh) {
        xrow = (xrow - g.rows) % g.T;
      } else {
        const int slot = g.perm_slot[xrow];
        if (slot < 0 || slot >= g.rows) {
          atomicOr(g.status, MOE_DEVFAULT_BAD_TILE);
          xrow = -1;
        } else {
          xrow = slot / g.k;
        }
      }
    }
  }
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[PAIR ? 2 : 1][4][4] = {};
  for (int k0 = 0; k0 < g.K; k0 += kTK) {
    const int kk = k0 + lc * 16;
    int4 v = make_int4(0, 0, 0, 0), u = v, u2 = v;
    if (kk < g.K) {
      if (xrow >= 0) v = *reinterpret_cast<const int4*>(g.qx + xrow * g.K + kk);
      if (n0 + lr < g.N) {
        u = *reinterpret_cast<const int4*>(w1 + (long long)(n0 + lr) * g.K + kk);
        if (PAIR) u2 = *reinterpret_cast<const int4*>(w2 + (long long)(n0 + lr) * g.K + kk);
      }
    }
    __syncthreads();
    const int c = lc * 4;
    xs[lr][c] = v.x, xs[lr][c + 1] = v.y, xs[lr][c + 2] = v.z, xs[lr][c + 3] = v.w;
    ws[0][lr][c] = u.x, ws[0][lr][c + 1] = u.y, ws[0][lr][c + 2] = u.z, ws[0][lr][c + 3] = u.w;
    if (PAIR) {
      int(*w)[kLd] = ws[PAIR ? 1 : 0];
      w[lr][c] = u2.x, w[lr][c + 1] = u2.y, w[lr][c + 2] = u2.z, w[lr][c + 3] = u2.w;
    }
    __syncthreads();
#pragma unroll 4
    for (int kw = 0; kw < kTK / 4; ++kw) {
      int av[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) av[i] = xs[ty + 16 * i][kw];
#pragma unroll
      for (int m = 0; m < (PAIR ? 2 : 1); ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int bv = ws[m][tx + 16 * j][kw];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][i][j] = __dp4a(av[i], bv, acc[m][i][j]);
        }
    }
  }
  uint32_t mx = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i;
    if (r >= seg_rows) continue;
    const long long p = seg_row0 + r;
    long long orow = p, srow = p;
    float gate = 1.0f;
    if (PASS != kInt8Matrix) {
      if (sh) {
        srow = PASS == kInt8SwiGLU ? (p - g.rows) % g.T : p;
      } else {
        const int slot = g.perm_slot[p];
        if (slot < 0 || slot >= g.rows) continue;
        if (PASS == kInt8SwiGLU) srow = slot / g.k;
        if (PASS == kInt8Slot) {
          orow = slot;
          if (g.topk_w != nullptr) gate = g.topk_w[slot];
        }
      }
    }
    const float sx = g.sx[srow];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 16 * j;
      if (n >= g.N) continue;
      float v = (float)acc[0][i][j] * (sx * (sh ? g.sh_sw : g.sw)[ex * g.N + n]);
      const long long at = orow * g.N + n;
      if (PASS == kInt8Matrix) {
        if (g.out_dtype == MOE_DTYPE_F32)
          static_cast<float*>(g.out)[at] = v;
        else if (g.out_dtype == MOE_DTYPE_BF16)
          static_cast<__nv_bfloat16*>(g.out)[at] = __float2bfloat16(v);
        else
          static_cast<__half*>(g.out)[at] = __float2half(v);
        continue;
      }
      if (PASS == kInt8SwiGLU) {
        const float up =
            (float)acc[PAIR ? 1 : 0][i][j] * (sx * (sh ? g.sh_sw2 : g.sw2)[ex * g.N + n]);
        static_cast<float*>(g.out)[at] = v / (1.0f + __expf(-v)) * up;
        continue;
      }
      v *= gate;
      mx = max(mx, mag_bits(v));
      static_cast<uint16_t*>(g.out)[at] = f16_sat(v);
    }
  }
  if (PASS == kInt8Slot && mx >= kF16Clamp) atomicOr(g.status, MOE_DEVFAULT_FP16_RANGE);
}

}  // namespace

cudaError_t launch_int8_gemm(Int8Pass pass, const Int8Gemm& g, cudaStream_t st) {
  const long long tiles =
      g.rows / kTM + g.n_mat + (long long)g.S * ((g.T + kTM - 1) / kTM);  // an upper bound
  if (tiles > 65535) return cudaErrorInvalidValue;
  const dim3 grid((g.N + kTN - 1) / kTN, (unsigned)tiles), block(kThreads);
  switch (pass) {
    case kInt8Matrix: return launch_k(int8_gemm_kernel<kInt8Matrix>, grid, block, 0, st, g);
    case kInt8SwiGLU: return launch_k(int8_gemm_kernel<kInt8SwiGLU>, grid, block, 0, st, g);
    default: return launch_k(int8_gemm_kernel<kInt8Slot>, grid, block, 0, st, g);
  }
}

}  // namespace moe
