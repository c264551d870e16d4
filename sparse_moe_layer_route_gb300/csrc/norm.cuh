// Norms around a block, residual, gates and dropout (norm.cu, norm_grad.cu): arguments, element access, the
// generator and sums over a row.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cooperative_groups.h>

#include "internal.h"
#include "ptx.cuh"

namespace moe {

constexpr int kNormMaxSize = 65536;  // d: eight CTAs of a cluster with 8192 channels each
constexpr int kNormMaxCtas = 320;    // of the gradient, each with partial sums in the workspace

// Rows of a matrix: element type, elements between rows, and whether every row starts on 16 bytes.
struct RowsIn {
  const void* p;
  long long ld;
  int dtype;
  bool wide;
};
struct RowsOut {
  void* p;
  long long ld;
  int dtype;
  bool wide;
};

struct Drop {
  const long long* rng;  // seed, step; nullptr: nothing is dropped
  uint32_t least;        // numbers from this one on keep their element
  float scale;
};

struct NormArgs {
  RowsIn h, y;           // y.p nullptr: no block, h' = alpha h
  RowsIn w_after, b_after, gate, w_before, b_before;
  RowsOut h_out, n;
  Drop drop;
  int T, d, after, before, gate_rows;
  float eps, alpha, beta;
};

struct NormGradArgs {
  RowsIn h, y, d_h_out, d_n;  // h: the stream after the block
  RowsIn w_after, b_after, gate, w_before;
  RowsOut d_h, d_y;
  float *d_w_after, *d_b_after, *d_gate, *d_w_before, *d_b_before;
  float* part;                // [CTAs][kNormParts][d]
  Drop drop;
  int T, d, after, before, gate_rows;
  float eps, alpha, beta;
};
// Partial sums of a CTA: gradients of w_after, b_after, w_before, b_before, and of the gates that it shares
// with the CTA before it and the one after it.
constexpr int kNormParts = 6;

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_grad(const NormGradArgs& a, cudaStream_t st);

struct DropoutArgs {
  RowsIn x, residual;  // residual.p nullptr: none
  RowsOut y;
  Drop drop;
  int T, d;
};
cudaError_t launch_dropout(const DropoutArgs& a, cudaStream_t st);

#ifdef __CUDACC__

// ---------------------------------------------------------------------------------- element access
__device__ __forceinline__ float from16(uint32_t bits, int dtype) {
  return dtype == MOE_DTYPE_BF16 ? __uint_as_float(bits << 16)
                                 : __half2float(__ushort_as_half((unsigned short)bits));
}
__device__ __forceinline__ uint32_t pack16(float a, float b, int dtype) {
  if (dtype == MOE_DTYPE_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight elements from channel c on; those past the d-th are 0.
__device__ __forceinline__ void load8(const RowsIn& m, long long row, int c, int d, float (&v)[8]) {
  const long long at = row * m.ld + c;
  if (m.wide && c + 8 <= d) {
    if (m.dtype == MOE_DTYPE_F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(m.p) + at);
      const float4 a = p[0], b = p[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(m.p) + at);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
      if (m.dtype == MOE_DTYPE_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          v[2 * i] = f.x;
          v[2 * i + 1] = f.y;
        }
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = 0.f;
    if (c + i < d)
      v[i] = m.dtype == MOE_DTYPE_F32 ? static_cast<const float*>(m.p)[at + i]
                                      : from16(static_cast<const uint16_t*>(m.p)[at + i], m.dtype);
  }
}

__device__ __forceinline__ void store8(const RowsOut& m, long long row, int c, int d,
                                       const float (&v)[8]) {
  const long long at = row * m.ld + c;
  if (m.wide && c + 8 <= d) {
    if (m.dtype == MOE_DTYPE_F32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(m.p) + at);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(m.p) + at) =
          make_uint4(pack16(v[0], v[1], m.dtype), pack16(v[2], v[3], m.dtype),
                     pack16(v[4], v[5], m.dtype), pack16(v[6], v[7], m.dtype));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < d) {
      if (m.dtype == MOE_DTYPE_F32)
        static_cast<float*>(m.p)[at + i] = v[i];
      else
        static_cast<uint16_t*>(m.p)[at + i] = (uint16_t)pack16(v[i], 0.f, m.dtype);
    }
}

// ---------------------------------------------------------------------------------------- dropout
// Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC'11):
// each round multiplies two words of the counter by constants, and mixes high halves, the other two
// words and the key, which moves on by a constant.
__device__ __forceinline__ void philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                       uint32_t k1, uint32_t (&r)[4]) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  r[0] = c0, r[1] = c1, r[2] = c2, r[3] = c3;
}

// Seed and step in the form the rounds take them.
struct DropState {
  uint32_t k0, k1, s0, s1;
  __device__ explicit DropState(const Drop& d) : k0(0), k1(0), s0(0), s1(0) {
    if (d.rng != nullptr) {
      const unsigned long long seed = d.rng[0], step = d.rng[1];
      k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
      s0 = (uint32_t)step, s1 = (uint32_t)(step >> 32);
    }
  }
};
// Factors of eight elements of a row from channel c (a multiple of 8) on: 0, or the scale of kept ones.
__device__ __forceinline__ void drop8(const Drop& d, const DropState& s, uint32_t row, uint32_t c,
                                      float (&m)[8]) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t r[4];
    philox((c >> 2) + half, row, s.s0, s.s1, s.k0, s.k1, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) m[4 * half + i] = r[i] >= d.least ? d.scale : 0.f;
  }
}

// ----------------------------------------------------------------------------------- sums of a row
// A row is shared by R threads of one CTA, or by all of the CL CTAs of a cluster (then R is the CTA).
// Sums go over lanes, warps and CTAs in a fixed order.
template <int R, int CL>
struct RowSum {
  static constexpr int kW = R / 32;
  float* buf;  // [2][kW + CL][2] floats of this row's threads
  int group, turn;

  __device__ RowSum(float* b, int g) : buf(b), group(g), turn(0) {}

  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    static_assert(N <= 2, "two at a time");
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    if constexpr (R > 32) {
      const int warp = threadIdx.x % R / 32, lane = threadIdx.x % 32;
      // two buffers in turn: between two uses of one there is the other's barrier
      float* b = buf + turn * (kW + CL) * 2;
      turn ^= 1;
      if (lane == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) b[warp * 2 + n] = v[n];
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(R) : "memory");
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] = lane < kW ? b[lane * 2 + n] : 0.f;
#pragma unroll
      for (int o = kW / 2; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] = __shfl_sync(0xffffffffu, v[n], 0);
      if constexpr (CL > 1) {
        namespace cg = cooperative_groups;
        cg::cluster_group cluster = cg::this_cluster();
        if (threadIdx.x < CL) {
          float* there = cluster.map_shared_rank(b + kW * 2, threadIdx.x);
#pragma unroll
          for (int n = 0; n < N; ++n) there[cluster.block_rank() * 2 + n] = v[n];
        }
        cluster.sync();
#pragma unroll
        for (int n = 0; n < N; ++n) {
          v[n] = 0.f;
          for (int i = 0; i < CL; ++i) v[n] += b[(kW + i) * 2 + n];
        }
      }
    }
  }
};

// Mean (0 for rms) and one over the deviation of a row whose threads hold x; what is past its end does not
// count.
template <int NC, typename Sum>
__device__ __forceinline__ void row_stats(Sum& sum, int kind, const float (&x)[NC][8], const int (&col)[NC],
                                          int d, float eps, float& mean, float& rstd) {
  const float inv = 1.f / (float)d;
  mean = 0.f;
  if (kind == MOE_NORM_LAYER) {
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += col[c] + i < d ? x[c][i] : 0.f;
    sum(s);
    mean = s[0] * inv;
  }
  float q[1] = {0.f};
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = col[c] + i < d ? x[c][i] - mean : 0.f;
      q[0] = fmaf(v, v, q[0]);
    }
  sum(q);
  rstd = 1.f / sqrtf(fmaf(q[0], inv, eps));
}

#endif  // __CUDACC__

// Calls F<R, NC, CL>(arguments) for the narrowest form that holds a row of d channels.
#define MOE_NORM_FORMS(F, d, ...)                                   \
  ((d) <= 256     ? F<32, 1, 1>(__VA_ARGS__)                        \
   : (d) <= 512   ? F<32, 2, 1>(__VA_ARGS__)                        \
   : (d) <= 1024  ? F<128, 1, 1>(__VA_ARGS__)                       \
   : (d) <= 2048  ? F<128, 2, 1>(__VA_ARGS__)                       \
   : (d) <= 4096  ? F<256, 2, 1>(__VA_ARGS__)                       \
   : (d) <= 8192  ? F<512, 2, 1>(__VA_ARGS__)                       \
   : (d) <= 16384 ? F<512, 2, 2>(__VA_ARGS__)                       \
   : (d) <= 32768 ? F<512, 2, 4>(__VA_ARGS__) : F<512, 2, 8>(__VA_ARGS__))

}  // namespace moe
