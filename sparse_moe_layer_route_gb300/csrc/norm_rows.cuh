// Rows of a matrix in a kernel that works on whole rows (norms around a block, dropout): element access, the
// generator, and sums over a row.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cooperative_groups.h>

#include "norm.cuh"
#include "ptx.cuh"

namespace moe {

// -------------------------------------------------------------------------------------- elements
// Types of elements. Kernels for rows that start on 16 bytes know theirs; Any looks at the argument.
struct F32 {};
struct BF16 {};
struct F16 {};
struct Any {};

template <class E>
__host__ __device__ __forceinline__ int bytes_of(int dtype) {
  if constexpr (std::is_same_v<E, Any>) return dtype == MOE_DTYPE_F32 ? 4 : 2;
  return std::is_same_v<E, F32> ? 4 : 2;
}

// Two floats as the instructions on pairs take them: one issue for two results.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pair(float a, float b) {
  F2 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ F2 twice(float a) { return pair(a, a); }
__device__ __forceinline__ float2 both(F2 v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}
// A thread's chunk of eight channels.
using Chunk = F2[4];
// f(i, value) for the eight channels of a chunk, whose value becomes what f returns.
template <class F>
__device__ __forceinline__ void each(F2 (&v)[4], F f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = both(v[i]);
    v[i] = pair(f(2 * i, x.x), f(2 * i + 1, x.y));
  }
}

// Eight elements as they lie in memory: 16-bit ones in a, 32-bit ones in a and b.
struct Raw {
  uint4 a, b;
};
__device__ __forceinline__ void f32_to(const Raw& r, F2 (&v)[4]) {
  v[0] = pair(__uint_as_float(r.a.x), __uint_as_float(r.a.y));
  v[1] = pair(__uint_as_float(r.a.z), __uint_as_float(r.a.w));
  v[2] = pair(__uint_as_float(r.b.x), __uint_as_float(r.b.y));
  v[3] = pair(__uint_as_float(r.b.z), __uint_as_float(r.b.w));
}
__device__ __forceinline__ void bf16_to(const Raw& r, F2 (&v)[4]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void f16_to(const Raw& r, F2 (&v)[4]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[i] = pair(f.x, f.y);
  }
}
template <class E>
__device__ __forceinline__ void to_float(const Raw& r, int dtype, F2 (&v)[4]) {
  if constexpr (std::is_same_v<E, F32>) {
    f32_to(r, v);
  } else if constexpr (std::is_same_v<E, BF16>) {
    bf16_to(r, v);
  } else if constexpr (std::is_same_v<E, F16>) {
    f16_to(r, v);
  } else {
    if (dtype == MOE_DTYPE_F32)
      f32_to(r, v);
    else if (dtype == MOE_DTYPE_BF16)
      bf16_to(r, v);
    else
      f16_to(r, v);
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t bf16_pair(F2 v) {
  const float2 f = both(v);
  return bf16_pair(f.x, f.y);
}
__device__ __forceinline__ uint32_t f16_pair(F2 v) {
  const float2 f = both(v);
  return f16_pair(f.x, f.y);
}

__device__ __forceinline__ uint4 shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// --------------------------------------------------------------------------------------- copies in
// A thread has chunks of eight channels, a warp 256 channels in a row. Rows come through shared memory of the
// warp's own, copied asynchronously while the rows before are worked on; no other warp reads them, so there is
// no barrier but the warp's. Where rows start on 16 bytes a lane copies and stores its own chunk, else the
// warp moves its 256 elements one per lane at a time.
constexpr int kWarpCols = 256;

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Until the oldest of `stages` groups of copies is there.
__device__ __forceinline__ void copies_wait_stage(int stages) {
  if (stages == 4)
    copies_wait<3>();
  else if (stages == 3)
    copies_wait<2>();
  else if (stages == 2)
    copies_wait<1>();
  else
    copies_wait<0>();
}

// One input of a warp and its place in shared memory, [chunk][256] at `at` (a stage's; this warp's). What a
// lane needs is worked out where it is used: the arguments stay where the launch put them, and few registers
// are held from row to row. E Any: for any alignment.
template <class E, int R, int NC>
struct Input {
  static constexpr int kBytes = std::is_same_v<E, F32> ? 4 : 2;  // but for Any
  static __host__ __device__ int bytes(int dtype) { return NC * kWarpCols * bytes_of<E>(dtype); }

  // Starts the copies of a row. Chunks past d: whole ones stay as clear() left them, elements become 0.
  static __device__ __forceinline__ void fetch(const RowsIn& m, int row, int w0, int lane, int d, uint32_t at) {
    const char* from = static_cast<const char*>(m.p) + (size_t)(uint32_t)row * (m.ld * bytes_of<E>(m.dtype));
    if constexpr (!std::is_same_v<E, Any>) {
      from += (w0 + lane * 8) * kBytes;
      at += lane * 8 * kBytes;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (w0 + c * R * 8 + lane * 8 < d) {
          copy16(at + c * kWarpCols * kBytes, from + c * R * 8 * kBytes);
          if constexpr (kBytes == 4) copy16(at + c * kWarpCols * 4 + 16, from + c * R * 32 + 16);
        }
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int left = d - (w0 + c * R * 8 + lane);  // this lane's elements are 32 apart
        if (w0 + c * R * 8 >= d) continue;
        if (m.dtype == MOE_DTYPE_F32) {
          const char* q = from + (w0 + c * R * 8 + lane) * 4ll;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const bool there = i * 32 < left;
            copy4(at + (c * kWarpCols + i * 32 + lane) * 4, there ? q + i * 128 : from, there ? 4 : 0);
          }
        } else {  // two bytes cannot be copied asynchronously
          uint16_t v[8];
          const uint16_t* q = reinterpret_cast<const uint16_t*>(from) + (w0 + c * R * 8 + lane);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = i * 32 < left ? q[i * 32] : (uint16_t)0;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + (c * kWarpCols + i * 32 + lane) * 2),
                         "h"(v[i])
                         : "memory");
        }
      }
    }
  }
  // Chunks past d are 0 from the start.
  static __device__ __forceinline__ void clear(const RowsIn& m, int w0, int lane, int d, uint32_t at) {
    const int b = bytes_of<E>(m.dtype);
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (w0 + c * R * 8 + (std::is_same_v<E, Any> ? 0 : lane * 8) >= d)
        for (int k = 0; k < b / 2; ++k)
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                           at + (c * kWarpCols + lane * 8) * b + 16 * k),
                       "r"(0)
                       : "memory");
  }
  // This lane's chunk c.
  static __device__ __forceinline__ void read(const RowsIn& m, int c, int lane, uint32_t at, F2 (&v)[4]) {
    Raw r;
    const int b = bytes_of<E>(m.dtype);
    const uint32_t from = at + (c * kWarpCols + lane * 8) * b;
    r.a = shared16(from);
    if (b == 4) r.b = shared16(from + 16);
    to_float<E>(r, m.dtype, v);
  }
};

// Warps of a row of d channels whose first chunk lies in it; the others have nothing to do (not of a cluster's rows:
// all its threads meet).
template <int R, bool CLUSTER>
__host__ __device__ __forceinline__ int live_warps(int d) {
  const int all = R / 32, wanted = (d + kWarpCols - 1) / kWarpCols;
  return CLUSTER || wanted > all ? all : wanted;
}

// -------------------------------------------------------------------------------------- parameters
// A thread's chunk of a row of parameters as it lies in memory, from channel c on, 0 past the d-th. They are
// small and stay in L1 from row to row. ANY: of any alignment.
template <bool ANY>
__device__ __forceinline__ Raw param_raw(const RowsIn& m, long long row, int c, int d) {
  Raw r = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (c >= d) return r;
  const bool f32 = m.dtype == MOE_DTYPE_F32;
  const long long at = row * m.ld + c;
  if (!ANY || (m.wide && c + 8 <= d)) {
    if (f32) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(m.p) + at);
      r.a = __ldg(p);
      r.b = __ldg(p + 1);
    } else {
      r.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(m.p) + at));
    }
    return r;
  }
  uint32_t v[8];
  if (f32) {
    const uint32_t* p = static_cast<const uint32_t*>(m.p) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < d ? __ldg(p + i) : 0u;
    r.a = make_uint4(v[0], v[1], v[2], v[3]);
    r.b = make_uint4(v[4], v[5], v[6], v[7]);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(m.p) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < d ? __ldg(p + i) : 0u;
    r.a = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
  return r;
}
// op(c, w) for every chunk c of a thread and its parameters w; all chunks' are under way before the first is used.
template <bool ANY, int NC, class Op>
__device__ __forceinline__ void with_params(const RowsIn& m, long long row, const int (&col)[NC], int d,
                                            Op op) {
  if (ANY || m.dtype == MOE_DTYPE_F32) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const Raw r = param_raw<ANY>(m, row, col[c], d);
      F2 w[4];
      to_float<Any>(r, m.dtype, w);
      op(c, w);
    }
    return;
  }
  const uint16_t* p = static_cast<const uint16_t*>(m.p) + row * m.ld;
  Raw r[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c)
    r[c].a = col[c] < d ? __ldg(reinterpret_cast<const uint4*>(p + col[c])) : make_uint4(0u, 0u, 0u, 0u);
  if (m.dtype == MOE_DTYPE_BF16) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      F2 w[4];
      bf16_to(r[c], w);
      op(c, w);
    }
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      F2 w[4];
      f16_to(r[c], w);
      op(c, w);
    }
  }
}

// x times the parameters, chunk by chunk.
template <bool ANY, int NC>
__device__ __forceinline__ void times_params(const RowsIn& m, long long row, const int (&col)[NC], int d,
                                             F2 (&x)[NC][4]) {
  with_params<ANY>(m, row, col, d, [&](int c, const F2 (&w)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[c][i] = mul2(x[c][i], w[i]);
  });
}

// (x - mean) * scale; centred: there is a mean.
template <int NC>
__device__ __forceinline__ void scale_rows(F2 (&x)[NC][4], bool centred, float mean, float scale) {
  const F2 m = twice(-mean), s = twice(scale);
  if (centred) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[c][i] = add2(x[c][i], m);
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) x[c][i] = mul2(x[c][i], s);
}

// ------------------------------------------------------------------------------------------ stores
// Past L1, where the parameters stay (16384 x 7168 forward: 172 -> 150 us).
__device__ __forceinline__ void store16(void* to, uint4 v) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(to), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
// Eight elements that start on 16 bytes. Of 32-bit ones two 16-byte stores past L1 would each write half sectors (8192
// x 4096 backward: 175 us instead of 171), so only one of 32 bytes goes there.
template <class E>
__device__ __forceinline__ void store_chunk(void* to, const F2 (&v)[4]) {
  if constexpr (std::is_same_v<E, F32>) {
    const float2 a = both(v[0]), b = both(v[1]), c = both(v[2]), d = both(v[3]);
    if (reinterpret_cast<uintptr_t>(to) % 32 == 0) {
      asm volatile("st.global.L1::no_allocate.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(a.x),
                   "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y)
                   : "memory");
    } else {
      static_cast<float4*>(to)[0] = make_float4(a.x, a.y, b.x, b.y);
      static_cast<float4*>(to)[1] = make_float4(c.x, c.y, d.x, d.y);
    }
  } else if constexpr (std::is_same_v<E, BF16>) {
    store16(to, make_uint4(bf16_pair(v[0]), bf16_pair(v[1]), bf16_pair(v[2]), bf16_pair(v[3])));
  } else {
    store16(to, make_uint4(f16_pair(v[0]), f16_pair(v[1]), f16_pair(v[2]), f16_pair(v[3])));
  }
}
// This lane's chunk c of a row. Any: `turn` (1 KB of the warp's shared memory) turns chunks round, as they
// cannot be stored as they are.
template <class E, int R>
__device__ __forceinline__ void store(const RowsOut& m, int row, int c, int w0, int lane, int d,
                                      const F2 (&v)[4], float* turn) {
  char* to = static_cast<char*>(m.p) + (size_t)(uint32_t)row * (m.ld * bytes_of<E>(m.dtype));
  const int w = w0 + c * R * 8;
  if constexpr (!std::is_same_v<E, Any>) {
    constexpr int b = std::is_same_v<E, F32> ? 4 : 2;
    if (w + lane * 8 < d) store_chunk<E>(to + (w0 + lane * 8) * b + c * R * 8 * b, v);
  } else {
    if (w >= d) return;
    F2* t = reinterpret_cast<F2*>(turn + lane * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = v[i];
    __syncwarp();
    const int left = d - w - lane;
    if (m.dtype == MOE_DTYPE_F32) {
      float* q = reinterpret_cast<float*>(to) + w + lane;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i * 32 < left) q[i * 32] = turn[i * 32 + lane];
    } else {
      uint16_t* q = reinterpret_cast<uint16_t*>(to) + w + lane;
      const bool bf16 = m.dtype == MOE_DTYPE_BF16;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f = turn[i * 32 + lane];
        if (i * 32 < left) q[i * 32] = (uint16_t)(bf16 ? bf16_pair(f, 0.f) : f16_pair(f, 0.f));
      }
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------------------- dropout
// Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC'11):
// each round multiplies two words of the counter by constants, and mixes high halves, the other two
// words and the key, which moves on by a constant. Seed and step in the form the rounds take them:
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
// The random numbers of eight elements of a row from channel c (a multiple of 8) on. Two counters at a time:
// they share the key.
__device__ __forceinline__ void philox8(const DropState& s, uint32_t row, uint32_t c, uint32_t (&r)[2][4]) {
  uint32_t k0 = s.k0, k1 = s.k1;
#pragma unroll
  for (int h = 0; h < 2; ++h) r[h][0] = (c >> 2) + h, r[h][1] = row, r[h][2] = s.s0, r[h][3] = s.s1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint64_t a = (uint64_t)0xD2511F53u * r[h][0], b = (uint64_t)0xCD9E8D57u * r[h][2];
      r[h][0] = (uint32_t)(b >> 32) ^ r[h][1] ^ k0;
      r[h][1] = (uint32_t)b;
      r[h][2] = (uint32_t)(a >> 32) ^ r[h][3] ^ k1;
      r[h][3] = (uint32_t)a;
    }
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}
// Eight elements of a row from channel c on, each times the scale or, dropped, 0 whatever it was.
__device__ __forceinline__ void drop8(const Drop& d, const DropState& s, uint32_t row, uint32_t c,
                                      F2 (&v)[4]) {
  uint32_t r[2][4];
  philox8(s, row, c, r);
  each(v, [&](int i, float x) { return r[i >> 2][i & 3] >= d.least ? x * d.scale : 0.f; });
}

// ----------------------------------------------------------------------------------- sums of a row
// A row is shared by R threads of one CTA, or by all threads of the cl CTAs of a cluster. Sums go over lanes,
// warps and CTAs in a fixed order. Of several sums a warp's halves (quarters) first take one each, so that four
// cost six shuffles, not twenty.
template <int R, bool CLUSTER>
struct RowSum {
  static constexpr int kW = (R / 32 + 3) / 4 * 4, kMost = CLUSTER ? 8 : 0;  // warps, read four at a time
  static constexpr int kBuf = 4 * (kW + kMost);  // of four sums: [sum][warp], then [CTA][sum]
  static constexpr int kFloats = 2 * kBuf;
  float* buf;                                    // 16-byte aligned
  int group, cl, turn, threads;

  // live: warps that take part, the first ones; the others' places are 0 from before the first barrier on.
  __device__ RowSum(float* b, int g, int n, int live) : buf(b), group(g), cl(n), turn(0), threads(32 * live) {
    const int tid = threadIdx.x % R;
    if constexpr (CLUSTER) {
      static_assert(R / 32 == kW, "no place to clear");
      cooperative_groups::this_cluster().barrier_arrive();
    } else if (R > 32 && tid < 8) {
      for (int w = live; w < kW; ++w) buf[tid / 4 * kBuf + tid % 4 * kW + w] = 0.f;
    }
  }

  // By all threads, once, before the first sum: a CTA may write to another's shared memory only when that has started.
  // Between this and the arrival above are the first rows' copies, so nothing waits long here.
  __device__ __forceinline__ void all_started() const {
    if constexpr (CLUSTER) {
      __syncwarp();
      cooperative_groups::this_cluster().barrier_wait();
    }
  }

  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    static_assert(N == 1 || N == 2 || N == 4, "one, two or four at a time");
    const int lane = threadIdx.x % 32;
    float s = v[0];
    if constexpr (N == 4) {
      const bool up = lane & 16;
      const float a = __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16) + (up ? v[2] : v[0]);
      const float b = __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16) + (up ? v[3] : v[1]);
      const bool odd = lane & 8;
      s = __shfl_xor_sync(0xffffffffu, odd ? a : b, 8) + (odd ? b : a);
    } else if constexpr (N == 2) {
      const bool up = lane & 16;
      s = __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16) + (up ? v[1] : v[0]);
    }
#pragma unroll
    for (int o = 16 / N; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    // lanes n * 32 / N and on have sum n
    if constexpr (R == 32) {
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] = N == 1 ? s : __shfl_sync(0xffffffffu, s, n * (32 / N));
    } else {
      const int warp = threadIdx.x % R / 32;
      // two buffers in turn: between two uses of one there is the other's barrier
      float* b = buf + turn * kBuf;
      turn ^= 1;
      if (lane % (32 / N) == 0) b[lane / (32 / N) * kW + warp] = s;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float part[kW / 4];
#pragma unroll
        for (int w = 0; w < kW / 4; ++w) {
          const float4 q = *reinterpret_cast<const float4*>(b + n * kW + 4 * w);
          part[w] = (q.x + q.y) + (q.z + q.w);
        }
#pragma unroll
        for (int w = 1; w < kW / 4; ++w) part[0] += part[w];
        v[n] = part[0];
      }
      if constexpr (CLUSTER) {
        namespace cg = cooperative_groups;
        cg::cluster_group cluster = cg::this_cluster();
        if (threadIdx.x < cl) {
          float* there = cluster.map_shared_rank(b + kW * 4, threadIdx.x);
#pragma unroll
          for (int n = 0; n < N; ++n) there[cluster.block_rank() * 4 + n] = v[n];
        }
        cluster.sync();
#pragma unroll
        for (int n = 0; n < N; ++n) {
          v[n] = 0.f;
          for (int i = 0; i < cl; ++i) v[n] += b[kW * 4 + i * 4 + n];
        }
      }
    }
  }
};

__device__ __forceinline__ float total(F2 a, F2 b, F2 c, F2 d) {
  const float2 f = both(add2(add2(a, b), add2(c, d)));
  return f.x + f.y;
}
// A thread's share of sum(x y).
template <int NC>
__device__ __forceinline__ float dot(const F2 (&x)[NC][4], const F2 (&y)[NC][4]) {
  F2 s[4] = {0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = fma2(x[c][i], y[c][i], s[i]);
  return total(s[0], s[1], s[2], s[3]);
}
template <int NC>
__device__ __forceinline__ float plain_sum(const F2 (&x)[NC][4]) {
  F2 s[4] = {0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = add2(x[c][i], s[i]);
  return total(s[0], s[1], s[2], s[3]);
}
// A thread's share of sum((x - mean)^2) over channels before d; EDGE: a chunk may lie across the end.
template <int NC, bool EDGE>
__device__ __forceinline__ float around(const F2 (&x)[NC][4], float mean, const int (&col)[NC], int d) {
  const F2 m = twice(-mean);
  F2 s[4] = {0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < NC; ++c)
    if (col[c] < d) {
      F2 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = add2(x[c][i], m);
      if constexpr (EDGE) each(v, [&](int i, float y) { return col[c] + i < d ? y : 0.f; });
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = fma2(v[i], v[i], s[i]);
    }
  return total(s[0], s[1], s[2], s[3]);
}
// One over the deviation from its squares' sum, within two units in the last place.
__device__ __forceinline__ float deviation(float squares, float inv, float eps) {
  return rsqrtf(fmaf(squares, inv, eps));
}

// Mean (0 for rms) and one over the deviation of a row (inv: one over its channels) whose threads hold x; what
// is past the channels that end at d is 0 in x and does not count.
template <int NC, bool EDGE, typename Sum>
__device__ __forceinline__ void row_stats(Sum& sum, int kind, const F2 (&x)[NC][4], const int (&col)[NC],
                                          int d, float inv, float eps, float& mean, float& rstd) {
  mean = 0.f;
  float q[1];
  if (kind == MOE_NORM_LAYER) {
    q[0] = plain_sum<NC>(x);
    sum(q);
    mean = q[0] * inv;
    q[0] = around<NC, EDGE>(x, mean, col, d);
  } else {
    q[0] = dot<NC>(x, x);
  }
  sum(q);
  rstd = deviation(q[0], inv, eps);
}

// How a row is shared: R threads with NC chunks of eight channels each, above 8192 channels a cluster.
template <int R>
__host__ __device__ constexpr int norm_threads() {
  return R < 256 ? 256 : R;
}

// Launches a kernel of rows: programmatic stream serialization (it waits before it touches memory), and a
// cluster of cl CTAs where it wants one.
template <bool CLUSTER, typename... K, typename... A>
cudaError_t launch_rows(void (*kernel)(K...), int grid, int threads, int smem, int cl, cudaStream_t st,
                        A&&... args) {
  if (smem > 46 * 1024) {  // a kernel has up to 2 KB of its own besides
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem - 1024);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cl;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace moe
