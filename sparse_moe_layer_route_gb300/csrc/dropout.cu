// Dropout by itself: y = residual + drop(x). Bound by its bytes; the generator's 40 multiplications for eight
// elements are about as much work (norm_rows.cuh). Measured: 16384 x 7168 onto a residual, bf16: 119 us (705 MB,
// 5.9 TB/s); 1000 x 1027 in fp32, rows 1032 apart: 6 us, the call's.
#include "norm_rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Eight elements that nobody reads again.
template <class E>
__device__ __forceinline__ Raw stream8(const void* p) {
  Raw r;
  auto load = [](const void* q) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(q)
                 : "memory");
    return v;
  };
  r.a = load(p);
  if constexpr (std::is_same_v<E, F32>) r.b = load(static_cast<const char*>(p) + 16);
  return r;
}

// Rows that start on 16 bytes: chunks of eight channels are numbered through, and a thread takes every
// `threads`-th; hop is that many as rows and chunks, so that none needs a division but the first.
template <class E>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropoutArgs a, int chunks,
                                                           int hop_rows, int hop_chunks) {
  constexpr int b = std::is_same_v<E, F32> ? 4 : 2;
  const long long first = (long long)blockIdx.x * kThreads + threadIdx.x;
  long long row = first / chunks;
  int k = (int)(first - row * chunks);
  griddep_wait();
  const DropState ds(a.drop);
  while (row < a.T) {
    const long long c = (long long)k * 8;
    const Raw x = stream8<E>(static_cast<const char*>(a.x.p) + (row * a.x.ld + c) * b);
    Raw r;
    if (a.residual.p != nullptr)
      r = stream8<E>(static_cast<const char*>(a.residual.p) + (row * a.residual.ld + c) * b);
    F2 v[4], s[4];
    if (a.drop.rng != nullptr) {
      uint32_t n[2][4];
      philox8(ds, (uint32_t)row, (uint32_t)c, n);  // while x is on its way
      to_float<E>(x, 0, v);
      each(v, [&](int i, float t) { return n[i >> 2][i & 3] >= a.drop.least ? t * a.drop.scale : 0.f; });
    } else {
      to_float<E>(x, 0, v);
    }
    if (a.residual.p != nullptr) {
      to_float<E>(r, 0, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = add2(v[i], s[i]);
    }
    store_chunk<E>(static_cast<char*>(a.y.p) + (row * a.y.ld + c) * b, v);
    row += hop_rows;
    k += hop_chunks;
    if (k >= chunks) {
      k -= chunks;
      ++row;
    }
  }
}

// Any rows: a warp has 256 channels of a row, which it reads and stores one per lane at a time.
__device__ __forceinline__ float element(const RowsIn& m, long long at) {
  if (m.dtype == MOE_DTYPE_F32) return static_cast<const float*>(m.p)[at];
  const uint32_t v = static_cast<const uint16_t*>(m.p)[at];
  return m.dtype == MOE_DTYPE_BF16 ? __uint_as_float(v << 16) : __half2float(__ushort_as_half((uint16_t)v));
}
__global__ void __launch_bounds__(kThreads) dropout_any_kernel(const __grid_constant__ DropoutArgs a) {
  __shared__ __align__(16) float turns[kThreads / 32][2][kWarpCols];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float *x = turns[warp][0], *r = turns[warp][1];
  griddep_wait();
  const DropState ds(a.drop);
  const int across = (a.d + kWarpCols - 1) / kWarpCols;
  const long long tiles = (long long)a.T * across, step = (long long)gridDim.x * (kThreads / 32);
  for (long long t = (long long)blockIdx.x * (kThreads / 32) + warp; t < tiles; t += step) {
    const long long row = t / across;
    const int w0 = (int)(t - row * across) * kWarpCols;
    float in[8], res[8];
    F2 v[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = w0 + i * 32 + lane;
      in[i] = c < a.d ? element(a.x, row * a.x.ld + c) : 0.f;
      res[i] = a.residual.p != nullptr && c < a.d ? element(a.residual, row * a.residual.ld + c) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i * 32 + lane] = in[i], r[i * 32 + lane] = res[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(x[lane * 8 + 2 * i], x[lane * 8 + 2 * i + 1]);
    if (a.drop.rng != nullptr) drop8(a.drop, ds, (uint32_t)row, (uint32_t)(w0 + lane * 8), v);
    if (a.residual.p != nullptr) {
      each(v, [&](int i, float t) { return t + r[lane * 8 + i]; });
    }
    __syncwarp();
    store<Any, 32>(a.y, (int)row, 0, w0, lane, a.d, v, x);
  }
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, cudaStream_t st) {
  const long long most = 8ll * num_sms();
  if (!a.wide) {
    const long long tiles = (long long)a.T * ((a.d + kWarpCols - 1) / kWarpCols);
    const long long need = (tiles + kThreads / 32 - 1) / (kThreads / 32);
    return launch_k(dropout_any_kernel, dim3((unsigned)(need < most ? need : most)), dim3(kThreads), 0, st, a);
  }
  const int chunks = a.d / 8;
  const long long need = ((long long)a.T * chunks + kThreads - 1) / kThreads;
  const int grid = (int)(need < most ? need : most), hop = grid * kThreads;
  auto run = [&](void (*kernel)(const DropoutArgs, int, int, int)) {
    return launch_k(kernel, dim3(grid), dim3(kThreads), 0, st, a, chunks, hop / chunks, hop % chunks);
  };
  return a.x.dtype == MOE_DTYPE_F32    ? run(dropout_kernel<F32>)
         : a.x.dtype == MOE_DTYPE_BF16 ? run(dropout_kernel<BF16>)
                                       : run(dropout_kernel<F16>);
}

}  // namespace moe
