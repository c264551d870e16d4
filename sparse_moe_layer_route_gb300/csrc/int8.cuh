// 8-bit expert products: the quantization rule and the launch interface between the entry points
// (int8_api.cu) and the kernels (int8_rows.cu, int8_gemv.cu, int8_gemm.cu, int8_split.cu).
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "internal.h"

namespace moe {

// Scale of a row from the largest magnitude bits among its values (sign cleared; in this order
// infinity follows every number and NaN follows infinity, so either becomes the scale).
__device__ __forceinline__ float int8_scale(uint32_t top_bits) {
  return __fmul_rn(__uint_as_float(top_bits), 1.0f / 127.0f);
}

// Code of one value: rint(x / scale) to nearest even. The clamp acts where the scale is subnormal
// (its rounding may leave x / scale past 127); a zero or non-finite scale gives 0.
__device__ __forceinline__ int int8_code(float x, float scale) {
  if (scale == 0.0f) return 0;
  const int v = __float2int_rn(__fdiv_rn(x, scale));  // NaN converts to 0
  return max(-127, min(127, v));
}

// Four codes to fp16: with the sign bit flipped a code c is the byte c + 128; 0x6400 | byte is the fp16
// 1024 + byte (fp16 counts by ones from 1024 to 2048), and subtracting 1152 is exact.
__device__ __forceinline__ void widen4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = codes ^ 0x80808080u;
  lo = __byte_perm(u, 0x64646464u, 0x4140);
  hi = __byte_perm(u, 0x64646464u, 0x4342);
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
}

// Whether offsets r0 and r1 bound a segment of the rows [0, rows). One that they do not is empty and reported
// by the product (MOE_DEVFAULT_BAD_TILE); the others are computed all the same, and where they share rows (only
// an unsound segment between two sound ones lets them) the first of them has those rows.
__device__ __forceinline__ bool segment_ok(int r0, int r1, int rows) {
  return r0 >= 0 && r1 >= r0 && r1 <= rows;
}

// One grouped product. Segment e < n_mat holds positions [offsets[e], offsets[e + 1]) (offsets
// NULL: all `rows`); with shared experts, segment n_mat + s is positions
// [rows + s * T, rows + (s + 1) * T). A sum takes the two scales one after the other: their product may be past
// fp32's range where the result is not. The activations' codes, in fp16 (exact) or 8 bits, have row p for
// position p, except that the SwiGLU pass's shared experts all read rows [rows, rows + T).
struct Int8Gemm {
  const uint16_t* xq;      // [x_rows, K] fp16 (tensor cores)
  const int8_t* x8;        // [x_rows, K] (launch_int8_gemv)
  const float* sx;         // [x_rows]
  long long x_rows;
  const int8_t *qw, *qw2;  // [n_mat, N, K]; qw2: the up projection of the SwiGLU pass
  const float *sw, *sw2;
  const int8_t *sh_qw, *sh_qw2;  // shared experts [S, N, K]
  const float *sh_sw, *sh_sw2;
  const int32_t* offsets;
  const int32_t* perm_slot;  // slot pass: position -> slot
  const float* topk_w;       // slot pass: gate per slot (NULL: 1)
  void* out;
  int* status;
  int rows, K, N, n_mat, S, T;
  int out_dtype;             // matrix pass
  int splits;                // partial pass: pieces of K
  int tile_rows;             // tensor cores: the tallest row tile
};

enum Int8Pass {
  kInt8Matrix = 0,  // out [rows, N] = product
  kInt8SwiGLU = 1,  // out [rows + S T, N] fp32 = silu(gate product) * (up product)
  kInt8Slot = 2,    // out [slot, N] fp16 = gate weight * product
  kInt8Partial = 3  // out [splits][rows, N] fp32 = sums over one piece of K, without scales
};

// Tensor cores (int8_gemm.cu).
cudaError_t launch_int8_gemm(Int8Pass pass, const Int8Gemm& g, cudaStream_t st);
// A few rows (int8_gemv.cu); most_rows: no segment has more.
cudaError_t launch_int8_gemv(Int8Pass pass, const Int8Gemm& g, int most_rows, cudaStream_t st);
// Pieces of K that give a product with few work units something to do on every SM (1: none), for a
// matrix pass of this shape; and that product: partial sums to `part` (int8_splits() * rows * int8_part_cols(N) floats),
// then their sums, scaled, to g.out.
int int8_splits(long long rows, int K, int N, int n_mat);
// The largest number of rows with the pieces of this one (more rows never have more).
long long int8_splits_end(long long rows, int n_mat);
// Floats of a row of partial sums: rows begin on 16 bytes whatever N, so they are stored in 16-byte pieces.
__host__ __device__ inline int int8_part_cols(int N) { return (N + 3) / 4 * 4; }
constexpr int kInt8StageK = 128;  // k per shared-memory stage
// Rows per segment (an even spread's) up to which row tiles have at most 64 and 128 rows, not 256.
constexpr int kInt8Mean64 = 24, kInt8Mean128 = 104;
// Height of a segment's row tiles, a multiple of 32 up to NT: as few tiles as NT allows, of equal heights,
// as a low tile costs the widening of its weights whatever it holds: about 400 clk per 64 k with two sets of
// widening warps, the MMAs of 194 rows; with three sets that of 130 rows. The rule's numbers are the two
// sets': past 192 rows a tile costs its MMAs, 2 clk a row, and about 40 for the overlap with the next one,
// taken where that is less than one more tile of 400 (400 rows: two of 224 and 176, not three). 64 segments of about 200 rows of
// [2048 x 2048] 91 us, with tiles of up to 192 rows 116; of about 300 rows 141, the same.
__host__ __device__ inline int int8_tile_height(int rows, int NT) {
  const int most = rows < 1 ? 1 : rows;
  int n = (most + NT - 1) / NT;
  int height = ((most + n - 1) / n + 31) / 32 * 32;
  if (height > 192) {
    const int m = (most + 191) / 192;
    if (n * (2 * height + 40) >= m * 400) {
      n = m;
      height = ((most + n - 1) / n + 31) / 32 * 32;
    }
  }
  return height;
}
cudaError_t launch_int8_split(const Int8Gemm& g, float* part, cudaStream_t st);
cudaError_t launch_quantize_rows(int T, int d, int dtype, const void* x, long long ld, int8_t* q,
                                 float* scale, cudaStream_t st);
cudaError_t launch_quantize_channels(int n_mat, int K, int N, const uint16_t* W, int8_t* q,
                                     float* scale, cudaStream_t st);
// fp16 copies of int8 codes (n a multiple of 16; both 16-byte aligned).
cudaError_t launch_widen_codes(const int8_t* q, uint16_t* xq, long long n, cudaStream_t st);
// The FFN's activations in expert order: rows [0, TK) from the token of slot perm_slot[p] (written
// for p < offsets[E]; a slot outside [0, TK) becomes a zero row and MOE_DEVFAULT_BAD_TILE), then,
// with shared experts, rows [TK, TK + T) from every token. Codes as uint16_t (fp16) or int8_t.
template <typename QT>
cudaError_t launch_quantize_gather(const Shape& s, const uint16_t* x, const int32_t* perm_slot,
                                   const int32_t* offsets, QT* xq, float* sx, int* status,
                                   cudaStream_t st);
// H [rows, f] fp32 to codes and scales; positions in [offsets[E], TK) are skipped.
template <typename QT>
cudaError_t launch_quantize_hidden(const Shape& s, const float* h, const int32_t* offsets, QT* hq,
                                   float* sh, cudaStream_t st);

}  // namespace moe
