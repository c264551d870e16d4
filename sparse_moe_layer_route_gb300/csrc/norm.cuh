// Norms around a block, residual, gates and dropout: arguments and launches. Kernels: norm_forward.cuh,
// norm_backward.cuh (compiled once per type of the stream in norm_f32.cu, norm_bf16.cu, norm_f16.cu, and for
// rows of any alignment in norm_any.cu) and dropout.cu.
#pragma once
#include "internal.h"

namespace moe {

constexpr int kNormMaxSize = 65536;  // d: eight CTAs of a cluster with 8192 channels each
// CTAs of the gradient at most, each with partial sums in the workspace: three an SM of narrow rows, else two.
__host__ __device__ __forceinline__ int norm_max_ctas(int d) { return d <= 2048 ? 480 : 320; }
constexpr int kNormSmem = 227 * 1024;

// Rows of a matrix: elements between rows, type, and whether every row starts on 16 bytes.
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
  bool wide;             // of every row that is read or written, and d % 8 == 0
  RowsIn h, y;           // y.p nullptr: no block, h' = alpha h
  RowsIn w_after, b_after, gate, w_before, b_before;
  RowsOut h_out, n;
  Drop drop;
  int T, d, after, before, gate_rows;
  float eps, alpha, beta;
};

struct NormGradArgs {
  bool wide;                  // as in NormArgs
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

// By y's type, for rows that start on 16 bytes (one per type of the stream), and for any.
cudaError_t launch_norm_f32(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_bf16(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_f16(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_any(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_grad_f32(const NormGradArgs& a, int* ctas, cudaStream_t st);
cudaError_t launch_norm_grad_bf16(const NormGradArgs& a, int* ctas, cudaStream_t st);
cudaError_t launch_norm_grad_f16(const NormGradArgs& a, int* ctas, cudaStream_t st);
cudaError_t launch_norm_grad_any(const NormGradArgs& a, int* ctas, cudaStream_t st);
// The sum over the CTAs' partial sums that a launch of the gradient leaves.
cudaError_t launch_norm_join(const NormGradArgs& a, int ctas, cudaStream_t st);

struct DropoutArgs {
  bool wide;           // as in NormArgs
  RowsIn x, residual;  // residual.p nullptr: none
  RowsOut y;
  Drop drop;
  int T, d;
};
cudaError_t launch_dropout(const DropoutArgs& a, cudaStream_t st);

// Tokens of a CTA of the gradient.
__host__ __device__ __forceinline__ int norm_rows_per_cta(int T, int ctas) {
  return (int)(((long long)T + ctas - 1) / ctas);
}

}  // namespace moe
