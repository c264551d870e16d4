// Norms around a block, residual, gates and dropout: arguments and launches. Kernels: norm_forward.cuh,
// norm_backward.cuh (compiled once per type of the stream in norm_f32.cu, norm_bf16.cu, norm_f16.cu, and for
// rows of any alignment in norm_any.cu) and dropout.cu.
#pragma once
#include "internal.h"

namespace moe {

constexpr int kNormMaxSize = 65536;  // d: eight CTAs of a cluster with 8192 channels each
constexpr int kNormMaxSms = 160;     // of a full GPU of this kind
constexpr int kNormSmem = 227 * 1024;

// Channels of a CTA of a cluster of cl, and the CTAs that share a row.
__host__ __device__ __forceinline__ int norm_width(int d, int cl) { return ((d + 7) / 8 + cl - 1) / cl * 8; }
__host__ __device__ __forceinline__ int norm_cluster(int d) {
  int cl = 1;
  while (norm_width(d, cl) > 8192) cl *= 2;
  return cl;
}
// Runs of tokens of the gradient at most (of a CTA, or of a cluster's), each with partial sums in the workspace: an SM
// has 512 threads of them, and up to 1024 channels a CTA has 256, above that as many warps as a row has pieces of 256
// channels.
__host__ __device__ __forceinline__ int norm_grad_threads(int d) {
  const int pieces = (d + 255) / 256;
  return d <= 1024 ? 256 : pieces < 16 ? 32 * pieces : 512;
}
__host__ __device__ __forceinline__ int norm_grad_runs(int d, int sms) {
  return 512 / norm_grad_threads(d) * sms / norm_cluster(d);
}

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
  float* part;                // [runs][kNormParts][d]
  Drop drop;
  int T, d, after, before, gate_rows;
  float eps, alpha, beta;
};
// Partial sums of a run: gradients of w_after, b_after, w_before, b_before, and of the gates that it shares
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
