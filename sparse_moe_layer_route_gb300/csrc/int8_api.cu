// Entry points of the 8-bit weights and activations (declarations and contracts: include/moe.h):
// validation, workspace carving and launch sequencing.
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#include "int8.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr size_t kHead = 512;  // status word and counter block, as in every workspace
// Where int8_gemv.cu is faster than the tensor cores: few rows, or so little work that a unit's long
// pipeline (and the launches in front of it) is most of a tensor-core product's time.
//   product: 8 rows of [14336 x 4096] 16 against 21.5 us, 12 rows 26 against 21; 0.3 G multiply-adds (150
//   rows of [1000 x 2048]) 11 against 16, 0.6 G (20 segments of 30 rows) 28 against 15; between them it
//   depends on the shape (300 rows in 20 segments of [1000 x 1024], 0.3 G, 17 against 14, of [600 x 512]
//   9.4 against 14).
//   experts: decode shape, 6 tokens 92 against 119 us, 12 tokens 162 against 183, 24 tokens 283 against 281;
//   64 + 2 experts of [2048 x 1408], 6 a token, 12 tokens 88 against 88, 16 tokens 101 against 93; of
//   small layers, 32 tokens, 60 M multiply-adds, 18 against 22, and 64 tokens, 100 M, 22 against 22.
bool few_rows(int rows, int K, int N) { return rows <= 8 || (double)rows * K * N <= 4e8; }
// Sums of up to 2^17 products of activations' and weights' codes (127 * 128) stay in 32 bits.
bool few_tokens(const Shape& s) {
  return s.d <= 131072 && s.f <= 131072 && (s.T <= 12 || 3.0 * s.rows * s.d * s.f <= 1e8);
}

// Rows and channels up to this: the kernels add a tile's or a block's size to them in 32 bits.
constexpr int32_t kMostSize = INT32_MAX - 1023;

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
int dtype_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
bool dtype_ok(int dtype) {
  return dtype == MOE_DTYPE_F32 || dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F16;
}
moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

moe_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  return ws == nullptr || !aligned(ws, 256) || ws_bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

moe_status check_matmul(int32_t rows, int32_t K, int32_t N, int32_t n_mat) {
  if (rows < 0 || K < 1 || N < 1 || n_mat < 1) return MOE_ERR_INVALID_ARG;
  if (rows > kMostSize || n_mat > 256 || K % 16 != 0 || K > 65536 || N >= (1 << 27))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Workspace of a product: the rows' codes in fp16, then the partial sums of a K that is done in pieces.
size_t matmul_part(int32_t rows, int32_t K) {
  return kHead + ((size_t)rows * K * 2 + 255) / 256 * 256;
}
size_t matmul_part_bytes(int32_t rows, int32_t K, int32_t N, int32_t n_mat) {
  const int splits = few_rows(rows, K, N) ? 1 : int8_splits(rows, K, N, n_mat);
  return splits > 1 ? 4ull * splits * rows * int8_part_cols(N) : 0;
}
size_t matmul_need(int32_t rows, int32_t K, int32_t N, int32_t n_mat) {
  return matmul_part(rows, K) + matmul_part_bytes(rows, K, N, n_mat);
}

// Buffers of one FFN call.
struct FfnLayout {
  size_t xq, sx, h, hq, sh, total;
};
FfnLayout ffn_layout(const Shape& s) {
  FfnLayout L;
  size_t o = kHead;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  const size_t x_rows = s.TK + (s.S > 0 ? s.T : 0);
  L.xq = take(2ull * x_rows * s.d);
  L.sx = take(4ull * x_rows);
  // fp32: an fp16 H (2^-12 of the value) would move about 1 code in 150 by one when H is quantized
  // (3.5e-3 of the layer output's norm measured), fp32 moves none to speak of
  L.h = take(4ull * s.rows * s.f);
  L.hq = take(2ull * s.rows * s.f);
  L.sh = take(4ull * s.rows);
  L.total = o;
  return L;
}

bool mat_ok(const moe_int8_matrix& m) {
  return m.q && m.scale && aligned(m.q, 16) && aligned(m.scale, 4);
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_quantize_rows(int32_t T, int32_t d, int32_t dtype, const void* x, int64_t ld,
                             int8_t* q, float* scale, moe_stream_t stream) {
  if (T < 0 || d < 1 || !dtype_ok(dtype) || (ld != 0 && ld < d)) return MOE_ERR_INVALID_ARG;
  if (d > kMostSize) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !q || !scale || !aligned(x, dtype_bytes(dtype)) || !aligned(scale, 4))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(
      launch_quantize_rows(T, d, dtype, x, ld != 0 ? ld : d, q, scale, (cudaStream_t)stream));
}

moe_status moe_quantize_channels(int32_t n_mat, int32_t K, int32_t N, const uint16_t* W, int8_t* q,
                                 float* scale, moe_stream_t stream) {
  if (n_mat < 1 || K < 1 || N < 1 || !W || !q || !scale) return MOE_ERR_INVALID_ARG;
  if (!aligned(W, 2) || !aligned(scale, 4)) return MOE_ERR_INVALID_ARG;
  if (n_mat > 65535 || K > kMostSize || N > kMostSize) return MOE_ERR_UNSUPPORTED;
  return cuda_status(launch_quantize_channels(n_mat, K, N, W, q, scale, (cudaStream_t)stream));
}

moe_status moe_int8_matmul_workspace_size(int32_t rows, int32_t K, int32_t N, int32_t n_mat,
                                          size_t* bytes) {
  const moe_status r = check_matmul(rows, K, N, n_mat);
  if (r != MOE_OK) return r;
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  // the most that any number of rows up to this one needs: fewer may have more pieces of K
  size_t most = matmul_need(rows, K, N, n_mat);
  for (long long r = 0; r < rows; ++r) {
    r = int8_splits_end(r, n_mat);
    if (r >= rows || int8_splits(r, K, N, n_mat) == 1) break;
    most = std::max(most, matmul_need((int32_t)r, K, N, n_mat));
  }
  *bytes = most;
  return MOE_OK;
}

moe_status moe_int8_matmul(int32_t rows, int32_t K, int32_t N, int32_t n_mat, const int8_t* q_x,
                           const float* s_x, const int8_t* q_w, const float* s_w,
                           const int32_t* offsets, int32_t y_dtype, void* y, void* ws,
                           size_t ws_bytes, moe_stream_t stream) {
  moe_status r = check_matmul(rows, K, N, n_mat);
  if (r != MOE_OK) return r;
  if (!dtype_ok(y_dtype) || (offsets == nullptr && n_mat != 1)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!q_x || !s_x || !q_w || !s_w || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned(q_x, 16) || !aligned(q_w, 16) || !aligned(s_x, 4) || !aligned(s_w, 4) ||
      !aligned(offsets, 4) || !aligned(y, dtype_bytes(y_dtype)))
    return MOE_ERR_INVALID_ARG;
  if ((r = check_ws(ws, ws_bytes, matmul_need(rows, K, N, n_mat))) != MOE_OK) return r;
  const cudaStream_t st = (cudaStream_t)stream;
  Int8Gemm g = {};
  g.x_rows = rows;
  g.sx = s_x;
  g.qw = q_w;
  g.sw = s_w;
  g.offsets = offsets;
  g.out = y;
  g.out_dtype = y_dtype;
  g.status = at<int>(ws, 0);
  g.rows = rows;
  g.K = K;
  g.N = N;
  g.n_mat = n_mat;
  g.T = 1;
  if (few_rows(rows, K, N)) {
    g.x8 = q_x;
    return cuda_status(launch_int8_gemv(kInt8Matrix, g, rows, st));
  }
  uint16_t* xq = at<uint16_t>(ws, kHead);
  g.xq = xq;
  const cudaError_t e = launch_widen_codes(q_x, xq, (long long)rows * K, st);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  if (matmul_part_bytes(rows, K, N, n_mat) > 0)
    return cuda_status(launch_int8_split(g, at<float>(ws, matmul_part(rows, K)), st));
  return cuda_status(launch_int8_gemm(kInt8Matrix, g, st));
}

moe_status moe_grouped_ffn_int8_workspace_size(const moe_config* cfg, size_t* bytes) {
  size_t plain = 0;
  const moe_status r = moe_workspace_size(cfg, &plain);  // the layer's checks of a configuration
  if (r != MOE_OK) return r;
  if (bytes == nullptr || cfg->weight_bits != 0) return MOE_ERR_INVALID_ARG;
  *bytes = cfg->T == 0 ? kHead : ffn_layout(make_shape(*cfg)).total;
  return MOE_OK;
}

moe_status moe_grouped_ffn_int8(const moe_config* cfg, const uint16_t* x, const int32_t* perm_slot,
                                const int32_t* offsets, const float* topk_w,
                                const moe_int8_weights* w, uint16_t* y_slot, void* ws,
                                size_t ws_bytes, moe_stream_t stream) {
  size_t need = 0;
  moe_status r = moe_grouped_ffn_int8_workspace_size(cfg, &need);
  if (r != MOE_OK) return r;
  if (cfg->T == 0) return MOE_OK;
  if (!x || !perm_slot || !offsets || !w || !y_slot) return MOE_ERR_INVALID_ARG;
  if (!mat_ok(w->gate) || !mat_ok(w->up) || !mat_ok(w->down)) return MOE_ERR_INVALID_ARG;
  if (cfg->n_shared > 0 && (!mat_ok(w->sh_gate) || !mat_ok(w->sh_up) || !mat_ok(w->sh_down)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y_slot, 16) || !aligned(perm_slot, 4) || !aligned(offsets, 4) ||
      !aligned(topk_w, 4))
    return MOE_ERR_INVALID_ARG;
  if ((r = check_ws(ws, ws_bytes, need)) != MOE_OK) return r;
  const Shape s = make_shape(*cfg);
  const FfnLayout L = ffn_layout(s);
  const cudaStream_t st = (cudaStream_t)stream;
  // few tokens: 8-bit codes and integer dot products, else fp16 codes and the tensor cores
  const bool few = few_tokens(s);
  int* status = at<int>(ws, 0);
  Int8Gemm g = {};
  g.xq = at<uint16_t>(ws, L.xq);
  g.x8 = at<int8_t>(ws, L.xq);
  g.x_rows = s.TK + (s.S > 0 ? s.T : 0);
  g.sx = at<float>(ws, L.sx);
  g.qw = w->gate.q;
  g.sw = w->gate.scale;
  g.qw2 = w->up.q;
  g.sw2 = w->up.scale;
  g.sh_qw = w->sh_gate.q;
  g.sh_sw = w->sh_gate.scale;
  g.sh_qw2 = w->sh_up.q;
  g.sh_sw2 = w->sh_up.scale;
  g.offsets = offsets;
  g.out = at<float>(ws, L.h);
  g.status = status;
  g.rows = (int)s.TK;
  g.K = s.d;
  g.N = s.f;
  g.n_mat = s.E;
  g.S = s.S;
  g.T = s.T;
  auto product = [&](Int8Pass pass) {
    return few ? launch_int8_gemv(pass, g, s.T, st) : launch_int8_gemm(pass, g, st);
  };
  cudaError_t e =
      few ? launch_quantize_gather(s, x, perm_slot, offsets, at<int8_t>(ws, L.xq),
                                   at<float>(ws, L.sx), status, st)
          : launch_quantize_gather(s, x, perm_slot, offsets, at<uint16_t>(ws, L.xq),
                                   at<float>(ws, L.sx), status, st);
  if (e == cudaSuccess) e = product(kInt8SwiGLU);
  if (e == cudaSuccess)
    e = few ? launch_quantize_hidden(s, at<float>(ws, L.h), offsets, at<int8_t>(ws, L.hq),
                                     at<float>(ws, L.sh), st)
            : launch_quantize_hidden(s, at<float>(ws, L.h), offsets, at<uint16_t>(ws, L.hq),
                                     at<float>(ws, L.sh), st);
  g.xq = at<uint16_t>(ws, L.hq);
  g.x8 = at<int8_t>(ws, L.hq);
  g.x_rows = s.rows;
  g.sx = at<float>(ws, L.sh);
  g.perm_slot = perm_slot;
  g.qw = w->down.q;
  g.sw = w->down.scale;
  g.sh_qw = w->sh_down.q;
  g.sh_sw = w->sh_down.scale;
  g.qw2 = g.sh_qw2 = nullptr;
  g.sw2 = g.sh_sw2 = nullptr;
  g.topk_w = topk_w;
  g.out = y_slot;
  g.K = s.f;
  g.N = s.d;
  if (e == cudaSuccess) e = product(kInt8Slot);
  return cuda_status(e);
}

}  // extern "C"
