// Entry points of the norms around a block and of dropout (declarations and contracts: include/moe.h):
// validation and launch.
#include <cuda_runtime.h>
#include <climits>
#include <cmath>
#include <cstdint>

#include "norm.cuh"

namespace moe {
namespace {

int dtype_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
bool dtype_ok(int dtype) {
  return dtype == MOE_DTYPE_F32 || dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F16;
}
bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Every row starts on 16 bytes.
bool wide(const void* p, long long ld, int dtype) {
  return aligned(p, 16) && ld * dtype_bytes(dtype) % 16 == 0;
}
RowsIn in(const void* p, long long ld, int dtype) { return {p, ld, dtype, wide(p, ld, dtype)}; }
RowsOut out(void* p, long long ld, int dtype) { return {p, ld, dtype, wide(p, ld, dtype)}; }

// Whether p is in [0, 1), and dropout's threshold and factor.
bool drop_of(float p, const int64_t* rng, Drop& d) {
  if (!(p >= 0.f && p < 1.f)) return false;
  d = {};
  if (p == 0.f) return true;
  if (rng == nullptr || !aligned(rng, 8)) return false;
  d.rng = reinterpret_cast<const long long*>(rng);
  d.least = (uint32_t)std::llrint((double)p * 4294967296.0);  // p <= 1 - 2^-24: below 2^32
  d.scale = (float)(1.0 / (1.0 - (double)p));
  return true;
}

bool norm_ok(int kind) { return kind >= MOE_NORM_NONE && kind <= MOE_NORM_LAYER; }

moe_status check_cfg(const moe_residual_norm_config* c) {
  if (c == nullptr || c->T < 0 || c->d < 1 || c->gate_rows < 0 || !norm_ok(c->after) ||
      !norm_ok(c->before) || !dtype_ok(c->h_dtype) || !dtype_ok(c->y_dtype) || !dtype_ok(c->w_dtype))
    return MOE_ERR_INVALID_ARG;
  if (!(c->eps >= 0.f && std::isfinite(c->eps)) || !std::isfinite(c->alpha) ||
      !std::isfinite(c->beta) || !(c->p_drop >= 0.f && c->p_drop < 1.f))
    return MOE_ERR_INVALID_ARG;
  if ((c->ld_h != 0 && c->ld_h < c->d) || (c->ld_y != 0 && c->ld_y < c->d)) return MOE_ERR_INVALID_ARG;
  if (c->d > kNormMaxSize) return MOE_ERR_UNSUPPORTED;
  // the last element's offset, in bytes, within 63 bits
  const long long most = c->ld_h > c->ld_y ? c->ld_h : c->ld_y;
  if (most > (LLONG_MAX >> 3) / (c->T > 0 ? c->T : 1)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The parameters fit the configuration and one another; y tells whether there is a block.
bool params_ok(const moe_residual_norm_config* c, const moe_residual_norm_params* p, const void* y) {
  const int w = dtype_bytes(c->w_dtype);
  if ((p->gate != nullptr) != (c->gate_rows > 0)) return false;
  for (const void* v : {p->w_after, p->b_after, p->gate, p->w_before, p->b_before})
    if (!aligned(v, w)) return false;
  if (c->after == MOE_NORM_NONE && (p->w_after || p->b_after)) return false;
  if (c->before == MOE_NORM_NONE && (p->w_before || p->b_before)) return false;
  return y != nullptr || (c->after == MOE_NORM_NONE && c->gate_rows == 0 && c->p_drop == 0.f);
}

size_t need(const moe_residual_norm_config* c) {
  const int most = norm_grad_runs(c->d, kNormMaxSms), runs = c->T < most ? c->T : most;
  return (4ull * kNormParts * c->d * runs + 255) / 256 * 256;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_residual_norm(const moe_residual_norm_config* cfg, const void* h, const void* y,
                             const moe_residual_norm_params* params, void* h_out, void* n,
                             moe_stream_t stream) {
  const moe_status r = check_cfg(cfg);
  if (r != MOE_OK) return r;
  if (cfg->T == 0) return MOE_OK;
  const int hs = dtype_bytes(cfg->h_dtype), ys = dtype_bytes(cfg->y_dtype);
  if (!h || !params || (n != nullptr) != (cfg->before != MOE_NORM_NONE) || (!h_out && !n) ||
      !aligned(h, hs) || !aligned(h_out, hs) || !aligned(y, ys) || !aligned(n, ys) ||
      !params_ok(cfg, params, y))
    return MOE_ERR_INVALID_ARG;
  NormArgs a = {};
  if (!drop_of(cfg->p_drop, params->rng, a.drop)) return MOE_ERR_INVALID_ARG;
  const long long d = cfg->d;
  a.h = in(h, cfg->ld_h ? cfg->ld_h : d, cfg->h_dtype);
  a.y = in(y, cfg->ld_y ? cfg->ld_y : d, cfg->y_dtype);
  a.w_after = in(params->w_after, 0, cfg->w_dtype);
  a.b_after = in(params->b_after, 0, cfg->w_dtype);
  a.gate = in(params->gate, d, cfg->w_dtype);
  a.w_before = in(params->w_before, 0, cfg->w_dtype);
  a.b_before = in(params->b_before, 0, cfg->w_dtype);
  a.h_out = out(h_out, d, cfg->h_dtype);
  a.n = out(n, d, cfg->y_dtype);
  a.wide = d % 8 == 0 && a.h.wide && (!y || a.y.wide) && (!h_out || a.h_out.wide) && (!n || a.n.wide);
  for (const RowsIn& m : {a.w_after, a.b_after, a.gate, a.w_before, a.b_before})
    a.wide = a.wide && (m.p == nullptr || m.wide);
  a.T = cfg->T;
  a.d = cfg->d;
  a.after = cfg->after;
  a.before = cfg->before;
  a.gate_rows = cfg->gate_rows;
  a.eps = cfg->eps;
  a.alpha = cfg->alpha;
  a.beta = cfg->beta;
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = !a.wide                          ? launch_norm_any(a, st)
                        : cfg->h_dtype == MOE_DTYPE_F32  ? launch_norm_f32(a, st)
                        : cfg->h_dtype == MOE_DTYPE_BF16 ? launch_norm_bf16(a, st)
                                                         : launch_norm_f16(a, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_residual_norm_workspace_size(const moe_residual_norm_config* cfg, size_t* bytes) {
  const moe_status r = check_cfg(cfg);
  if (r != MOE_OK) return r;
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = need(cfg);
  return MOE_OK;
}

moe_status moe_residual_norm_backward(const moe_residual_norm_config* cfg, const void* h_out,
                                      const void* y, const void* d_h_out, const void* d_n,
                                      const moe_residual_norm_params* params, void* d_h, void* d_y,
                                      const moe_residual_norm_grads* grads, void* ws, size_t ws_bytes,
                                      moe_stream_t stream) {
  const moe_status r = check_cfg(cfg);
  if (r != MOE_OK) return r;
  const cudaStream_t st = (cudaStream_t)stream;
  if (!grads || !params) return MOE_ERR_INVALID_ARG;
  for (const float* g : {grads->w_after, grads->b_after, grads->gate, grads->w_before, grads->b_before})
    if (!aligned(g, 4)) return MOE_ERR_INVALID_ARG;
  // a gradient for a parameter of a norm or gate that there is not
  if ((cfg->after == MOE_NORM_NONE && (grads->w_after || grads->b_after)) ||
      (cfg->before == MOE_NORM_NONE && (grads->w_before || grads->b_before)) ||
      (cfg->gate_rows == 0 && grads->gate))
    return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) {
    for (float* g : {grads->w_after, grads->b_after, grads->w_before, grads->b_before})
      if (g != nullptr && cudaMemsetAsync(g, 0, 4ull * cfg->d, st) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  const int hs = dtype_bytes(cfg->h_dtype), ys = dtype_bytes(cfg->y_dtype);
  if ((!d_h_out && !d_n) || !d_h || (y != nullptr) != (d_y != nullptr) ||
      (d_n != nullptr && (cfg->before == MOE_NORM_NONE || !h_out)) || !aligned(h_out, hs) ||
      !aligned(d_h_out, hs) || !aligned(d_h, hs) || !aligned(y, ys) || !aligned(d_n, ys) ||
      !aligned(d_y, ys) || !params_ok(cfg, params, y))
    return MOE_ERR_INVALID_ARG;
  NormGradArgs a = {};
  if (!drop_of(cfg->p_drop, params->rng, a.drop)) return MOE_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws, 256) || ws_bytes < need(cfg)) return MOE_ERR_WORKSPACE;
  const long long d = cfg->d;
  a.h = in(h_out, cfg->ld_h ? cfg->ld_h : d, cfg->h_dtype);
  a.y = in(y, cfg->ld_y ? cfg->ld_y : d, cfg->y_dtype);
  a.d_h_out = in(d_h_out, d, cfg->h_dtype);
  a.d_n = in(d_n, d, cfg->y_dtype);
  a.w_after = in(params->w_after, 0, cfg->w_dtype);
  a.b_after = in(params->b_after, 0, cfg->w_dtype);
  a.gate = in(params->gate, d, cfg->w_dtype);
  a.w_before = in(params->w_before, 0, cfg->w_dtype);
  a.d_h = out(d_h, d, cfg->h_dtype);
  a.d_y = out(d_y, d, cfg->y_dtype);
  a.d_w_after = grads->w_after;
  a.d_b_after = grads->b_after;
  a.d_gate = grads->gate;
  a.d_w_before = grads->w_before;
  a.d_b_before = grads->b_before;
  a.part = static_cast<float*>(ws);
  a.wide = d % 8 == 0 && a.d_h.wide && (!d_n || (a.h.wide && a.d_n.wide)) && (!d_h_out || a.d_h_out.wide) &&
           (!y || (a.y.wide && a.d_y.wide)) && wide(grads->gate, d, MOE_DTYPE_F32);
  for (const RowsIn& m : {a.w_after, a.b_after, a.gate, a.w_before})
    a.wide = a.wide && (m.p == nullptr || m.wide);
  a.T = cfg->T;
  a.d = cfg->d;
  a.after = cfg->after;
  a.before = cfg->before;
  a.gate_rows = cfg->gate_rows;
  a.eps = cfg->eps;
  a.alpha = cfg->alpha;
  a.beta = cfg->beta;
  int ctas = 0;
  cudaError_t e = !a.wide                          ? launch_norm_grad_any(a, &ctas, st)
                  : cfg->h_dtype == MOE_DTYPE_F32  ? launch_norm_grad_f32(a, &ctas, st)
                  : cfg->h_dtype == MOE_DTYPE_BF16 ? launch_norm_grad_bf16(a, &ctas, st)
                                                   : launch_norm_grad_f16(a, &ctas, st);
  if (e == cudaSuccess) e = launch_norm_join(a, ctas, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_dropout(int32_t T, int32_t d, int32_t dtype, const void* x, int64_t ld_x, float p,
                       const int64_t* rng, const void* residual, int64_t ld_r, void* y,
                       moe_stream_t stream) {
  if (T < 0 || d < 1 || !dtype_ok(dtype) || !(p >= 0.f && p < 1.f) || (ld_x != 0 && ld_x < d) ||
      (ld_r != 0 && ld_r < d))
    return MOE_ERR_INVALID_ARG;
  const long long most = ld_x > ld_r ? ld_x : ld_r;
  if (d > INT32_MAX - 4096 || most > (LLONG_MAX >> 3) / (T > 0 ? T : 1)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const int size = dtype_bytes(dtype);
  if (!x || !y || !aligned(x, size) || !aligned(y, size) || !aligned(residual, size))
    return MOE_ERR_INVALID_ARG;
  DropoutArgs a = {};
  if (!drop_of(p, rng, a.drop)) return MOE_ERR_INVALID_ARG;
  a.x = in(x, ld_x ? ld_x : d, dtype);
  a.residual = in(residual, ld_r ? ld_r : d, dtype);
  a.y = out(y, d, dtype);
  a.wide = d % 8 == 0 && a.x.wide && a.y.wide && (!residual || a.residual.wide);
  a.T = T;
  a.d = d;
  return launch_dropout(a, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
