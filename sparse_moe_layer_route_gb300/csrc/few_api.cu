// Entry points of the MoE layer for a few tokens (declarations and contracts: include/moe.h):
// validation, workspace carving and launch.
#include <cuda_runtime.h>
#include <climits>
#include <cstdint>

#include "few.cuh"
#include "internal.h"

namespace moe {
namespace {

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

moe_status check(const moe_config* cfg) {
  size_t plain = 0;
  const moe_status r = moe_workspace_size(cfg, &plain);  // the layer's checks of a configuration
  if (r != MOE_OK) return r;
  if (cfg->T > MOE_FEW_MAX_TOKENS || cfg->weight_bits != 0 || cfg->d > kFewMaxSize ||
      cfg->d_ff > kFewMaxSize || make_shape(*cfg).reroute)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool experts_ok(const moe_config* cfg, const moe_weights* w) {
  if (!w || !w->W_gate || !w->W_up || !w->W_down) return false;
  if (!aligned(w->W_gate, 16) || !aligned(w->W_up, 16) || !aligned(w->W_down, 16)) return false;
  if (cfg->n_shared == 0) return true;
  return w->Wsh_gate && w->Wsh_up && w->Wsh_down && aligned(w->Wsh_gate, 16) &&
         aligned(w->Wsh_up, 16) && aligned(w->Wsh_down, 16);
}

// The arguments that both entry points share.
FewArgs common(const Shape& s, const FewLayout& L, const moe_weights* w, const uint16_t* x,
               uint16_t* out, void* ws) {
  FewArgs a = {};
  a.x = x;
  a.gate = w->W_gate;
  a.up = w->W_up;
  a.down = w->W_down;
  a.sh_gate = w->Wsh_gate;
  a.sh_up = w->Wsh_up;
  a.sh_down = w->Wsh_down;
  a.out = out;
  a.logits = at<float>(ws, L.logits);
  a.xf = at<uint16_t>(ws, L.xf);
  a.h = at<uint32_t>(ws, L.h);
  a.count = at<int>(ws, L.count);
  a.part = at<float>(ws, L.part);
  a.status = at<int>(ws, 0);
  a.meta = at<FewMeta>(ws, L.meta);
  a.T = s.T;
  a.d = s.d;
  a.E = s.E;
  a.k = s.k;
  a.f = s.f;
  a.S = s.S;
  a.mode = s.mode;
  a.G = s.G;
  a.Gk = s.Gk;
  a.C = s.C;
  a.tau = s.tau;
  a.limit_ns = kFewWaitNs;
  return a;
}

moe_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  return ws == nullptr || !aligned(ws, 256) || ws_bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_few_workspace_size(const moe_config* cfg, size_t* bytes) {
  const moe_status r = check(cfg);
  if (r != MOE_OK) return r;
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = cfg->T == 0 ? 512 : few_layout(make_shape(*cfg)).total;
  return MOE_OK;
}

moe_status moe_layer_forward_few(const moe_config* cfg, const moe_weights* w, const uint16_t* x,
                                 const float* gumbel_u, uint16_t* out, moe_route_out* route_out,
                                 void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status r = check(cfg);
  if (r != MOE_OK) return r;
  const cudaStream_t st = (cudaStream_t)stream;
  if (route_out != nullptr)
    for (const void* p : {(const void*)route_out->topk_idx, (const void*)route_out->topk_w,
                          (const void*)route_out->counts, (const void*)route_out->offsets,
                          (const void*)route_out->perm_slot, (const void*)route_out->slot_pos})
      if (!aligned(p, 4)) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) {  // as in moe_layer_forward: every expert receives nothing
    if (route_out == nullptr) return MOE_OK;
    cudaError_t e = cudaSuccess;
    if (route_out->counts) e = cudaMemsetAsync(route_out->counts, 0, 4ull * cfg->E, st);
    if (e == cudaSuccess && route_out->offsets)
      e = cudaMemsetAsync(route_out->offsets, 0, 4ull * (cfg->E + 1), st);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  if (!x || !out || !aligned(x, 16) || !aligned(out, 16) || !experts_ok(cfg, w) || !w->W_g ||
      !aligned(w->W_g_t, 16))
    return MOE_ERR_INVALID_ARG;
  if (cfg->mode == MOE_ROUTE_BIAS_SELECT && (!w->expert_bias || !aligned(w->expert_bias, 4)))
    return MOE_ERR_INVALID_ARG;
  if (cfg->mode == MOE_ROUTE_GUMBEL && (!gumbel_u || !aligned(gumbel_u, 4)))
    return MOE_ERR_INVALID_ARG;
  const Shape s = make_shape(*cfg);
  const FewLayout L = few_layout(s);
  if ((r = check_ws(ws, ws_bytes, L.total)) != MOE_OK) return r;
  FewArgs a = common(s, L, w, x, out, ws);
  a.bias = w->expert_bias;
  a.u = gumbel_u;
  a.W_g_t = w->W_g_t;
  if (route_out != nullptr) a.ro = *route_out;
  if (a.W_g_t == nullptr) {
    uint16_t* t = at<uint16_t>(ws, L.wg_t);
    if (launch_router_transpose(s.d, s.E, w->W_g, t, st) != cudaSuccess) return MOE_ERR_CUDA;
    a.W_g_t = t;
  }
  return launch_few(a, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"

namespace {

// moe_experts_few up to its launch.
moe_status prepare_experts(const moe_config* cfg, const moe_weights* w, const uint16_t* x, const int32_t* topk_idx,
                           const float* topk_w, uint16_t* out, void* ws, size_t ws_bytes, FewArgs& a) {
  if (!x || !topk_idx || !out || !aligned(x, 16) || !aligned(out, 16) || !aligned(topk_idx, 4) ||
      !aligned(topk_w, 4) || !experts_ok(cfg, w))
    return MOE_ERR_INVALID_ARG;
  const Shape s = make_shape(*cfg);
  const FewLayout L = few_layout(s);
  const moe_status r = check_ws(ws, ws_bytes, L.total);
  if (r != MOE_OK) return r;
  a = common(s, L, w, x, out, ws);
  a.idx_in = topk_idx;
  a.w_in = topk_w;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_experts_few(const moe_config* cfg, const moe_weights* w, const uint16_t* x,
                           const int32_t* topk_idx, const float* topk_w, uint16_t* out, void* ws,
                           size_t ws_bytes, moe_stream_t stream) {
  moe_status r = check(cfg);
  if (r != MOE_OK) return r;
  if (cfg->T == 0) return MOE_OK;
  FewArgs a = {};
  if ((r = prepare_experts(cfg, w, x, topk_idx, topk_w, out, ws, ws_bytes, a)) != MOE_OK) return r;
  return launch_few(a, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_check_few_waits(const moe_config* cfg, const moe_weights* w, const uint16_t* x,
                               const int32_t* topk_idx, uint16_t* out, void* ws, size_t ws_bytes, int32_t which,
                               int64_t limit_ns, moe_stream_t stream) {
  moe_status r = check(cfg);
  if (r != MOE_OK) return r;
  if (cfg->T == 0 || which < 0 || which > 2 || limit_ns < 100000 || limit_ns > (int64_t)kFewWaitNs)
    return MOE_ERR_INVALID_ARG;
  FewArgs a = {};
  if ((r = prepare_experts(cfg, w, x, topk_idx, nullptr, out, ws, ws_bytes, a)) != MOE_OK) return r;
  a.limit_ns = (unsigned long long)limit_ns;
  a.absent = which < 2;
  a.withheld = which == 2;
  // With one CTA more to wait for than there are, a count from 0 leaves the first barrier short by one; from 1 it is
  // the second one's turn. (The count's low byte comes first in memory.)
  const cudaStream_t st = (cudaStream_t)stream;
  const bool ok = cudaMemsetAsync(&a.meta->arrived, 0, 8, st) == cudaSuccess &&
                  (which != 1 || cudaMemsetAsync(&a.meta->arrived, 1, 1, st) == cudaSuccess) &&
                  launch_few(a, st) == cudaSuccess && cudaMemsetAsync(&a.meta->arrived, 0, 8, st) == cudaSuccess;
  return ok ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
