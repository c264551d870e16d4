// Routing from given logits (softmax or sigmoid scores, balance bias, expert groups, top-k,
// renormalised weights) and the gradient of its weights and scores to the logits.
//
// One warp per token. Lane l holds the logits of experts [l * NV, (l + 1) * NV), NV the power of two
// with 32 * NV >= E, so the lowest lane that holds a value also holds its lowest index.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "internal.h"

namespace moe {
namespace {

constexpr int kWarps = 8;  // tokens per CTA
constexpr unsigned kFull = 0xffffffffu;

// Order-preserving key of a rank: larger float, larger key. 0 is below every key (an expert that
// cannot be chosen), kMaskedKey is the key of -infinity (a switched-off expert).
constexpr uint32_t kMaskedKey = 0x007fffffu;
__device__ __forceinline__ uint32_t rank_key(float r) {
  const uint32_t u = __float_as_uint(r + 0.0f);  // -0 becomes +0: the two compare equal
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_rank(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// a + b as an unevaluated pair (hi, lo) added to (hi, lo): the softmax denominator in about 46
// bits. Rounded once to fp32 it does not depend on the order of the sum, so neither does a choice
// that adds the bias to the probabilities (fp64 adds run at a small fraction of this rate here).
__device__ __forceinline__ void pair_add(float& hi, float& lo, float b_hi, float b_lo) {
  const float s = __fadd_rn(hi, b_hi);
  const float bb = __fsub_rn(s, hi);
  const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, bb)), __fsub_rn(b_hi, bb));
  const float t = __fadd_rn(err, __fadd_rn(lo, b_lo));
  hi = __fadd_rn(s, t);
  lo = __fsub_rn(t, __fsub_rn(hi, s));
}

struct GateArgs {
  const void* logits;
  const float* bias;
  int32_t* idx;
  float* w;
  float* scores;
  long long ld;
  int T, E, k, G, Gk;
  bool top2, renorm;
  float scale;
};

// Softmax of the warp's logits (experts beyond E are -infinity): s and nothing else. An all
// switched-off row has every score 0.
template <int NV>
__device__ __forceinline__ void softmax_scores(const float (&l)[NV], float (&s)[NV]) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) m = fmaxf(m, l[i]);
  m = warp_max(m);
  const float top = m == -INFINITY ? 0.0f : m;
  float hi = 0.0f, lo = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    s[i] = expf(l[i] - top);
    pair_add(hi, lo, s[i], 0.0f);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1)
    pair_add(hi, lo, __shfl_xor_sync(kFull, hi, o), __shfl_xor_sync(kFull, lo, o));
  // lanes may differ in the last place of lo only; lane 0's pair is everyone's
  const float total = __shfl_sync(kFull, __fadd_rn(hi, lo), 0);
#pragma unroll
  for (int i = 0; i < NV; ++i) s[i] = s[i] / (total == 0.0f ? 1.0f : total);
}

template <int NV, typename LT, bool SIGMOID>
__global__ void __launch_bounds__(32 * kWarps) gate_kernel(const GateArgs a) {
  extern __shared__ uint32_t group_smem[];  // [kWarps][E] keys, only with groups
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long t = (long long)blockIdx.x * kWarps + warp;
  if (t >= a.T) return;
  const LT* row = static_cast<const LT*>(a.logits) + t * a.ld;
  const int e0 = lane * NV;
  float l[NV], s[NV];
  bool bad = false;  // a NaN (softmax: or +infinity) in the row
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    l[i] = e0 + i < a.E ? load_logit(row + e0 + i) : -INFINITY;
    bad |= l[i] != l[i] || (!SIGMOID && l[i] == INFINITY);
  }
  bad = __any_sync(kFull, bad);
  const bool need_scores = SIGMOID || a.bias != nullptr || a.scores != nullptr || !a.renorm;
  if (need_scores) {
    if (SIGMOID) {
#pragma unroll
      for (int i = 0; i < NV; ++i) s[i] = sigmoid(l[i]);
    } else {
      softmax_scores<NV>(l, s);
    }
    if (a.scores != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (e0 + i < a.E) a.scores[t * a.E + e0 + i] = s[i];
    }
  }
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float r = l[i];
    if (a.bias != nullptr)
      r = e0 + i < a.E ? s[i] + a.bias[e0 + i] : -INFINITY;
    else if (SIGMOID)
      r = s[i];
    // r is NaN where the logit, the softmax or the bias is
    key[i] = e0 + i >= a.E ? 0u : (r != r || l[i] != l[i] || l[i] == -INFINITY) ? kMaskedKey
                                                                               : rank_key(r);
  }
  if (a.G > 0) {
    uint32_t* mine = group_smem + warp * a.E;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e0 + i < a.E) mine[e0 + i] = key[i];
    __syncwarp();
    const int size = a.E / a.G;
    uint32_t gk[2];  // ranks of groups lane and lane + 32
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int g = lane + 32 * h;
      gk[h] = 0u;
      if (g < a.G) {
        uint32_t b1 = 0u, b2 = 0u;
        for (int i = 0; i < size; ++i) {
          const uint32_t v = mine[g * size + i];
          b2 = max(b2, min(b1, v));
          b1 = max(b1, v);
        }
        gk[h] = a.top2 && b2 > kMaskedKey ? rank_key(key_rank(b1) + key_rank(b2)) : b1;
      }
    }
    // a group is kept when fewer than Gk groups precede it
    int before[2] = {0, 0};
    for (int g = 0; g < a.G; ++g) {
      const uint32_t v = __shfl_sync(kFull, g < 32 ? gk[0] : gk[1], g & 31);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        before[h] += v > gk[h] || (v == gk[h] && g < lane + 32 * h);
    }
    const unsigned keep0 = __ballot_sync(kFull, lane < a.G && before[0] < a.Gk);
    const unsigned keep1 = __ballot_sync(kFull, lane + 32 < a.G && before[1] < a.Gk);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int g = (e0 + i) / size;
      if (e0 + i < a.E && !(((g < 32 ? keep0 : keep1) >> (g & 31)) & 1u)) key[i] = 0u;
    }
  }
  // top-k: the warp's largest key, lowest lane and lowest slot first
  int my_idx = 0;  // lane j: the j-th choice
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(kFull, best);
    const int owner = __ffs(__ballot_sync(kFull, best == top)) - 1;
    int slot = 0;
#pragma unroll
    for (int i = NV - 1; i >= 0; --i)
      if (key[i] == top) slot = i;
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i == slot) key[i] = 0u;
    }
    const int e = __shfl_sync(kFull, e0 + slot, owner);
    if (lane == j) my_idx = e;
  }
  // weights: lane j < k recomputes its choice's score from the logit
  const bool on = lane < a.k;
  float w = 0.0f;
  if (SIGMOID) {
    w = on ? sigmoid(load_logit(row + my_idx)) : 0.0f;
  } else if (a.renorm) {  // softmax over the chosen logits: the same quotient without underflow
    const float sel = on ? load_logit(row + my_idx) : -INFINITY;
    const float m = warp_max(sel);
    w = on ? expf(sel - (m == -INFINITY ? 0.0f : m)) : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float v = __shfl_sync(kFull, s[i], my_idx / NV);
      if (my_idx % NV == i) w = v;
    }
    w = on ? w : 0.0f;
  }
  if (a.renorm) {
    const float total = warp_sum(w);
    w = total == 0.0f ? 0.0f : w / total;
  }
  if (on) {
    a.idx[t * a.k + lane] = my_idx;
    a.w[t * a.k + lane] = bad ? NAN : a.scale * w;
  }
}

struct GateGradArgs {
  const void* logits;
  const int32_t* idx;
  const float* d_w;
  const float* d_scores;
  void* d_logits;
  long long ld;
  int T, E, k;
  bool renorm;
  float scale;
};

// Gradient to the logits. With c = scale, dw the gradient of the weights and ds that of the scores:
//   softmax, renormalised: u = softmax over the chosen logits, dl_j = c u_j (dw_j - sum_i u_i dw_i)
//   sigmoid, renormalised: D = sum of the chosen s, ds_j += c (dw_j - sum_i dw_i s_i / D) / D
//   not renormalised: ds_j += c dw_j
//   then softmax: dl += s (ds - sum_e s_e ds_e);  sigmoid: dl = ds s (1 - s).
template <int NV, typename LT, bool SIGMOID>
__global__ void __launch_bounds__(32 * kWarps) gate_grad_kernel(const GateGradArgs a) {
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long t = (long long)blockIdx.x * kWarps + warp;
  if (t >= a.T) return;
  const LT* row = static_cast<const LT*>(a.logits) + t * a.ld;
  LT* out = static_cast<LT*>(a.d_logits) + t * a.E;
  const int e0 = lane * NV;
  // the chosen experts: lane j < k
  int my_idx = lane < a.k ? a.idx[t * a.k + lane] : -1;
  if (my_idx >= a.E) my_idx = -1;
  const bool on = my_idx >= 0;
  const float dw = on && a.d_w != nullptr ? a.scale * a.d_w[t * a.k + lane] : 0.0f;
  const float sel = on ? load_logit(row + my_idx) : -INFINITY;
  float g = dw;  // gradient of the choice: to its score, or (softmax, renormalised) to its logit
  if (a.renorm) {
    if (SIGMOID) {
      const float sj = on ? sigmoid(sel) : 0.0f;
      const float total = warp_sum(sj);
      const float dot = warp_sum(dw * sj);
      g = total == 0.0f ? 0.0f : (dw - dot / total) / total;
    } else {
      const float m = warp_max(sel);
      float u = on ? expf(sel - (m == -INFINITY ? 0.0f : m)) : 0.0f;
      const float total = warp_sum(u);
      u = total == 0.0f ? 0.0f : u / total;
      g = u * (dw - warp_sum(u * dw));
    }
  }
  const bool to_logit = !SIGMOID && a.renorm;  // g is already a logit's gradient
  float ds[NV], gl[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    ds[i] = a.d_scores != nullptr && e0 + i < a.E ? a.d_scores[t * a.E + e0 + i] : 0.0f;
    gl[i] = 0.0f;
  }
  for (int j = 0; j < a.k; ++j) {
    const int e = __shfl_sync(kFull, my_idx, j);
    const float v = __shfl_sync(kFull, g, j);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e == e0 + i) (to_logit ? gl[i] : ds[i]) += v;
  }
  if (SIGMOID) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (e0 + i < a.E) {
        // s (1 - s) = x / (1 + x)^2 with x = exp(-|l|): no cancellation at either end
        const float x = expf(-fabsf(load_logit(row + e0 + i)));
        gl[i] = ds[i] * (x / ((1.0f + x) * (1.0f + x)));
      }
    }
  } else if (a.d_scores != nullptr || !a.renorm) {
    float l[NV], s[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = e0 + i < a.E ? load_logit(row + e0 + i) : -INFINITY;
    softmax_scores<NV>(l, s);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) dot += s[i] * ds[i];
    dot = warp_sum(dot);
#pragma unroll
    for (int i = 0; i < NV; ++i) gl[i] += s[i] * (ds[i] - dot);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (e0 + i < a.E) store_logit(out + e0 + i, gl[i]);
}

int lane_values(int E) {
  int nv = 1;
  while (32 * nv < E) nv *= 2;
  return nv;
}

template <int NV, typename LT, bool SIGMOID>
cudaError_t gate_one(const GateArgs& a, cudaStream_t st) {
  const size_t smem = a.G > 0 ? sizeof(uint32_t) * kWarps * a.E : 0;
  return launch_k(gate_kernel<NV, LT, SIGMOID>, dim3((a.T + kWarps - 1) / kWarps),
                  dim3(32 * kWarps), smem, st, a);
}
template <int NV, typename LT, bool SIGMOID>
cudaError_t gate_grad_one(const GateGradArgs& a, cudaStream_t st) {
  return launch_k(gate_grad_kernel<NV, LT, SIGMOID>, dim3((a.T + kWarps - 1) / kWarps),
                  dim3(32 * kWarps), 0, st, a);
}

#define MOE_BY_NV(fn, LT, SIG, args, E, st)                                                     \
  switch (lane_values(E)) {                                                                     \
    case 1: return fn<1, LT, SIG>(args, st);                                                    \
    case 2: return fn<2, LT, SIG>(args, st);                                                    \
    case 4: return fn<4, LT, SIG>(args, st);                                                    \
    default: return fn<8, LT, SIG>(args, st);                                                   \
  }

moe_status check_gate(const moe_gate_config* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->T < 0 || c->E < 1 || c->top_k < 1) return MOE_ERR_INVALID_ARG;
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_DTYPE_F32 && c->dtype != MOE_DTYPE_BF16 && c->dtype != MOE_DTYPE_F16)
    return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->scale)) return MOE_ERR_INVALID_ARG;
  if ((c->renormalize & ~1) != 0 || (c->group_top2 & ~1) != 0) return MOE_ERR_INVALID_ARG;
  if (c->ld != 0 && c->ld < c->E) return MOE_ERR_INVALID_ARG;
  if (c->E > 256 || c->top_k > 8 || c->top_k > c->E) return MOE_ERR_UNSUPPORTED;
  if (c->dtype == MOE_DTYPE_F16) return MOE_ERR_UNSUPPORTED;
  if (c->n_groups < 0) return MOE_ERR_INVALID_ARG;
  if (c->n_groups > 0) {
    if (c->n_groups > 64 || c->E % c->n_groups != 0) return MOE_ERR_UNSUPPORTED;
    if (c->topk_groups < 1 || c->topk_groups > c->n_groups) return MOE_ERR_INVALID_ARG;
    if ((long long)c->top_k > (long long)c->topk_groups * (c->E / c->n_groups))
      return MOE_ERR_INVALID_ARG;
  }
  if ((long long)c->T * c->top_k >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_route_logits(const moe_gate_config* cfg, const void* logits,
                            const float* expert_bias, int32_t* topk_idx, float* topk_w,
                            float* scores, moe_stream_t stream) {
  const moe_status r = check_gate(cfg);
  if (r != MOE_OK) return r;
  if (cfg->T == 0) return MOE_OK;
  const bool bf16 = cfg->dtype == MOE_DTYPE_BF16;
  if (!logits || !topk_idx || !topk_w || !aligned(logits, bf16 ? 2 : 4)) return MOE_ERR_INVALID_ARG;
  if (!aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(expert_bias, 4) ||
      !aligned(scores, 4))
    return MOE_ERR_INVALID_ARG;
  GateArgs a;
  a.logits = logits;
  a.bias = expert_bias;
  a.idx = topk_idx;
  a.w = topk_w;
  a.scores = scores;
  a.ld = cfg->ld != 0 ? cfg->ld : cfg->E;
  a.T = cfg->T;
  a.E = cfg->E;
  a.k = cfg->top_k;
  a.G = cfg->n_groups;
  a.Gk = cfg->topk_groups;
  a.top2 = cfg->group_top2 != 0;
  a.renorm = cfg->renormalize != 0;
  a.scale = cfg->scale;
  const bool sig = cfg->score == MOE_SCORE_SIGMOID;
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = [&]() -> cudaError_t {
    if (bf16 && sig) MOE_BY_NV(gate_one, __nv_bfloat16, true, a, a.E, st)
    if (bf16) MOE_BY_NV(gate_one, __nv_bfloat16, false, a, a.E, st)
    if (sig) MOE_BY_NV(gate_one, float, true, a, a.E, st)
    MOE_BY_NV(gate_one, float, false, a, a.E, st)
  }();
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_route_logits_backward(const moe_gate_config* cfg, const void* logits,
                                     const int32_t* topk_idx, const float* d_topk_w,
                                     const float* d_scores, void* d_logits, moe_stream_t stream) {
  const moe_status r = check_gate(cfg);
  if (r != MOE_OK) return r;
  if (cfg->T == 0) return MOE_OK;
  const bool bf16 = cfg->dtype == MOE_DTYPE_BF16;
  if (!logits || !topk_idx || !d_logits || (!d_topk_w && !d_scores)) return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, bf16 ? 2 : 4) || !aligned(d_logits, bf16 ? 2 : 4) ||
      !aligned(topk_idx, 4) || !aligned(d_topk_w, 4) || !aligned(d_scores, 4))
    return MOE_ERR_INVALID_ARG;
  GateGradArgs a;
  a.logits = logits;
  a.idx = topk_idx;
  a.d_w = d_topk_w;
  a.d_scores = d_scores;
  a.d_logits = d_logits;
  a.ld = cfg->ld != 0 ? cfg->ld : cfg->E;
  a.T = cfg->T;
  a.E = cfg->E;
  a.k = cfg->top_k;
  a.renorm = cfg->renormalize != 0;
  a.scale = cfg->scale;
  const bool sig = cfg->score == MOE_SCORE_SIGMOID;
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = [&]() -> cudaError_t {
    if (bf16 && sig) MOE_BY_NV(gate_grad_one, __nv_bfloat16, true, a, a.E, st)
    if (bf16) MOE_BY_NV(gate_grad_one, __nv_bfloat16, false, a, a.E, st)
    if (sig) MOE_BY_NV(gate_grad_one, float, true, a, a.E, st)
    MOE_BY_NV(gate_grad_one, float, false, a, a.E, st)
  }();
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
