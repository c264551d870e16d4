// Routing from given logits (softmax or sigmoid scores, balance bias, expert groups, top-k,
// renormalised weights) and the gradient of its weights and scores to the logits.
//
// Forward: one warp per token and persistent warps, so the bias stays in registers and the next row is
// on its way. Lane l holds experts [l * NV, (l + 1) * NV), NV the power of two with 32 * NV >= E. Bound by
// instructions, not bytes: a row of 256 fp32 logits is 1 KB, 0.15 us of one SM's share of HBM, and its
// 256 sigmoids alone are about 110 warp instructions. So the choice looks at few experts one by one: the
// k-th largest of the lanes' maxima is a bound that at least k experts reach and few others do (about
// 10 of 256 for k = 8); those, one per lane, are ranked against each other, four per shared load. Weights
// are found for four tokens at once, eight lanes each.
// 65536 rows of 256 (sigmoid, bias, 8 groups, top-8) 43 us, 590 warp instructions a token and three
// quarters of the issue slots; with k rounds of a warp maximum over all experts, and one token's weights
// at a time, 80.
// Backward: one warp per token, or per four tokens where only the chosen experts have a gradient: zeroed
// rows in 16-byte pieces, then the chosen experts' values. Bound by HBM, whose reads
// come 64 bytes at a time: 65536 rows of 256 with eight chosen 16.6 us, 67 MB written and about 30 read. With a
// gradient of every score 40 us (sigmoid) and 44 (softmax), 205 MB: one row a warp, and nothing in flight for
// the next.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "internal.h"

namespace moe {
namespace {

constexpr int kWarps = 8;      // tokens at a time per CTA
constexpr int kCtasPerSm = 4;  // resident CTAs of the forward kernel (its registers)
constexpr unsigned kFull = 0xffffffffu;

// The smallest (largest) of the values, NaN if one is NaN, three at a time.
template <int N>
__device__ __forceinline__ float least_or_nan(const float (&v)[N]) {
  float m = v[0];
  if (N == 2) asm("min.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(v[N - 1]));
#pragma unroll
  for (int i = 1; i < N - 1; i += 2)
    asm("min.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(v[i]), "f"(v[i + 1]));
  if (N > 2 && N % 2 == 0) asm("min.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(v[N - 1]));
  return m;
}
template <int N>
__device__ __forceinline__ float most_or_nan(const float (&v)[N]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(v[i]));
  return m;
}
__device__ __forceinline__ float warp_reduce_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
// One logit of a row that is not read otherwise: 64 bytes of it from HBM and not the 128 that come by
// default (65536 rows of 256, eight chosen: 49 MB read, 19.4 against 17.4 us for the whole gradient).
__device__ __forceinline__ float load_single(const float* p) {
  float v;
  asm volatile("ld.global.L2::64B.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float load_single(const __nv_bfloat16* p) {
  uint16_t v;
  asm volatile("ld.global.L2::64B.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return __uint_as_float((uint32_t)v << 16);
}
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

// The same value for -80 <= l, without the division's branch: one Newton step from a reciprocal within
// an ulp is the correctly rounded one (Markstein 1990) unless the divisor's mantissa is all ones.
__device__ __forceinline__ float sigmoid_fast(float l) {
  const float d = 1.0f + expf(-l);
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d));
  return fmaf(fmaf(-d, y, 1.0f), y, y);
}

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
  bool vec, vec_scores;  // rows of logits / scores are in 16-byte pieces
  int lanes;             // lanes per group where a group is a power of two of whole lanes, else 0
  float scale;
};

// Softmax of the warp's logits (experts beyond E are -infinity). top and total: the row's exp offset and
// denominator (1 for an all switched-off row, whose scores are 0).
template <int NV>
__device__ __forceinline__ void softmax_scores(const float (&l)[NV], float (&s)[NV], float& top,
                                               float& total) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) m = fmaxf(m, l[i]);
  m = warp_max(m);
  top = m == -INFINITY ? 0.0f : m;
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
  total = __shfl_sync(kFull, __fadd_rn(hi, lo), 0);
  total = total == 0.0f ? 1.0f : total;
  // the quotient by one correction of e * (1 / total) (Markstein 1990): correctly rounded for normal
  // quotients, without a branch per element
  const float inv = 1.0f / total;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float q = s[i] * inv;
    s[i] = fmaf(fmaf(-q, total, s[i]), inv, q);
  }
}

// NV consecutive elements from p; vec: p is aligned to min(16, their bytes) and all are there.
template <int NV>
__device__ __forceinline__ void load_run(const float* p, float (&v)[NV]) {
  if constexpr (NV >= 4) {
#pragma unroll
    for (int i = 0; i < NV; i += 4)
      *reinterpret_cast<float4*>(v + i) = *reinterpret_cast<const float4*>(p + i);
  } else if constexpr (NV == 2) {
    *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(p);
  } else {
    v[0] = p[0];
  }
}
template <int NV>
__device__ __forceinline__ void load_run(const __nv_bfloat16* p, float (&v)[NV]) {
  if constexpr (NV == 1) {
    v[0] = __bfloat162float(p[0]);
  } else {
    uint32_t w[NV / 2];
    if constexpr (NV == 8)
      *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
    else if constexpr (NV == 4)
      *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
    else
      w[0] = *reinterpret_cast<const uint32_t*>(p);
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
// This lane's logits of a row; `fill` past E.
template <int NV, typename LT>
__device__ __forceinline__ void load_row(const LT* row, int e0, int E, bool vec, float fill,
                                         float (&l)[NV]) {
  if (vec && e0 + NV <= E) {
    load_run<NV>(row + e0, l);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = e0 + i < E ? load_logit(row + e0 + i) : fill;
  }
}

// The two largest of r[FIRST ... FIRST + N), the second -infinity where there is one only.
template <int FIRST, int N, int NV>
__device__ __forceinline__ void two_largest(const float (&r)[NV], float& b1, float& b2) {
  if constexpr (N == 1) {
    b1 = r[FIRST];
    b2 = -INFINITY;
  } else {
    float h1, h2, l1, l2;
    two_largest<FIRST, N / 2>(r, h1, l1);
    two_largest<FIRST + N / 2, N / 2>(r, h2, l2);
    b1 = fmaxf(h1, h2);
    b2 = N == 2 ? fminf(h1, h2) : fmaxf(fminf(h1, h2), fmaxf(l1, l2));
  }
}

// This lane's ranks to its place in the warp's row.
template <int NV>
__device__ __forceinline__ void store_ranks(float* row, int lane, const float (&r)[NV]) {
  if constexpr (NV >= 4) {
#pragma unroll
    for (int i = 0; i < NV; i += 4)
      *reinterpret_cast<float4*>(row + lane * NV + i) =
          make_float4(r[i], r[i + 1], r[i + 2], r[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) row[lane * NV + i] = r[i];
  }
}

// Groups of any size: lane g ranks groups g and g + 32 from the warp's row of ranks. Sets the bits of
// `gone` whose experts' groups are not kept.
template <int NV>
__device__ __forceinline__ void drop_groups(const GateArgs& a, const float* mine, int e0, int lane,
                                            uint32_t& gone) {
  const int size = a.E / a.G;
  float best[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int g = lane + 32 * h;
    best[h] = -INFINITY;
    if (g < a.G) {
      float b1 = -INFINITY, b2 = -INFINITY;
      for (int i = 0; i < size; ++i) {
        const float v = mine[g * size + i];
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
      }
      best[h] = a.top2 && b2 > -INFINITY ? b1 + b2 : b1;
    }
  }
  int before[2] = {0, 0};
  for (int g = 0; g < a.G; ++g) {
    const float v = __shfl_sync(kFull, g < 32 ? best[0] : best[1], g & 31);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      before[h] += v > best[h] || (v == best[h] && g < lane + 32 * h);
  }
  const unsigned keep0 = __ballot_sync(kFull, lane < a.G && before[0] < a.Gk);
  const unsigned keep1 = __ballot_sync(kFull, lane + 32 < a.G && before[1] < a.Gk);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int g = min(e0 + i, a.E - 1) / size;
    if (!(((g < 32 ? keep0 : keep1) >> (g & 31)) & 1u)) gone |= 1u << i;
  }
}

template <int NV, typename LT, bool SIGMOID>
__global__ void __launch_bounds__(32 * kWarps, kCtasPerSm) gate_kernel(const GateArgs a) {
  __shared__ __align__(16) float ranks[kWarps][32 * NV];   // a row's ranks
  __shared__ __align__(16) float picked_rank[kWarps][32];  // its candidates' ranks
  __shared__ int picked[kWarps][32];                       // and experts
  __shared__ int chosen[kWarps][32];                       // the experts of four rows, eight each
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned below = (1u << lane) - 1u;  // lanes before this one
  const int e0 = lane * NV;
  const int group = a.lanes > 0 ? lane / a.lanes : 0;
  const LT* logits = static_cast<const LT*>(a.logits);
  const long long step = (long long)gridDim.x * kWarps;
  // sigmoids of -infinity take a detour: past E a 0 stands, whose rank is taken back
  constexpr float kFill = SIGMOID ? 0.0f : -INFINITY;
  float bias[NV];
  uint32_t past = 0u;  // slots past E
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    bias[i] = a.bias != nullptr && e0 + i < a.E ? a.bias[e0 + i] : 0.0f;
    past |= e0 + i >= a.E ? 1u << i : 0u;
  }
  const bool need_scores = SIGMOID || a.bias != nullptr || a.scores != nullptr;

  // Weights of up to four rows at once, eight lanes each: the chosen experts' scores once more from
  // their logits. q < rows: row t0 + q step, the q-th bit of bad: it holds a NaN (softmax: or +infinity).
  auto weigh = [&](long long t0, int rows, unsigned bad, float top, float total) {
    const int q = lane >> 3, j = lane & 7;
    const long long t = t0 + q * step;
    const bool on = q < rows && j < a.k;
    __syncwarp();
    const int e = on ? chosen[warp][lane] : 0;
    const float sel = on ? load_logit(logits + t * a.ld + e) : -INFINITY;
    float w;
    if (SIGMOID) {
      w = on ? sigmoid(sel) : 0.0f;
    } else if (a.renorm) {  // softmax over the chosen logits: the same quotient without underflow
      float m = sel;
#pragma unroll
      for (int o = 4; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      w = on ? expf(sel - (m == -INFINITY ? 0.0f : m)) : 0.0f;
    } else {
      w = expf(sel - top) / total;
    }
    if (a.renorm) {
      float sum = w;
#pragma unroll
      for (int o = 4; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      w = sum == 0.0f ? 0.0f : w / sum;
    }
    if (on) {
      a.idx[t * a.k + j] = e;
      a.w[t * a.k + j] = (bad >> q) & 1u ? NAN : a.scale * w;
    }
    __syncwarp();
  };

  long long t = (long long)blockIdx.x * kWarps + warp;
  float l[NV];
  if (t < a.T) load_row<NV>(logits + t * a.ld, e0, a.E, a.vec, kFill, l);
  int held = 0;            // rows in `chosen`, and of each:
  unsigned bad_rows = 0u;  // a NaN (softmax: or +infinity) in it
  float held_top = 0.0f, held_total = 1.0f;
  for (; t < a.T; t += step) {
    float next[NV];
    if (t + step < a.T) load_row<NV>(logits + (t + step) * a.ld, e0, a.E, a.vec, kFill, next);
    const float edge = SIGMOID ? least_or_nan(l) : most_or_nan(l);
    if (__any_sync(kFull, SIGMOID ? edge != edge : !(edge < INFINITY))) bad_rows |= 1u << held;
    float s[NV], top = 0.0f, total = 1.0f;
    if (need_scores || (!SIGMOID && !a.renorm)) {
      if (SIGMOID) {
        // a logit of -infinity gives NaN, which ranks as switched off; finite ones that low take the
        // division
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = sigmoid_fast(l[i]);
        if (!(edge >= -80.0f)) {
          bool low = false;
#pragma unroll
          for (int i = 0; i < NV; ++i) low |= l[i] < -80.0f && l[i] > -INFINITY;
          if (low) {
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] = l[i] == -INFINITY ? NAN : sigmoid(l[i]);
          }
        }
      } else {
        softmax_scores<NV>(l, s, top, total);
        if (lane >> 3 == held) {
          held_top = top;
          held_total = total;
        }
      }
      if (a.scores != nullptr) {
        float* to = a.scores + t * a.E + e0;
        float o[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) o[i] = SIGMOID && l[i] == -INFINITY ? 0.0f : s[i];
        if (a.vec_scores && e0 + NV <= a.E) {
          if constexpr (NV >= 4) {
#pragma unroll
            for (int i = 0; i < NV; i += 4)
              *reinterpret_cast<float4*>(to + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) to[i] = o[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (e0 + i < a.E) to[i] = o[i];
        }
      }
    }
    // The ranks: -infinity for a switched-off expert and where the logit, the score or the bias is NaN
    // (the larger of NaN and -infinity is -infinity). Without a bias its registers are 0, which leaves a
    // sigmoid as it is; a softmax without one is ranked by its logits.
    float r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (SIGMOID)
        r[i] = fmaxf(s[i] + bias[i], -INFINITY);
      else if (a.bias != nullptr)
        r[i] = l[i] > -INFINITY ? fmaxf(s[i] + bias[i], -INFINITY) : -INFINITY;
      else
        r[i] = fmaxf(l[i], -INFINITY);
    }
    if (past != 0u) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((past >> i) & 1u) r[i] = -INFINITY;
    }
    float* const mine = ranks[warp];
    store_ranks<NV>(mine, lane, r);
    float b1, b2;  // this lane's two largest ranks
    two_largest<0, NV>(r, b1, b2);
    uint32_t gone = past;  // slots whose experts cannot be chosen
    __syncwarp();
    if (a.G > 0) {
      if (a.lanes > 0) {  // a group is `lanes` whole lanes, a power of two
        float g1 = b1;
        if (a.top2) {
          float g2 = b2;
#pragma unroll 1
          for (int o = 1; o < a.lanes; o <<= 1) {
            const float p1 = __shfl_xor_sync(kFull, g1, o), p2 = __shfl_xor_sync(kFull, g2, o);
            g2 = fmaxf(fminf(g1, p1), fmaxf(g2, p2));
            g1 = fmaxf(g1, p1);
          }
          if (g2 > -INFINITY) g1 += g2;
        } else {
#pragma unroll 1
          for (int o = 1; o < a.lanes; o <<= 1) g1 = fmaxf(g1, __shfl_xor_sync(kFull, g1, o));
        }
        // kept when fewer than Gk groups precede it; each of a group's lanes counts some
        int before = 0, g = lane & (a.lanes - 1);
#pragma unroll 1
        for (int g0 = 0; g0 < a.G; g0 += a.lanes, g += a.lanes) {
          const float v = __shfl_sync(kFull, g1, g * a.lanes);
          before += g < a.G && (v > g1 || (v == g1 && g < group));
        }
#pragma unroll 1
        for (int o = 1; o < a.lanes; o <<= 1) before += __shfl_xor_sync(kFull, before, o);
        if (before >= a.Gk) {
          b1 = -INFINITY;
          gone = 0xffffffffu;
        }
      } else {
        drop_groups<NV>(a, mine, e0, lane, gone);
        b1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) b1 = fmaxf(b1, (gone >> i) & 1u ? -INFINITY : r[i]);
      }
    }
    // the k-th largest of the lanes' maxima (equal ones count once): at least k experts reach it, or it
    // is -infinity, which all do
    float bound = -INFINITY;
    auto lower = [&] {
      bound = warp_reduce_max(b1);
      b1 = b1 == bound ? -INFINITY : b1;
    };
    switch (a.k) {  // one jump, not a test per step
      default: lower();
      case 7: lower();
      case 6: lower();
      case 5: lower();
      case 4: lower();
      case 3: lower();
      case 2: lower();
      case 1: lower();
    }
    uint32_t cand = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i) cand |= r[i] >= bound ? 1u << i : 0u;
    cand &= ~gone;
    int n = 0;  // candidates, the first 32 of which go to `picked`
    for (unsigned more = __ballot_sync(kFull, cand != 0u); more != 0u;
         more = __ballot_sync(kFull, cand != 0u)) {
      const int at = n + __popc(more & below);
      if (cand != 0u && at < 32) picked[warp][at] = e0 + __ffs(cand) - 1;
      cand &= cand - 1u;
      n += __popc(more);
    }
    __syncwarp();
    if (n <= 32) {
      // one candidate per lane, ranked against each other
      const int my_idx = lane < n ? picked[warp][lane] : 0;
      const float my_rank = lane < n ? mine[my_idx] : -INFINITY;
      picked_rank[warp][lane] = my_rank;
      __syncwarp();
      int place = 0;
      for (int j = 0; j < n; j += 4) {
        const float4 v = *reinterpret_cast<const float4*>(&picked_rank[warp][j]);
        place += (v.x > my_rank) + (v.y > my_rank) + (v.z > my_rank) + (v.w > my_rank);
      }
      // equal ranks share a place: then the lower expert goes first
      if (__popc(__reduce_or_sync(kFull, lane < n ? 1u << place : 0u)) != n) {
        place = 0;
        for (int j = 0; j < n; ++j) {
          const float v = __shfl_sync(kFull, my_rank, j);
          const int e = __shfl_sync(kFull, my_idx, j);
          place += v > my_rank || (v == my_rank && e < my_idx);
        }
      }
      if (lane < n && place < a.k) chosen[warp][held * 8 + place] = my_idx;
    } else {
      // more than 32 share the bound (many equal logits): one warp-wide maximum per choice, lowest lane
      // and slot first
      for (int j = 0; j < a.k; ++j) {
        float best = -INFINITY;
        int slot = -1;
#pragma unroll
        for (int i = NV - 1; i >= 0; --i) {
          const bool better = !((gone >> i) & 1u) && r[i] >= best;
          slot = better ? i : slot;
          best = better ? r[i] : best;
        }
        const float first = warp_reduce_max(best);
        const int owner = __ffs(__ballot_sync(kFull, slot >= 0 && best == first)) - 1;
        if (lane == owner) {
          gone |= 1u << slot;
          chosen[warp][held * 8 + j] = e0 + slot;
        }
      }
    }
    if (++held == 4) {
      weigh(t - 3 * step, 4, bad_rows, held_top, held_total);
      held = 0;
      bad_rows = 0u;
    } else {
      __syncwarp();  // picked and ranks are written again for the warp's next row
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = next[i];
  }
  if (held > 0) weigh(t - held * step, held, bad_rows, held_top, held_total);
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
  bool vec;  // rows of logits, scores and d_logits are in pieces of four experts
  float scale;
};

// Gradient to the logits. With c = scale, dw the gradient of the weights and ds that of the scores:
//   softmax, renormalised: u = softmax over the chosen logits, dl_j = c u_j (dw_j - sum_i u_i dw_i)
//   sigmoid, renormalised: u = s / sum of the chosen s, dl_j = c u_j (dw_j - sum_i u_i dw_i) (1 - s_j); the
//     gradient to s_j itself, with the sum as a divisor, would be past fp32's range where the scores are tiny
//   not renormalised: ds_j += c dw_j
//   then softmax: dl += s (ds - sum_e s_e ds_e);  sigmoid: dl = ds s (1 - s).
__device__ __forceinline__ float lanes_sum(float v, int W) {
#pragma unroll
  for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return W > 8 ? __shfl_sync(kFull, v, 0) : v;  // the other lanes' values are 0
}
__device__ __forceinline__ float lanes_max(float v, int W) {
#pragma unroll
  for (int o = 4; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return W > 8 ? __shfl_sync(kFull, v, 0) : v;
}

// g of a token's chosen experts, one per lane (at most eight) of a row of W = 8 or 32 lanes: the
// gradient to its logit. Not renormalised, and where other experts have a gradient too (!TO_LOGIT): to its
// score.
template <bool SIGMOID, bool TO_LOGIT, int W>
__device__ __forceinline__ float chosen_gradient(const GateGradArgs& a, bool on, float sel,
                                                 float dw) {
  if (!a.renorm) {
    if (!SIGMOID || !TO_LOGIT) return dw;
    // s (1 - s) = x / (1 + x)^2 with x = exp(-|l|): no cancellation at either end
    const float x = expf(-fabsf(sel));
    return on ? dw * (x / ((1.0f + x) * (1.0f + x))) : 0.0f;
  }
  float u, rest = 1.0f;  // rest: 1 - s without cancellation
  if (SIGMOID) {
    const float e = expf(-sel), sj = 1.0f / (1.0f + e);
    u = on ? sj : 0.0f;
    rest = sel < 0.0f ? 1.0f - sj : e * sj;
  } else {
    const float m = lanes_max(sel, W);
    u = on ? expf(sel - (m == -INFINITY ? 0.0f : m)) : 0.0f;
  }
  const float total = lanes_sum(u, W), dot = lanes_sum(u * dw, W);
  return total == 0.0f ? 0.0f : u / total * (dw - dot / total) * rest;
}

// Adds the chosen experts' values to a zeroed row of E floats in shared memory (an index that comes twice
// adds twice).
template <int NV>
__device__ __forceinline__ void scatter_row(float* mine, int lane, int my_idx, float g) {
#pragma unroll
  for (int i = 0; i < NV; i += 4)
    if (NV >= 4)
      *reinterpret_cast<float4*>(mine + i / 4 * 128 + lane * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
  if (NV < 4) {
#pragma unroll
    for (int i = 0; i < NV; ++i) mine[i * 32 + lane] = 0.0f;
  }
  __syncwarp();
  if (my_idx >= 0) atomicAdd(mine + my_idx, g);
  __syncwarp();
}

__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float a, float b, float c, float d) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                            *reinterpret_cast<const uint32_t*>(&hi));
}

// Only the chosen experts have a gradient (no d_scores, and not a softmax without renormalisation).
// Eight lanes per token, four consecutive tokens per warp, whose rows of d_logits are one run of 4 E
// elements: zeros in 16-byte pieces, then the chosen experts' values on top (the warp's barrier orders
// the two; put together in shared memory first, 65536 rows of 256 took 4 us more).
template <int NV, typename LT, bool SIGMOID>
__global__ void __launch_bounds__(32 * kWarps) gate_grad_chosen_kernel(const GateGradArgs a) {
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long t0 = ((long long)blockIdx.x * kWarps + warp) * 4;
  if (t0 >= a.T) return;
  const int j = lane & 7, n = (int)min(4LL, a.T - t0);
  const long long t = t0 + (lane >> 3);
  int my_idx = j < a.k && t < a.T ? a.idx[t * a.k + j] : -1;
  if (my_idx >= a.E) my_idx = -1;
  const bool on = my_idx >= 0;
  const float dw = on ? a.scale * a.d_w[t * a.k + j] : 0.0f;
  const float sel =
      on ? load_single(static_cast<const LT*>(a.logits) + t * a.ld + my_idx) : -INFINITY;
  LT* out = static_cast<LT*>(a.d_logits) + t0 * a.E;
  if (a.vec) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * 32 + lane) * 4;
      if (e < n * a.E) store4(out + e, 0.0f, 0.0f, 0.0f, 0.0f);
    }
  } else {
    for (int e = lane; e < n * a.E; e += 32) store_logit(out + e, 0.0f);
  }
  float g = chosen_gradient<SIGMOID, true, 8>(a, on, sel, dw);
  // the choices of a token are different experts; should one come twice all the same, it adds twice
  const int place = on ? (lane >> 3) * a.E + my_idx : -1 - lane;
  const unsigned same = __match_any_sync(kFull, place);
  if (__any_sync(kFull, (same & (same - 1u)) != 0u)) {
    float sum = 0.0f;
    for (int l = 0; l < 32; ++l) {
      const float v = __shfl_sync(kFull, g, l);
      if ((same >> l) & 1u) sum += v;
    }
    g = sum;
  }
  __syncwarp();
  if (on) store_logit(out + place, g);
}

// Every expert has a gradient. Lane l holds experts i / 4 * 128 + 4 l + i % 4 (NV >= 4), so that rows
// move in whole lines.
template <int NV, typename LT, bool SIGMOID>
__global__ void __launch_bounds__(32 * kWarps) gate_grad_kernel(const GateGradArgs a) {
  __shared__ __align__(16) float rows[kWarps][32 * NV];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long t = (long long)blockIdx.x * kWarps + warp;
  if (t >= a.T) return;
  const LT* row = static_cast<const LT*>(a.logits) + t * a.ld;
  LT* out = static_cast<LT*>(a.d_logits) + t * a.E;
  const float* dsr = a.d_scores != nullptr ? a.d_scores + t * a.E : nullptr;
  auto expert = [&](int i) { return NV >= 4 ? i / 4 * 128 + lane * 4 + i % 4 : i * 32 + lane; };
  float l[NV], ds[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    ds[i] = 0.0f;
    l[i] = -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = expert(i);
    if (NV >= 4 && a.vec) {
      if (i % 4 == 0 && e < a.E) {
        load_run<4>(row + e, *reinterpret_cast<float(*)[4]>(l + i));
        if (dsr != nullptr) load_run<4>(dsr + e, *reinterpret_cast<float(*)[4]>(ds + i));
      }
    } else if (e < a.E) {
      l[i] = load_logit(row + e);
      if (dsr != nullptr) ds[i] = dsr[e];
    }
  }
  int my_idx = lane < a.k && a.d_w != nullptr ? a.idx[t * a.k + lane] : -1;
  if (my_idx >= a.E) my_idx = -1;
  const bool on = my_idx >= 0;
  const float dw = on ? a.scale * a.d_w[t * a.k + lane] : 0.0f;
  const float sel = on ? load_logit(row + my_idx) : -INFINITY;
  const float g = chosen_gradient<SIGMOID, false, 32>(a, on, sel, dw);
  float* mine = rows[warp];
  scatter_row<NV>(mine, lane, my_idx, g);
  float gl[NV];
  // renormalised, the chosen values are logits' gradients already; else scores'
  if (SIGMOID) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float x = expf(-fabsf(l[i]));
      const float slope = x / ((1.0f + x) * (1.0f + x)), g_i = mine[expert(i)];
      gl[i] = a.renorm ? ds[i] * slope + g_i : (ds[i] + g_i) * slope;
    }
  } else {
    float s[NV], top, total, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      gl[i] = mine[expert(i)];
      if (!a.renorm) {
        ds[i] += gl[i];
        gl[i] = 0.0f;
      }
    }
    softmax_scores<NV>(l, s, top, total);
#pragma unroll
    for (int i = 0; i < NV; ++i) dot += s[i] * ds[i];
    dot = warp_sum(dot);
#pragma unroll
    for (int i = 0; i < NV; ++i) gl[i] += s[i] * (ds[i] - dot);
  }
  if (NV >= 4 && a.vec) {
#pragma unroll
    for (int i = 0; i < NV; i += 4)
      if (expert(i) < a.E)
        store4(out + expert(i), gl[i], gl[(i + 1) % NV], gl[(i + 2) % NV], gl[(i + 3) % NV]);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (expert(i) < a.E) store_logit(out + expert(i), gl[i]);
  }
}

int lane_values(int E) {
  int nv = 1;
  while (32 * nv < E) nv *= 2;
  return nv;
}

template <int NV, typename LT, bool SIGMOID>
cudaError_t gate_one(const GateArgs& a, cudaStream_t st) {
  // persistent: at most as many CTAs as the GPU holds at once
  const long long ctas = ((long long)a.T + kWarps - 1) / kWarps;
  return launch_k(gate_kernel<NV, LT, SIGMOID>,
                  dim3((unsigned)std::min(ctas, (long long)num_sms() * kCtasPerSm)),
                  dim3(32 * kWarps), 0, st, a);
}
template <int NV, typename LT, bool SIGMOID>
cudaError_t gate_grad_one(const GateGradArgs& a, cudaStream_t st) {
  const bool chosen = a.d_scores == nullptr && (SIGMOID || a.renorm);
  if (chosen)
    return launch_k(gate_grad_chosen_kernel<NV, LT, SIGMOID>,
                    dim3((unsigned)(((long long)a.T + 4 * kWarps - 1) / (4 * kWarps))),
                    dim3(32 * kWarps), 0, st, a);
  return launch_k(gate_grad_kernel<NV, LT, SIGMOID>,
                  dim3((unsigned)(((long long)a.T + kWarps - 1) / kWarps)), dim3(32 * kWarps), 0, st, a);
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
  a.vec = aligned(logits, 16) && a.ld * (bf16 ? 2 : 4) % 16 == 0;
  a.vec_scores = aligned(scores, 16) && a.E % 4 == 0;
  const int nv = lane_values(a.E), size = a.G > 0 ? a.E / a.G : 0;
  const int lanes = size % nv == 0 ? size / nv : 0;
  a.lanes = (lanes & (lanes - 1)) == 0 ? lanes : 0;
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
  const int piece = bf16 ? 8 : 16;  // four logits
  a.vec = a.E % 4 == 0 && aligned(logits, piece) && a.ld % 4 == 0 && aligned(d_logits, piece) &&
          aligned(d_scores, 16);
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
