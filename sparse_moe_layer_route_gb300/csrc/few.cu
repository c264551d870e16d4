// The whole MoE layer for up to 16 tokens in one kernel: router, choice, gate/up, SwiGLU, down, combine.
//
// With few tokens the layer is the reading of the chosen experts' weights, each once: 6 d f bytes an
// expert, no more than one token for most of them. One persistent CTA per SM (cooperative launch) goes
// through four parts, with a grid barrier after the first and the third:
//   router   one expert per CTA: logits of all tokens. Eight products at a time are summed in fp32, the
//            sums of eight in an unevaluated pair of floats, so the choice is that of the exact logits but
//            for gaps of about 1e-8 of the logits' size;
//   choice   every CTA makes it for itself, one warp per token, and lists the experts that were hit,
//            their tokens ("columns") and gates;
//   gate/up  H = silu(x W_gate) * (x W_up) of the listed experts' columns;
//   down     out = sum over experts of gate * (H W_down), summed over all of them at once.
// Gate/up and down are cut into tiles of 64 weight channels; the tiles' K steps, one after the other,
// are dealt out to the CTAs in equal runs, so every SM streams the same number of bytes whatever the
// number of experts. A tile that is cut between CTAs leaves partial sums in the workspace; the CTA that
// finishes last adds them in order of their pieces (the result does not depend on who that is).
//
// Weights go through mma.sync m16n8k16 as the M operand, eight columns as N. Every warp has a ring of tiles of
// 16 K rows x 64 channels that TMA brings (128-byte swizzle) and that no other warp reads. They lie with the
// output channel contiguous, so a lane reads four rows of 8 channels, 16 bytes each, and pairs rows by byte
// permutes into the fragments of four MMAs; which channel is which fragment row is settled when results are
// stored. (The same pieces by cp.async or plain loads, 16 bytes a lane, come at 3.8 to 4.1 TB/s however many are
// under way, by TMA at 5.4.) The columns' values come by cp.async into slots that only their lane reads.
// tcgen05 would want 128 rows of a token operand that has one.
// H is carried as two bf16 numbers (value and remainder, 2^-17 of it), as the second MMA is free here.
#include <cuda_bf16.h>
#include <cuda.h>
#include <cmath>

#include "few.cuh"
#include "ptx.cuh"
#include "route_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kSlots = MOE_FEW_MAX_TOKENS * 8;          // T * top_k at most
constexpr int kSegs = kSlots + 4;                       // hit experts and shared ones
constexpr int kCols = kSlots + 4 * MOE_FEW_MAX_TOKENS;  // columns of all of them
constexpr int kAccLd = 68;       // floats between rows of 64 sums in shared memory (16-byte pieces)
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Order-preserving bits of a float that is not NaN, above 0 (0 stands for "not to be chosen").
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 becomes 0
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// What every CTA knows about the choice.
struct Plan {
  int idx[kSlots];
  float w[kSlots];
  int seg_e[kSegs];          // expert, or E + s
  int seg_base[kSegs + 1];   // first column
  uint8_t tok[kCols];        // token of a column
  float gate[kCols];
  int n_seg;
  volatile int fail;  // a wait ran past its limit
  int last[2];
  unsigned gen;
};
// Scratch of router and choice, in the ring's memory before the ring is used.
struct Scratch {
  float2 red[kWarps];
  float score[MOE_FEW_MAX_TOKENS][256];
  unsigned all[256][kSlots / 32];   // slots of an expert
  unsigned keep[256][kSlots / 32];  // those that are a column: kept, the first of their token
  int off[257];
};

// ------------------------------------------------------------------------------------ grid barrier
// Arrival and wait are apart, so that copies that need nothing of the other CTAs can be started
// between them. The wait is bounded; past it the status word says so and the kernel ends.
__device__ __forceinline__ void barrier_arrive(const FewArgs& a, Plan& p) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&a.meta->arrive, 1u) == gridDim.x - 1) {
      atomicExch(&a.meta->arrive, 0u);
      __threadfence();
      atomicExch(&a.meta->gen, p.gen + 1);
    }
  }
}
__device__ __forceinline__ bool barrier_wait(const FewArgs& a, Plan& p) {
  if (threadIdx.x == 0) {
    const unsigned g = p.gen;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (unsigned it = 1;; ++it) {
      unsigned now;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(now) : "l"(&a.meta->gen) : "memory");
      if (now != g) break;
      if ((it & 63u) == 0 && ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
        atomicOr(a.status, MOE_DEVFAULT_PIPELINE_TIMEOUT);
        p.fail = 1;
        break;
      }
    }
    __threadfence();
    p.gen = g + 1;
  }
  __syncthreads();
  return p.fail == 0;
}

// A CTA's run of K steps begins and ends inside tiles, as a rule: at most two of its pieces, the first (0)
// and the last (1), are parts of a tile whose other parts are other CTAs'. Those leave their sums in the
// workspace, and only when the run is done does the CTA say so (under load a fence and an atomic take 4 us, in
// which nothing would be read) and sees which tiles it has to join: those that it was the last to bring a part of.
struct Cuts {
  int head = -1, tail = -1;  // their tiles
};
__device__ __forceinline__ float* cut_sums(const FewArgs& a, int cta, int which) {
  return a.part + (size_t)cta * a.part_floats + which * (a.part_floats / 2);
}
// Which of its two cut pieces of a tile of K steps is CTA b's, when a run is `per` steps.
__device__ __forceinline__ int cut_of(int b, int per, int tile, int K) { return b * per <= tile * K ? 1 : 0; }

__device__ __forceinline__ unsigned bring_part(const FewArgs& a, int tile, int K, int per) {
  if (tile < 0) return 0;
  const int owner = tile * K / per;
  return atomicAdd(&a.meta->piece[owner >> 2], 1u << (owner & 3) * 8);
}
__device__ __forceinline__ int was_last(const FewArgs& a, unsigned before, int tile, int K, int per) {
  if (tile < 0) return 0;
  const int owner = tile * K / per, at = (owner & 3) * 8;
  const unsigned n = ((tile + 1) * K - 1) / per - owner + 1;
  if ((before >> at & 255u) != n - 1) return 0;
  atomicSub(&a.meta->piece[owner >> 2], n << at);  // zero again for the next part and the next call
  return 1;
}
__device__ __forceinline__ void say_cuts(const FewArgs& a, Plan& p, const Cuts& cuts, int K, int per) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const unsigned head = bring_part(a, cuts.head, K, per), tail = bring_part(a, cuts.tail, K, per);
    p.last[0] = was_last(a, head, cuts.head, K, per);
    p.last[1] = was_last(a, tail, cuts.tail, K, per);
    __threadfence();
  }
  __syncthreads();
}

// ------------------------------------------------------------------------------------------ router
// hi + s exactly: the rounding error of the sum (Knuth) goes to lo.
__device__ __forceinline__ void add_exact(float& hi, float& lo, float s) {
  const float sum = hi + s, back = sum - hi;
  lo += (hi - (sum - back)) + (s - back);
  hi = sum;
}
// logits[t, e] of expert e for every token; warps share out tokens, then the pieces of d.
__device__ void router(const FewArgs& a, Scratch& sc, int warp, int lane) {
  int wpt = kWarps;  // warps per token
  while (wpt * a.T > kWarps) wpt >>= 1;
  const int t = warp / wpt, part = warp % wpt;
  const int nv = a.d / 8;
  for (int e = blockIdx.x; e < a.E; e += gridDim.x) {
    if (t < a.T) {
      const uint4* w = reinterpret_cast<const uint4*>(a.W_g_t + (size_t)e * a.d);
      const uint4* x = reinterpret_cast<const uint4*>(a.x + (size_t)t * a.d);
      float hi = 0.f, lo = 0.f;
#pragma unroll 4
      for (int i = part * 32 + lane; i < nv; i += wpt * 32) {
        const uint4 wv = __ldg(w + i), xv = __ldg(x + i);
        float s = bf16_lo(wv.x) * bf16_lo(xv.x);
        s = fmaf(bf16_hi(wv.x), bf16_hi(xv.x), s);
        s = fmaf(bf16_lo(wv.y), bf16_lo(xv.y), s);
        s = fmaf(bf16_hi(wv.y), bf16_hi(xv.y), s);
        s = fmaf(bf16_lo(wv.z), bf16_lo(xv.z), s);
        s = fmaf(bf16_hi(wv.z), bf16_hi(xv.z), s);
        s = fmaf(bf16_lo(wv.w), bf16_lo(xv.w), s);
        s = fmaf(bf16_hi(wv.w), bf16_hi(xv.w), s);
        add_exact(hi, lo, s);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        lo += __shfl_xor_sync(kFull, lo, o);
        add_exact(hi, lo, __shfl_xor_sync(kFull, hi, o));
      }
      if (lane == 0) sc.red[warp] = make_float2(hi, lo);
    }
    __syncthreads();
    if (threadIdx.x < a.T) {
      float2 v = sc.red[threadIdx.x * wpt];
      for (int i = 1; i < wpt; ++i) {
        const float2 w = sc.red[threadIdx.x * wpt + i];
        v.y += w.y;
        add_exact(v.x, v.y, w.x);
      }
      // of an infinite sum only the first part says which
      a.logits[threadIdx.x * a.E + e] = isfinite(v.x) ? v.x + v.y : v.x;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------------ choice
// Token t's experts and gates from its logits, by one warp; lane l has experts l + 32 j.
__device__ void choose(const FewArgs& a, Plan& p, float* score, int t, int lane) {
  float l[8], s[8];
  uint32_t key[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = lane + 32 * j;
    l[j] = s[j] = 0.f;
    key[j] = 0;
    if (e < a.E) {
      l[j] = __ldcg(a.logits + t * a.E + e);
      s[j] = selection_score(a.mode, l[j], a.mode == MOE_ROUTE_BIAS_SELECT ? __ldg(a.bias + e) : 0.f,
                             a.mode == MOE_ROUTE_GUMBEL ? __ldg(a.u + (size_t)t * a.E + e) : 0.5f,
                             a.tau);
      key[j] = order_key(s[j]);
      score[e] = s[j];
    }
  }
  if (a.G > 0) {
    __syncwarp();
    const int per = a.E / a.G;
    uint32_t gk[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int g = lane + 32 * i;
      if (g < a.G) {
        float m = score[g * per];
        for (int j = 1; j < per; ++j) m = fmaxf(m, score[g * per + j]);
        gk[i] = order_key(m);
      }
    }
    unsigned long long live = 0;
    for (int r = 0; r < a.Gk; ++r) {
      const uint32_t best = __reduce_max_sync(kFull, max(gk[0], gk[1]));
      const int mine = gk[0] == best ? lane : gk[1] == best ? lane + 32 : 64;
      const int g = (int)__reduce_min_sync(kFull, (unsigned)mine);
      live |= 1ull << g;
      if (g == lane) gk[0] = 0;
      if (g == lane + 32) gk[1] = 0;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = lane + 32 * j;
      if (e < a.E && !(live >> (e / per) & 1)) key[j] = 0;
    }
  }
  float val = -INFINITY;  // of lane i: what the i-th choice's gate is made of
  int mine = 0;
  for (int r = 0; r < a.k; ++r) {
    uint32_t best = 0;
    int e = 0;
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (key[j] > best) {
        best = key[j];
        e = lane + 32 * j;
        v = a.mode == MOE_ROUTE_GUMBEL ? s[j] : l[j];
      }
    const uint32_t top = __reduce_max_sync(kFull, best);
    const unsigned e_top = __reduce_min_sync(kFull, best == top ? (unsigned)e : 0xffffu);
    v = __shfl_sync(kFull, v, e_top & 31);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e_top == (unsigned)(lane + 32 * j)) key[j] = 0;
    if (lane == r) {
      val = v;
      mine = (int)e_top;
    }
  }
  float m = -INFINITY;
  for (int r = 0; r < a.k; ++r) m = fmaxf(m, __shfl_sync(kFull, val, r));
  const float ex = lane < a.k ? expf(val - m) : 0.f;
  float sum = 0.f;
  for (int r = 0; r < a.k; ++r) sum += __shfl_sync(kFull, ex, r);
  if (lane < a.k) {
    p.idx[t * a.k + lane] = mine;
    p.w[t * a.k + lane] = ex / sum;
  }
}

// Number of set bits of a slot mask below slot s.
__device__ __forceinline__ int rank_of(const unsigned (&m)[kSlots / 32], int s) {
  int n = 0;
#pragma unroll
  for (int w = 0; w < kSlots / 32; ++w) {
    const int lo = s - 32 * w;
    n += __popc(lo >= 32 ? m[w] : lo > 0 ? m[w] & ((1u << lo) - 1u) : 0u);
  }
  return n;
}

// Lists the experts that were hit, shared ones first, with their columns and gates. A token that was given
// the same expert twice has one column with both gates. Of an expert's slots the first C count.
__device__ void make_plan(const FewArgs& a, Plan& p, Scratch& sc, int warp, int lane) {
  const int n = a.T * a.k, tid = threadIdx.x;
  for (int i = tid; i < a.E * (kSlots / 32); i += kThreads) {
    (&sc.all[0][0])[i] = 0;
    (&sc.keep[0][0])[i] = 0;
  }
  __syncthreads();
  const int e = tid < n ? p.idx[tid] : -1;
  const bool sound = (unsigned)e < (unsigned)a.E;
  if (tid < n) {
    if (sound)
      atomicOr(&sc.all[e][tid >> 5], 1u << (tid & 31));
    else if (blockIdx.x == 0)
      atomicOr(a.status, MOE_DEVFAULT_BAD_EXPERT_INDEX);
  }
  __syncthreads();
  int rank = 0;
  bool column = false;
  float gate = 0.f;
  if (sound) {
    rank = rank_of(sc.all[e], tid);
    column = rank < a.C;
    const int t0 = tid / a.k * a.k;
    for (int s = t0; s < tid; ++s)
      if (p.idx[s] == e) column = false;  // the token's earlier slot has the column
    if (column) {
      gate = p.w[tid];
      int r = rank;
      for (int s = tid + 1; s < t0 + a.k; ++s)
        if (p.idx[s] == e && ++r < a.C) gate += p.w[s];
      atomicOr(&sc.keep[e][tid >> 5], 1u << (tid & 31));
    }
  }
  __syncthreads();
  if (warp == 0) {
    int segs = a.S, cols = a.S * a.T;
    if (lane < a.S) {
      p.seg_e[lane] = a.E + lane;
      p.seg_base[lane] = lane * a.T;
    }
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      int cnt = 0;
      if (e0 + lane < a.E)
        for (int w = 0; w < kSlots / 32; ++w) cnt += __popc(sc.keep[e0 + lane][w]);
      const unsigned hit = __ballot_sync(kFull, cnt > 0);
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += v;
      }
      if (cnt > 0) {
        const int at = segs + __popc(hit & ((1u << lane) - 1u));
        p.seg_e[at] = e0 + lane;
        p.seg_base[at] = cols + incl - cnt;
        sc.off[e0 + lane] = cols + incl - cnt;
      }
      segs += __popc(hit);
      cols += __shfl_sync(kFull, incl, 31);
    }
    if (lane == 0) {
      p.n_seg = segs;
      p.seg_base[segs] = cols;
    }
  }
  __syncthreads();
  if (column) {
    const int c = sc.off[e] + rank_of(sc.keep[e], tid);
    p.tok[c] = (uint8_t)(tid / a.k);
    p.gate[c] = gate;
  }
  for (int i = tid; i < a.S * a.T; i += kThreads) {
    p.tok[i] = (uint8_t)(i % a.T);
    p.gate[i] = 1.f;
  }
  // the results that moe_layer_forward also offers
  const moe_route_out& ro = a.ro;
  if (blockIdx.x == 0 && (ro.topk_idx || ro.topk_w) && tid < n) {
    if (ro.topk_idx) ro.topk_idx[tid] = p.idx[tid];
    if (ro.topk_w) ro.topk_w[tid] = p.w[tid];
  }
  if (blockIdx.x == 0 && (ro.counts || ro.offsets || ro.perm_slot || ro.slot_pos)) {
    __syncthreads();
    if (warp == 0) {
      int base = 0;
      for (int e0 = 0; e0 < a.E; e0 += 32) {
        int cnt = 0;
        if (e0 + lane < a.E)
          for (int w = 0; w < kSlots / 32; ++w) cnt += __popc(sc.all[e0 + lane][w]);
        if (ro.counts && e0 + lane < a.E) ro.counts[e0 + lane] = cnt;
        cnt = min(cnt, a.C);
        int incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(kFull, incl, o);
          if (lane >= o) incl += v;
        }
        if (e0 + lane < a.E) sc.off[e0 + lane] = base + incl - cnt;
        base += __shfl_sync(kFull, incl, 31);
      }
      if (lane == 0) sc.off[a.E] = base;
    }
    __syncthreads();
    if (ro.offsets)
      for (int i = tid; i <= a.E; i += kThreads) ro.offsets[i] = sc.off[i];
    if (tid < n) {
      const int pos = sound && rank < a.C ? sc.off[e] + rank : -1;
      if (ro.slot_pos) ro.slot_pos[tid] = pos;
      if (ro.perm_slot) {
        if (tid >= sc.off[a.E]) ro.perm_slot[tid] = -1;
        if (pos >= 0) ro.perm_slot[pos] = tid;
      }
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------------------------------------- tiles
// How the K steps of `tiles` tiles of K steps each are dealt out: run i is [i * per, (i + 1) * per).
struct Deal {
  int K, total, per;
  __device__ Deal(int K_, int tiles, int least) : K(K_), total(K_ * tiles) {
    per = max((total + (int)gridDim.x - 1) / (int)gridDim.x, min(K, least));
  }
  __device__ int begin() const { return min(total, (int)blockIdx.x * per); }
  __device__ int end() const { return min(total, ((int)blockIdx.x + 1) * per); }
};

// A warp's ring: kStages tiles of weights (16 rows of 64 channels, 2 KB) and, for each, its lanes' pieces of the
// columns' values (16 bytes per lane and 8 columns). Tiles are taken in the order they were asked for.
template <int NT, int kStages>
struct Ring {
  static constexpr int kTile = 2048, kPiece = 512 * NT;
  uint32_t w, b, bar;  // slot 0: the tile, this lane's piece, the tile's mbarrier
  int slot;            // the next tile to be taken
  uint32_t phase;

  __device__ __forceinline__ uint32_t tile(int i) const { return w + i * kTile; }
  __device__ __forceinline__ uint32_t piece(int i) const { return b + i * kPiece; }
  __device__ __forceinline__ int later(int i) const {  // the slot i places on
    const int k = slot + i;
    return k >= kStages ? k - kStages : k;
  }
  __device__ __forceinline__ void next() {
    if (++slot == kStages) {
      slot = 0;
      phase ^= 1u;
    }
  }
  // Until the tile and this lane's piece are there. A wait that runs past its limit lets the kernel go on with
  // what there is (later waits give up at once), and the status word says so.
  __device__ __forceinline__ void wait(const FewArgs& a, Plan& p) const {
    ptx::mbar_wait_bounded_warp(bar + 8 * slot, phase, &p.fail, a.status, MOE_DEVFAULT_PIPELINE_TIMEOUT,
                                kWaitLimitNs);
    cp_wait<kStages - 1>();
  }
  // One lane asks for a tile. What the warp read of the slot before is in registers.
  __device__ __forceinline__ void ask(int i, const CUtensorMap* map, int c, int row, int matrix) const {
    const uint32_t m = bar + 8 * i;
    ptx::mbar_arrive_expect_tx(m, kTile);
    ptx::tma_load_3d(tile(i), map, m, c, row, matrix);
  }
};

// Reads a tile into the fragments of four MMAs: rows of fragment j are channels 8 g + 2 j (its rows 0-7) and
// 8 g + 2 j + 1 (rows 8-15) for lane 4 g + q, whose K rows are 2 q, 2 q + 1, 2 q + 8, 2 q + 9. Swizzled: 16-byte
// piece c of row r is at c ^ (r % 8), so the eight lanes of a quarter of a load read eight different ones.
__device__ __forceinline__ void fragments(uint32_t tile, int lane, uint32_t (&f)[4][4]) {
  const int g = lane >> 2, q = lane & 3;
  const uint32_t even = tile + q * 256 + ((g ^ (2 * q)) << 4);
  const uint32_t odd = tile + q * 256 + 128 + ((g ^ (2 * q + 1)) << 4);
  const uint4 r0 = lds16(even), r1 = lds16(odd), r2 = lds16(even + 1024), r3 = lds16(odd + 1024);
  const uint32_t a0[4] = {r0.x, r0.y, r0.z, r0.w}, a1[4] = {r1.x, r1.y, r1.z, r1.w};
  const uint32_t a2[4] = {r2.x, r2.y, r2.z, r2.w}, a3[4] = {r3.x, r3.y, r3.z, r3.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j][0] = __byte_perm(a0[j], a1[j], 0x5410);
    f[j][1] = __byte_perm(a0[j], a1[j], 0x7632);
    f[j][2] = __byte_perm(a2[j], a3[j], 0x5410);
    f[j][3] = __byte_perm(a2[j], a3[j], 0x7632);
  }
}

// Where a warp is in its K steps of gate/up: tile j (expert and 64 channels), step s of it.
template <int NT, int kStages>
struct UpFeed {
  const FewArgs& a;
  const FewMaps& maps;
  const Plan& p;
  const Deal& deal;
  int slice, lane, mat, j, s, kend, channel, matrix;
  const CUtensorMap* map;
  const uint16_t* x[NT];
  uint32_t bytes[NT];
  bool more;

  __device__ UpFeed(const FewArgs& a_, const FewMaps& m_, const Plan& p_, const Deal& d_, int warp, int lane_)
      : a(a_), maps(m_), p(p_), deal(d_), slice(warp >> 1), lane(lane_), mat(warp & 1) {
    j = deal.begin() / deal.K;
    s = deal.begin() - j * deal.K + slice;
    kend = min(deal.K, deal.end() - j * deal.K);
    more = deal.begin() < deal.end();
    if (more) {
      tile();
      settle();
    }
  }
  __device__ void tile() {
    const int nfb = a.f / 64, seg = j / nfb, e = p.seg_e[seg];
    map = e < a.E ? (mat ? &maps.up : &maps.gate) : (mat ? &maps.sh_up : &maps.sh_gate);
    matrix = e < a.E ? e : e - a.E;
    channel = (j - seg * nfb) * 64;
    const int g = lane >> 2, q = lane & 3, base = p.seg_base[seg], cnt = p.seg_base[seg + 1] - base;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool there = g + 8 * n < cnt;
      bytes[n] = there ? 4 : 0;
      x[n] = a.x + (size_t)(there ? p.tok[base + g + 8 * n] : 0) * a.d + 2 * q;
    }
  }
  __device__ void settle() {
    while (s >= kend) {
      ++j;
      if (j * deal.K >= deal.end()) {
        more = false;
        return;
      }
      s = slice;
      kend = min(deal.K, deal.end() - j * deal.K);
      tile();
    }
  }
  __device__ __forceinline__ void issue(const Ring<NT, kStages>& r, int slot) {
    if (more) {
      if (lane == 0) r.ask(slot, map, channel, s * 16, matrix);
      const uint32_t to = r.piece(slot);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        cp_async4(to + 512 * n, x[n] + s * 16, bytes[n]);
        cp_async4(to + 512 * n + 4, x[n] + s * 16 + 8, bytes[n]);
      }
      s += 8;
      if (s >= kend) settle();
    }
    cp_commit();
  }
};

// A warp's sums to shared memory: row `column` of 64 channels, for the columns that there are.
template <int NT>
__device__ __forceinline__ void store_sums(float* acc_s, const float (&acc)[NT][4][4], int cnt,
                                           int lane) {
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = 8 * n + 2 * q + i;
      if (c < cnt) {
        float4* row = reinterpret_cast<float4*>(acc_s + c * kAccLd + 8 * g);
        row[0] = make_float4(acc[n][0][i], acc[n][0][2 + i], acc[n][1][i], acc[n][1][2 + i]);
        row[1] = make_float4(acc[n][2][i], acc[n][2][2 + i], acc[n][3][i], acc[n][3][2 + i]);
      }
    }
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// Four channels of H, 4 c4 and on, of a column's row. 16 channels are 64 bytes: for each q the bf16 values of
// channels 2 q, 2 q + 1, 2 q + 8, 2 q + 9, then the four remainders (a lane's K rows of an MMA).
__device__ __forceinline__ void store_h(uint32_t* row, int c4, float4 g, float4 u) {
  const float gv[4] = {g.x, g.y, g.z, g.w}, uv[4] = {u.x, u.y, u.z, u.w};
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float h = gv[i] / (1.f + expf(-gv[i])) * uv[i];
    const __nv_bfloat16 b = __float2bfloat16_rn(h);
    const float back = __bfloat162float(b);
    hi[i] = __bfloat16_as_ushort(b);
    // an infinite or NaN value has no remainder
    lo[i] = isfinite(back) ? __bfloat16_as_ushort(__float2bfloat16_rn(h - back)) : 0;
  }
  uint32_t* to = row + (c4 >> 2) * 16 + (c4 & 1) * 8 + ((c4 >> 1) & 1);
  to[0] = hi[0] | hi[1] << 16;
  to[2] = lo[0] | lo[1] << 16;
  to[4] = hi[2] | hi[3] << 16;
  to[6] = lo[2] | lo[3] << 16;
}

template <int NT, int kStages>
__device__ void gate_up(const FewArgs& a, const FewMaps& maps, Plan& p, float* acc_s,
                        Ring<NT, kStages>& ring, int warp, int lane) {
  const int nfb = a.f / 64;
  // a tile of up to 32 steps (four of a warp) is not cut: joining the pieces would take longer
  const Deal deal(a.d / 16, p.n_seg * nfb, 32);
  UpFeed<NT, kStages> feed(a, maps, p, deal, warp, lane);
#pragma unroll
  for (int i = 0; i < kStages; ++i) feed.issue(ring, ring.later(i));
  const int slice = warp >> 1, begin = deal.begin(), end = deal.end();
  Cuts cuts;
  for (int at = begin; at < end;) {
    const int j = at / deal.K, k0 = at - j * deal.K, k1 = min(deal.K, end - j * deal.K);
    const int seg = j / nfb, fb = j - seg * nfb;
    const int base = p.seg_base[seg], cnt = p.seg_base[seg + 1] - base;
    float acc[NT][4][4] = {};
    for (int s = k0 + slice; s < k1; s += 8) {
      ring.wait(a, p);
      uint32_t f[4][4];
      fragments(ring.tile(ring.slot), lane, f);
      uint2 b[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) b[n] = lds8(ring.piece(ring.slot) + 512 * n);
      __syncwarp();
      feed.issue(ring, ring.slot);
      ring.next();
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n == 0 || cnt > 8)
#pragma unroll
          for (int m = 0; m < 4; ++m) mma(acc[n][m], f[m], b[n].x, b[n].y);
    }
    store_sums<NT>(acc_s + warp * (8 * NT) * kAccLd, acc, cnt, lane);
    __syncthreads();
    const bool whole = k0 == 0 && k1 == deal.K;
    const int which = k0 == 0 ? 1 : 0;
    if (!whole) (k0 == 0 ? cuts.tail : cuts.head) = j;
    float4* part = reinterpret_cast<float4*>(cut_sums(a, blockIdx.x, which));
    for (int i = threadIdx.x; i < cnt * 16; i += kThreads) {
      const int c = i >> 4, c4 = i & 15;
      float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
#pragma unroll
      for (int w = 0; w < kWarps; w += 2) {
        const float* row = acc_s + (w * (8 * NT) + c) * kAccLd + 4 * c4;
        g = add4(g, *reinterpret_cast<const float4*>(row));
        u = add4(u, *reinterpret_cast<const float4*>(row + (8 * NT) * kAccLd));
      }
      if (whole) {
        store_h(a.h + (size_t)(base + c) * a.f, fb * 16 + c4, g, u);
      } else {
        part[i] = g;
        part[16 * MOE_FEW_MAX_TOKENS + i] = u;
      }
    }
    at = j * deal.K + k1;
    __syncthreads();  // the sums' memory is free again
  }
  cp_wait<0>();
  say_cuts(a, p, cuts, deal.K, deal.per);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!p.last[k]) continue;
    const int j = k == 0 ? cuts.head : cuts.tail, seg = j / nfb, fb = j - seg * nfb;
    const int base = p.seg_base[seg], cnt = p.seg_base[seg + 1] - base;
    const int first = j * deal.K / deal.per, last = ((j + 1) * deal.K - 1) / deal.per;
    for (int i = threadIdx.x; i < cnt * 16; i += kThreads) {
      float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
#pragma unroll 4
      for (int b = first; b <= last; ++b) {
        const float4* from = reinterpret_cast<const float4*>(cut_sums(a, b, cut_of(b, deal.per, j, deal.K)));
        g = add4(g, __ldcg(from + i));
        u = add4(u, __ldcg(from + 16 * MOE_FEW_MAX_TOKENS + i));
      }
      store_h(a.h + (size_t)(base + (i >> 4)) * a.f, fb * 16 + (i & 15), g, u);
    }
  }
}

// Where a warp is in its K steps of down: tile j (64 channels), step s of all experts' channels in a row.
template <int NT, int kStages>
struct DownFeed {
  const FewArgs& a;
  const FewMaps& maps;
  const Plan& p;
  const Deal& deal;
  int slice, lane, fs, j, s, kend, seg, matrix;
  const CUtensorMap* map;
  const uint4* h[NT];
  uint32_t bytes[NT];
  bool more;

  __device__ DownFeed(const FewArgs& a_, const FewMaps& m_, const Plan& p_, const Deal& d_, int warp, int lane_)
      : a(a_), maps(m_), p(p_), deal(d_), slice(warp), lane(lane_), fs(a_.f / 16) {
    j = deal.begin() / deal.K;
    s = deal.begin() - j * deal.K + slice;
    kend = min(deal.K, deal.end() - j * deal.K);
    more = deal.begin() < deal.end();
    if (more) settle();
  }
  __device__ void expert() {
    const int e = p.seg_e[seg], g = lane >> 2, q = lane & 3;
    map = e < a.E ? &maps.down : &maps.sh_down;
    matrix = e < a.E ? e : e - a.E;
    const int base = p.seg_base[seg], cnt = p.seg_base[seg + 1] - base;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool there = g + 8 * n < cnt;
      bytes[n] = there ? 16 : 0;
      h[n] = reinterpret_cast<const uint4*>(a.h + (size_t)(base + (there ? g + 8 * n : 0)) * a.f) + q;
    }
  }
  __device__ void settle() {
    while (s >= kend) {
      ++j;
      if (j * deal.K >= deal.end()) {
        more = false;
        return;
      }
      s = slice;
      kend = min(deal.K, deal.end() - j * deal.K);
    }
    seg = s / fs;
    expert();
  }
  __device__ __forceinline__ void issue_w(const Ring<NT, kStages>& r, int slot) const {
    if (more && lane == 0) r.ask(slot, map, j * 64, (s - seg * fs) * 16, matrix);
  }
  __device__ __forceinline__ void issue_h(const Ring<NT, kStages>& r, int slot) const {
    if (more) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        cp_async16(r.piece(slot) + 512 * n, h[n] + (s - seg * fs) * 4, bytes[n]);
    }
    cp_commit();
  }
  __device__ __forceinline__ void next() {
    if (!more) return;
    s += kWarps;
    if (s >= kend) {
      settle();
    } else if (s >= (seg + 1) * fs) {
      seg = s / fs;
      expert();
    }
  }
};

// Adds gate * sums of an expert's columns to the rows of their tokens, which are different ones.
template <int NT>
__device__ __forceinline__ void add_sums(float* acc_s, float (&acc)[NT][4][4], const Plan& p, int seg,
                                         int lane) {
  const int g = lane >> 2, q = lane & 3;
  const int base = p.seg_base[seg], cnt = p.seg_base[seg + 1] - base;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = 8 * n + 2 * q + i;
      if (c < cnt) {
        const float w = p.gate[base + c];
        float4* row = reinterpret_cast<float4*>(acc_s + p.tok[base + c] * kAccLd + 8 * g);
        float4 v = row[0];
        row[0] = make_float4(fmaf(w, acc[n][0][i], v.x), fmaf(w, acc[n][0][2 + i], v.y),
                             fmaf(w, acc[n][1][i], v.z), fmaf(w, acc[n][1][2 + i], v.w));
        v = row[1];
        row[1] = make_float4(fmaf(w, acc[n][2][i], v.x), fmaf(w, acc[n][2][2 + i], v.y),
                             fmaf(w, acc[n][3][i], v.z), fmaf(w, acc[n][3][2 + i], v.w));
      }
    }
  __syncwarp();
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][m][i] = 0.f;
}

__device__ __forceinline__ uint2 bf16x4(float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

template <int NT, int kStages>
__device__ void down(const FewArgs& a, const FewMaps& maps, Plan& p, float* acc_s, Ring<NT, kStages>& ring,
                     int warp, int lane) {
  const int fs = a.f / 16;
  // as in gate/up a tile is not cut below four steps of a warp
  const Deal deal(p.n_seg * fs, a.d / 64, 4 * kWarps);
  const int begin = deal.begin(), end = deal.end();
  Cuts cuts;
  DownFeed<NT, kStages> feed(a, maps, p, deal, warp, lane);
  {
    // the first weights are on their way while the other CTAs finish H
    DownFeed<NT, kStages> ahead = feed;
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      ahead.issue_w(ring, ring.later(i));
      ahead.next();
    }
  }
  float* mine = acc_s + warp * (8 * NT) * kAccLd;
  for (int i = lane; i < a.T * kAccLd; i += 32) mine[i] = 0.f;
  __syncwarp();
  barrier_wait(a, p);  // past its limit the rest runs on what there is, and takes the copies under way
#pragma unroll
  for (int i = 0; i < kStages; ++i) {
    feed.issue_h(ring, ring.later(i));
    feed.next();
  }
  for (int at = begin; at < end;) {
    const int j = at / deal.K, k0 = at - j * deal.K, k1 = min(deal.K, end - j * deal.K);
    float acc[NT][4][4] = {};
    int seg = 0, cnt = 0, seg_end = 0;
    for (int s = k0 + warp; s < k1; s += kWarps) {
      if (s >= seg_end) {
        if (seg_end > 0) add_sums<NT>(mine, acc, p, seg, lane);
        seg = s / fs;
        seg_end = (seg + 1) * fs;
        cnt = p.seg_base[seg + 1] - p.seg_base[seg];
      }
      ring.wait(a, p);
      uint32_t f[4][4];
      fragments(ring.tile(ring.slot), lane, f);
      uint4 b[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) b[n] = lds16(ring.piece(ring.slot) + 512 * n);
      __syncwarp();
      feed.issue_w(ring, ring.slot);
      feed.issue_h(ring, ring.slot);
      feed.next();
      ring.next();
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n == 0 || cnt > 8)
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            mma(acc[n][m], f[m], b[n].x, b[n].y);
            mma(acc[n][m], f[m], b[n].z, b[n].w);
          }
    }
    if (seg_end > 0) add_sums<NT>(mine, acc, p, seg, lane);
    __syncthreads();
    const bool whole = k0 == 0 && k1 == deal.K;
    const int which = k0 == 0 ? 1 : 0;
    if (!whole) (k0 == 0 ? cuts.tail : cuts.head) = j;
    float4* part = reinterpret_cast<float4*>(cut_sums(a, blockIdx.x, which));
    for (int i = threadIdx.x; i < a.T * 16; i += kThreads) {
      const int t = i >> 4, c4 = i & 15;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        v = add4(v, *reinterpret_cast<const float4*>(acc_s + (w * (8 * NT) + t) * kAccLd + 4 * c4));
      if (whole)
        *reinterpret_cast<uint2*>(a.out + (size_t)t * a.d + j * 64 + 4 * c4) = bf16x4(v);
      else
        part[i] = v;
    }
    at = j * deal.K + k1;
    __syncthreads();
    if (at < end) {
      for (int i = lane; i < a.T * kAccLd; i += 32) mine[i] = 0.f;
      __syncwarp();
    }
  }
  cp_wait<0>();
  say_cuts(a, p, cuts, deal.K, deal.per);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!p.last[k]) continue;
    const int j = k == 0 ? cuts.head : cuts.tail, first = j * deal.K / deal.per, last = ((j + 1) * deal.K - 1) / deal.per;
    for (int i = threadIdx.x; i < a.T * 16; i += kThreads) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int b = first; b <= last; ++b)
        v = add4(v, __ldcg(reinterpret_cast<const float4*>(
                               cut_sums(a, b, cut_of(b, deal.per, j, deal.K))) +
                           i));
      *reinterpret_cast<uint2*>(a.out + (size_t)(i >> 4) * a.d + j * 64 + 4 * (i & 15)) = bf16x4(v);
    }
  }
}

template <int NT, int kStages>
constexpr int ring_bytes() {
  return kWarps * kStages * (Ring<NT, kStages>::kTile + Ring<NT, kStages>::kPiece);
}
template <int NT, int kStages>
constexpr int smem_bytes() {
  return 1024 + ring_bytes<NT, kStages>() + kWarps * 8 * NT * kAccLd * 4;  // 1024: swizzled tiles' alignment
}

template <int NT, int kStages>
__global__ void __launch_bounds__(kThreads, 1)
    few_kernel(const __grid_constant__ FewArgs a, const __grid_constant__ FewMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Plan p;
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  uint8_t* smem = smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Scratch& sc = *reinterpret_cast<Scratch*>(smem);
  static_assert(sizeof(Scratch) <= ring_bytes<NT, kStages>(), "it lies in the ring");
  float* acc_s = reinterpret_cast<float*>(smem + ring_bytes<NT, kStages>());
  Ring<NT, kStages> ring;
  ring.w = ptx::smem_u32(smem) + warp * kStages * ring.kTile;
  ring.b = ptx::smem_u32(smem) + kWarps * kStages * ring.kTile + warp * kStages * ring.kPiece + lane * 16;
  ring.bar = ptx::smem_u32(&bars[warp][0]);
  ring.slot = 0;
  ring.phase = 0;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) ptx::mbar_init(ring.bar + 8 * i, 1);
    ptx::fence_mbarrier_init();
  }
  if (threadIdx.x == kThreads - 1) {
    ptx::prefetch_tmap(&maps.gate);
    ptx::prefetch_tmap(&maps.up);
    ptx::prefetch_tmap(&maps.down);
    if (a.S > 0) {
      ptx::prefetch_tmap(&maps.sh_gate);
      ptx::prefetch_tmap(&maps.sh_up);
      ptx::prefetch_tmap(&maps.sh_down);
    }
  }
  if (threadIdx.x == 0) {
    p.fail = 0;
    p.gen = *reinterpret_cast<volatile unsigned*>(&a.meta->gen);
  }
  if (a.W_g_t != nullptr) {
    router(a, sc, warp, lane);
    barrier_arrive(a, p);
    if (!barrier_wait(a, p)) return;
    for (int t = warp; t < a.T; t += kWarps) choose(a, p, sc.score[t], t, lane);
  } else {
    for (int i = threadIdx.x; i < a.T * a.k; i += kThreads) {
      p.idx[i] = __ldg(a.idx_in + i);
      p.w[i] = a.w_in != nullptr ? __ldg(a.w_in + i) : 1.f;
    }
  }
  __syncthreads();
  make_plan(a, p, sc, warp, lane);
  if (p.n_seg == 0) {  // not one sound index
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < a.T * a.d / 4; i += gridDim.x * kThreads)
      reinterpret_cast<uint2*>(a.out)[i] = make_uint2(0u, 0u);
    return;
  }
  ptx::fence_proxy_async_smem();  // the scratch gives way to tiles that TMA writes
  __syncthreads();
  gate_up<NT, kStages>(a, maps, p, acc_s, ring, warp, lane);
  barrier_arrive(a, p);
  down<NT, kStages>(a, maps, p, acc_s, ring, warp, lane);
}

template <int NT, int kStages>
cudaError_t launch(const FewArgs& a, const FewMaps& maps, cudaStream_t st) {
  constexpr int smem = smem_bytes<NT, kStages>();
  cudaError_t e = cudaFuncSetAttribute(few_kernel<NT, kStages>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms() < kFewMaxCtas ? num_sms() : kFewMaxCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_kernel<NT, kStages>, a, maps);
}

}  // namespace

FewLayout few_layout(const Shape& s) {
  FewLayout L;
  size_t o = 512;  // status word and counter block, as in every workspace
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  L.meta = 256;
  L.logits = take(4ull * s.T * s.E);
  L.h = take(4ull * s.T * (s.k + s.S) * s.f);
  L.part_floats = 2 * 2 * MOE_FEW_MAX_TOKENS * 64;  // two pieces of a CTA, of gate and up: 64 channels, 16 columns
  L.part = take(4ull * kFewMaxCtas * L.part_floats);
  L.wg_t = take(2ull * s.d * s.E);
  L.total = o;
  return L;
}

cudaError_t launch_few(const FewArgs& a, cudaStream_t st) {
  FewMaps maps = {};
  const auto map = [&](CUtensorMap& m, const uint16_t* w, int n, int rows, int cols) {
    return make_tmap_3d(&m, w, n, rows, cols, 64, 16, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, false);
  };
  bool ok = map(maps.gate, a.gate, a.E, a.d, a.f) && map(maps.up, a.up, a.E, a.d, a.f) &&
            map(maps.down, a.down, a.E, a.f, a.d);
  if (a.S > 0)
    ok = ok && map(maps.sh_gate, a.sh_gate, a.S, a.d, a.f) && map(maps.sh_up, a.sh_up, a.S, a.d, a.f) &&
         map(maps.sh_down, a.sh_down, a.S, a.f, a.d);
  if (!ok) return cudaErrorInvalidValue;
  return a.T <= 8 ? launch<1, 4>(a, maps, st) : launch<2, 3>(a, maps, st);
}

}  // namespace moe
