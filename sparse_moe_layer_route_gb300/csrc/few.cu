// The whole MoE layer for up to 16 tokens in one kernel: router, choice, gate/up, SwiGLU, down, combine.
//
// With few tokens the layer is the reading of the chosen experts' weights, each once: 6 d f bytes an
// expert, no more than one token for most of them. One persistent CTA per SM (cooperative launch) goes
// through four parts, with a grid barrier after the first and the third:
//   router   one expert per CTA: logits of all tokens. Eight products (exact in fp32) at a time are summed in fp32, the
//            sums of eight in an unevaluated pair of floats, which becomes one fp32 logit. So a logit is off by at most
//            7 * 2^-24 of sum |x_i w_i|, from the seven adds inside the eights, and 2^-24 of itself; experts whose
//            scores are nearer to one another than that may change places;
//   choice   every CTA makes it for itself, one warp per token, and lists the experts that were hit,
//            their tokens ("columns") and gates;
//   gate/up  H = silu(x W_gate) * (x W_up) of the listed experts' columns;
//   down     out = sum over experts of gate * (H W_down), summed over all of them at once.
// Gate/up and down are cut into tiles of 64 weight channels, and where those are few, along K as well, into units
// of work. CTAs take units as they get free. Of a tile that is cut the units leave partial sums in the
// workspace, and the CTA that finishes last adds them in order (the result does not depend on who that is).
//
// Weights go through mma.sync m16n8k16 as the M operand, eight columns as N. Every warp has a ring of tiles of
// 32 K rows x 64 channels that TMA brings (128-byte swizzle) and that no other warp reads. They lie with the
// output channel contiguous, so a lane reads four rows of 8 channels, 16 bytes each, and pairs rows by byte
// permutes into the fragments of four MMAs; which channel is which fragment row is settled when results are
// stored. (The same pieces by cp.async or plain loads, 16 bytes a lane, come at 3.8 to 4.1 TB/s however many are
// under way, by TMA at 5.4.) The columns' values come by cp.async into slots that only their lane reads.
// tcgen05 would want 128 rows of a token operand that has one.
// H is carried as two bf16 numbers (value and remainder, 2^-17 of it), as the second MMA is free here.
//
// Measured with 128 + 1 experts, d 7168, d_ff 2048, top-2 (decode): one token 60 us (266 MB, 4.4 TB/s), of which 9
// pass before the first weight is asked for, 29 in gate/up (6.1 TB/s), 3 at the barrier, 14 in down; 16 tokens 370
// to 421 us (2.4 to 2.7 GB by how many experts are hit, and by the GPU: 386 us on equal inputs, 6.7 TB/s). With 64 + 2
// experts, d 2048, d_ff 1408, top-6, five tokens: 77 to 88 us (465 MB). A layer of d 256, d_ff 512: 21 us, the launch's
// and the barriers'. The layer of many tokens (nine launches, tiles of 128 rows) takes 117 us for one token of the
// decode shape where this takes 60, 259 for eight (226) and 429 for sixteen (416); with 16 experts of d 4096, d_ff 14336
// 597 for eight (557) and 748 for sixteen (755): at sixteen tokens the two are alike. Bringing the shared
// experts' weights to L2 before the choice is known slows the router by what it gains (60 us with 16 MB, 62 with 64).
#include <cuda_bf16.h>
#include <cuda.h>
#include <climits>
#include <cmath>

#include "few.cuh"
#include "ptx.cuh"
#include "route_common.cuh"

namespace moe {
namespace {

constexpr int kMostWarps = 16;
// A CTA's warps: W that stream weights (the workers), one that deals units of work out, one that joins them.
constexpr int workers(int W) { return 32 * W; }
constexpr int threads(int W) { return 32 * W + 64; }
constexpr int kQueue = 8;                   // units known ahead
constexpr int kList = 16;                   // tiles for the workers to join
constexpr int kSlots = MOE_FEW_MAX_TOKENS * 8;          // T * top_k at most
constexpr int kSegs = kSlots + 4;                       // hit experts and shared ones
constexpr int kCols = kSlots + 4 * MOE_FEW_MAX_TOKENS;  // columns of all of them
constexpr int kAccLd = 68;       // floats between rows of 64 sums in shared memory (16-byte pieces)
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
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
  unsigned long long target;  // of the barrier that this CTA has arrived at
  // units of work: numbers of the first `known` (a ring), how many are done and accounted for, and where an
  // overrun ended the list
  volatile int unit[kQueue], known, done, joined, limit;
  int list[kList], n_list;  // tiles whose last unit this CTA brought
};
// Scratch of router and choice, in the ring's memory before the ring is used.
struct Scratch {
  float2 red[kMostWarps];
  float score[MOE_FEW_MAX_TOKENS][256];
  unsigned all[256][kSlots / 32];   // slots of an expert
  unsigned keep[256][kSlots / 32];  // those that are a column: kept, the first of their token
  int off[257];
};

// ------------------------------------------------------------------------------------ grid barrier
// Arrivals are counted through, call after call: the count a barrier waits for is the next multiple of the number
// of CTAs above what it was before this CTA's own arrival. That is one atomic and one line to watch.
// Arrival and wait are apart, so that copies that need nothing of the other CTAs can be started
// between them. The wait is bounded; past it the status word says so. a.absent: 1 in the check of these waits, for
// which a CTA more than there are has to arrive.
__device__ __forceinline__ void barrier_arrive(const FewArgs& a, Plan& p) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const unsigned long long n = gridDim.x + a.absent, before = atomicAdd(&a.meta->arrived, 1ull);
    p.target = (before / n + 1) * n;
  }
}
// All threads get the same answer: whether all CTAs have arrived and no wait of this one has given up. They may come
// from different branches, so it is a barrier by number: warps with different tasks wait at different places.
__device__ __forceinline__ bool barrier_wait(const FewArgs& a, Plan& p) {
  int late = p.fail;
  if (threadIdx.x == 0) {
    uint64_t t0 = 0;
    for (unsigned it = 1;; ++it) {
      unsigned long long now;
      asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(now) : "l"(&a.meta->arrived) : "memory");
      if (now >= p.target) break;
      if ((it & 63u) == 0) {
        const uint64_t t = ptx::globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > a.limit_ns) {
          atomicOr(a.status, MOE_DEVFAULT_PIPELINE_TIMEOUT);
          p.fail = late = 1;
          break;
        }
      }
    }
    __threadfence();
  }
  __syncwarp();
  int any;
  asm volatile(
      "{\n .reg .pred l, o;\n setp.ne.s32 l, %1, 0;\n bar.red.or.pred o, 2, l;\n selp.s32 %0, 1, 0, o;\n}"
      : "=r"(any)
      : "r"(late)
      : "memory");
  return any == 0;
}

// ------------------------------------------------------------------------------------------- units
// A part of the kernel (gate/up, down) is `tiles` tiles of 64 channels with K steps each. A tile is cut into
// `parts` units where there would be fewer than five for eight CTAs, and the first few units are a CTA's by its
// number, the rest go to whoever is next: SMs get up to a fifth more or less of the memory's rate than others, which
// equal shares wait for (of one token of the decode shape CTAs with equal shares were done with gate/up 35 to 48 us
// after its start). Smaller units cost more than they even
// out: with 5, 8, 12, 16 and 32 for eight CTAs one token of the decode shape took 66, 81, 79, 84 and 90 us, 16 tokens
// 419, 443, 458, 458 and 450, as every cut tile's sums go through the workspace. (Measured on that layer alone, whose 96
// and 112 tiles five for eight CTAs leaves whole; 56 of 152 SMs then have no unit of gate/up.) Which CTA took a unit
// does not matter to the result: a cut tile's units leave their sums there, and whoever brings the last one adds
// them in order.
//
// Numbers are fetched, and done units made known, by two warps of their own while the workers stream: fences and
// atomics take microseconds under load. The tiles that a CTA has to join wait for the end of its units, when all
// its warps are free for them.
struct Units {
  int K, tiles, parts, total, ahead;
  bool dealt;  // false: every slice of K has too few steps to look ahead by units, a CTA's are by its number
  __device__ Units(int K_, int tiles_, int slices, int stages) : K(K_), tiles(tiles_) {
    const int want = (kFewUnits * (int)gridDim.x / 8 + tiles - 1) / tiles;
    parts = max(1, min(want, K / (kFewSteps * slices)));
    total = tiles * parts;
    const int steps = K / parts / slices;
    dealt = steps > 0;
    ahead = 1 + (dealt ? (stages + steps - 1) / steps : 0);  // units that a warp's copies may run ahead
  }
  __device__ int begin(int q) const { return (int)((long long)q * K / parts); }
  // The i-th unit of this CTA, one that is known; total or more: there is none.
  __device__ int number(const Plan& p, int i) const {
    if (!dealt) return (long long)i * gridDim.x + blockIdx.x < total ? i * (int)gridDim.x + (int)blockIdx.x : total;
    return i < p.limit ? p.unit[i % kQueue] : total;
  }
  // By one thread, before a barrier of the CTA.
  __device__ void start(Plan& p) const {
    for (int i = 0; i <= ahead; ++i) p.unit[i] = min(total, i * (int)gridDim.x + (int)blockIdx.x);
    p.known = ahead + 1;
    p.done = 0;
    p.joined = parts > 1 ? 0 : INT_MAX;
    p.limit = INT_MAX;
    p.n_list = 0;
  }
};

// Until `now()`; past the limit the status word says so.
template <class F>
__device__ __forceinline__ bool wait_units(const FewArgs& a, Plan& p, F now) {
  const uint64_t t0 = ptx::globaltimer_ns();
  for (unsigned it = 1; !now(); ++it)
    if ((it & 63u) == 0 && (p.fail || ptx::globaltimer_ns() - t0 > 2 * a.limit_ns)) {
      atomicOr(a.status, MOE_DEVFAULT_PIPELINE_TIMEOUT);
      p.fail = 1;
      return false;
    }
  __threadfence_block();
  return true;
}

template <int W>
__device__ __forceinline__ void workers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(workers(W)) : "memory");
}
// After a unit's sums are in the workspace or its results stored, and before anything reuses their memory: the
// next units are known.
template <int W>
__device__ __forceinline__ void unit_done(const FewArgs& a, Plan& p, const Units& units, int i) {
  // the list ends where no more is known, for all workers after the same unit
  if (threadIdx.x == 0 && units.dealt &&
      !wait_units(a, p, [&] { return p.known >= i + 2 + units.ahead; }))
    p.limit = i + 1;
  workers_sync<W>();
  if (threadIdx.x == 0) {
    __threadfence_block();
    p.done = i + 1;
  }
}

// The dealer: while unit i is worked on, the number of the unit after the known ones.
__device__ void deal_units(const FewArgs& a, Plan& p, const Units& units, int* work, int lane) {
  if (!units.dealt || lane != 0) return;
  for (int i = 0; units.number(p, i) < units.total; ++i) {
    const int next = i + units.ahead + 1;  // in the place of unit i + ahead - 7, that is i - 2 or earlier
    int v = units.total;
    if (p.unit[(next - 1) % kQueue] < units.total)
      v = min(units.total, (units.ahead + 1) * (int)gridDim.x + atomicAdd(work, 1));
    if (!wait_units(a, p, [&] { return p.joined >= i - 1; })) return;
    p.unit[next % kQueue] = v;
    __threadfence_block();
    p.known = next + 1;
    if (!wait_units(a, p, [&] { return p.done > i; })) return;
  }
}

// The joiner: says that units are done, and lists the tiles that are complete with them. Past the list's end it
// joins them itself. tile_of(unit): the tile that a unit is of; join(tile, row): adds a row's parts, by a warp.
template <class Tile, class Rows, class Join>
__device__ void join_units(const FewArgs& a, Plan& p, const Units& units, int* brought, int lane, Tile tile_of,
                           Rows rows_of, Join join) {
  if (!units.dealt || units.parts == 1) return;
  for (int i = 0;; ++i) {
    int tile = -1;
    if (lane == 0) {
      const int u = units.number(p, i);
      if (u < units.total && wait_units(a, p, [&] { return p.done > i; })) {
        tile = tile_of(u);
        __threadfence();
        const bool last = atomicAdd(brought + tile, 1) == units.parts - 1;
        p.joined = i + 1;
        if (!last)
          tile = -2;
        else if (p.n_list < kList) {
          p.list[p.n_list++] = tile;
          tile = -2;
        }
      }
    }
    tile = __shfl_sync(kFull, tile, 0);
    if (tile == -1) break;
    if (tile >= 0) {
      __threadfence();
      const int2 rows = rows_of(tile);
      for (int r = rows.x; r < rows.y; ++r) join(tile, r, lane);
    }
  }
}
// After a barrier behind both: the listed tiles, rows by warps of the whole CTA.
template <class Rows, class Join>
__device__ void join_list(const Plan& p, int warp, int lane, Rows rows_of, Join join) {
  if (p.n_list == 0) return;
  __threadfence();
  for (int k = 0; k < p.n_list; ++k) {
    const int2 rows = rows_of(p.list[k]);
    for (int r = rows.x + warp; r < rows.y; r += (int)blockDim.x / 32) join(p.list[k], r, lane);
  }
}

// x may be out, which this kernel writes later, so its loads are ordinary ones (__ldg is for what no thread of the
// kernel writes).
__device__ __forceinline__ uint4 load_x(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load_x(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// ------------------------------------------------------------------------------------------ router
// hi + s exactly: the rounding error of the sum (Knuth) goes to lo.
__device__ __forceinline__ void add_exact(float& hi, float& lo, float s) {
  const float sum = hi + s, back = sum - hi;
  lo += (hi - (sum - back)) + (s - back);
  hi = sum;
}
// logits[t, e] of expert e for every token; warps share out tokens, then the pieces of d.
template <int W>
__device__ void router(const FewArgs& a, Scratch& sc, int warp, int lane) {
  int wpt = W;  // warps per token
  while (wpt > 1 && wpt * a.T > W) wpt >>= 1;
  const int part = warp % wpt, nv = a.d / 8;
  for (int e = blockIdx.x; e < a.E; e += gridDim.x) {
    for (int t = warp / wpt; warp < W && t < a.T; t += W / wpt) {
      const uint4* w = reinterpret_cast<const uint4*>(a.W_g_t + (size_t)e * a.d);
      const uint4* x = reinterpret_cast<const uint4*>(a.x + (size_t)t * a.d);
      float hi = 0.f, lo = 0.f;
#pragma unroll 4
      for (int i = part * 32 + lane; i < nv; i += wpt * 32) {
        const uint4 wv = __ldg(w + i), xv = load_x(x + i);
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
      if (lane == 0) sc.red[t * wpt + part] = make_float2(hi, lo);
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

// The plan of up to 32 slots, by one warp: lane i has slot i.
__device__ void plan_warp(const FewArgs& a, Plan& p, int lane) {
  const int n = a.T * a.k, e = lane < n ? p.idx[lane] : -1;
  const bool sound = (unsigned)e < (unsigned)a.E;
  if (lane < n && !sound && blockIdx.x == 0) atomicOr(a.status, MOE_DEVFAULT_BAD_EXPERT_INDEX);
  const unsigned below = (1u << lane) - 1u, same = __match_any_sync(kFull, sound ? e : -1 - lane);
  const int t0 = lane / a.k * a.k, rank = __popc(same & below);
  // the token's own slots of this expert, the earliest of which has the column
  const unsigned own = same & (a.k == 32 ? kFull : ((1u << a.k) - 1u) << t0);
  const bool column = sound && rank < a.C && !(own & below);
  float gate = 0.f;
  for (int j = 0; j < a.k; ++j) {
    const int s = t0 + j;
    const float w = __shfl_sync(kFull, lane < n ? p.w[lane] : 0.f, s & 31);
    if ((own >> (s & 31) & 1) && __popc(same & ((1u << (s & 31)) - 1u)) < a.C) gate += w;
  }
  const unsigned columns = __ballot_sync(kFull, column), mine = same & columns;
  const bool leader = column && !(mine & below);
  const unsigned leaders = __ballot_sync(kFull, leader);
  // in ascending order of experts, as below
  int place = 0, before = 0, total = 0;
  for (unsigned rest = leaders; rest; rest &= rest - 1) {
    const int l = __ffs(rest) - 1, other = __shfl_sync(kFull, e, l);
    const int cnt = __popc(__shfl_sync(kFull, mine, l));
    total += cnt;
    if (other < e) {
      ++place;
      before += cnt;
    }
  }
  const int shared = a.S * a.T;
  const int base = shared + before;
  if (lane < a.S) {
    p.seg_e[lane] = a.E + lane;
    p.seg_base[lane] = lane * a.T;
  }
  if (leader) {
    p.seg_e[a.S + place] = e;
    p.seg_base[a.S + place] = base;
  }
  if (column) {
    const int c = base + __popc(mine & below);
    p.tok[c] = (uint8_t)(lane / a.k);
    p.gate[c] = gate;
  }
  for (int i = lane; i < shared; i += 32) {
    p.tok[i] = (uint8_t)(i % a.T);
    p.gate[i] = 1.f;
  }
  if (lane == 0) {
    p.n_seg = a.S + __popc(leaders);
    p.seg_base[p.n_seg] = shared + total;
  }
}

// Lists the experts that were hit, shared ones first, with their columns and gates. A token that was given
// the same expert twice has one column with both gates. Of an expert's slots the first C count.
__device__ void make_plan(const FewArgs& a, Plan& p, Scratch& sc, int warp, int lane) {
  const int n = a.T * a.k, tid = threadIdx.x;
  for (int i = tid; i < a.E * (kSlots / 32); i += (int)blockDim.x) {
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
  for (int i = tid; i < a.S * a.T; i += (int)blockDim.x) {
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
      for (int i = tid; i <= a.E; i += (int)blockDim.x) ro.offsets[i] = sc.off[i];
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
// The rest of a wait for a tile that was not there at once; with_others: a wait elsewhere that gave up ends this one.
__device__ __noinline__ bool wait_long(uint32_t m, uint32_t phase, unsigned long long limit_ns, int* status,
                                       volatile int* fail, bool with_others) {
  uint64_t t0 = 0;  // the timer is slow to read: not before a tile is very late
  for (unsigned it = 1; !ptx::mbar_try_wait(m, phase); ++it) {
    if ((it & 15u) == 0 && with_others && *fail) return false;
    if ((it & 255u) == 0) {
      const uint64_t now = ptx::globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) {
        atomicOr(status, MOE_DEVFAULT_PIPELINE_TIMEOUT);
        *fail = 1;
        return false;
      }
    }
  }
  return true;
}

// A warp's ring: kStages tiles of weights (32 rows of 64 channels, 4 KB) and, for each, its lanes' pieces of the
// columns' values (32 bytes per lane and 8 columns: a value in bf16 or, for down, two). Tiles are taken in the order
// they were asked for. A tile costs a warp about a microsecond from wait to MMAs, so one of 2 KB would hold an SM
// to 30 GB/s of the 44 that it has to take.
template <int NT>
struct Ring {
  // tiles under way: with 3 and 12 workers, 4 and 10, one token of the decode shape took 70 us, with 2 and 14 66
  static constexpr int kStages = 2;
  static constexpr int kTile = 4096, kPiece = 1024 * NT;
  uint32_t w, b, bar;  // slot 0: the tile, this lane's piece, the tile's mbarrier
  int slot;            // the next tile to be taken
  uint32_t phase;
  int out;             // tiles asked for and not taken

  __device__ __forceinline__ uint32_t tile(int i) const { return w + i * kTile; }
  __device__ __forceinline__ uint32_t piece(int i) const { return b + i * kPiece; }
  __device__ __forceinline__ int later(int i) const {  // the slot i places on
    const int k = slot + i;
    return k >= kStages ? k - kStages : k;
  }
  __device__ __forceinline__ void next() {
    --out;
    if (++slot == kStages) {
      slot = 0;
      phase ^= 1u;
    }
  }
  // Until the tile and this lane's piece are there; false if a wait gave up, here or elsewhere in the CTA. The lane
  // then asks for nothing more (the caller sees to that), stays at this tile (next() comes back to it) and goes on to
  // the end of its units with what is there. Lanes need not agree on it: whatever one of them takes for a tile lies in
  // the ring, and the copies are lane 0's affair.
  __device__ __forceinline__ bool wait(const FewArgs& a, Plan& p) {
    bool there = ptx::mbar_try_wait(bar + 8 * slot, phase);
    if (!there) {
      there = wait_long(bar + 8 * slot, phase, a.limit_ns, a.status, &p.fail, true);
      if (!there) {
        ++out;
        phase ^= slot == 0;
        slot = later(kStages - 1);
      }
    }
    __syncwarp();
    cp_wait<kStages - 1>();
    return there;
  }
  // Takes what is still on its way (there is nothing unless a wait gave up), so that no copy is left that would write to
  // shared memory of a CTA that has ended. A tile gets the whole limit once more, whatever happened elsewhere; the ones
  // asked for after it have had as long.
  __device__ void drain(const FewArgs& a, Plan& p, int lane) {
    if (lane == 0)
      while (out > 0 && wait_long(bar + 8 * slot, phase, a.limit_ns, a.status, &p.fail, false)) next();
    cp_wait<0>();
    __syncwarp();
  }
  // One lane asks for a tile. What the warp read of the slot before is in registers.
  __device__ __forceinline__ void ask(int i, const CUtensorMap* map, int c, int row, int matrix) const {
    const uint32_t m = bar + 8 * i;
    ptx::mbar_arrive_expect_tx(m, kTile);
    ptx::tma_load_3d(tile(i), map, m, c, row, matrix);
  }
};

// Reads 16 rows of a tile into the fragments of four MMAs: rows of fragment j are channels 8 g + 2 j (its rows 0-7)
// and 8 g + 2 j + 1 (rows 8-15) for lane 4 g + q, whose K rows are 2 q, 2 q + 1, 2 q + 8, 2 q + 9. Swizzled: 16-byte
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
// The columns' values of 32 K rows lie so that a lane's are 16 bytes: for each q the bf16 values of rows 2 q,
// 2 q + 1, 2 q + 8, 2 q + 9 and those 16 later. x is put in that order first (its bytes are few), H is stored so.
__device__ __forceinline__ void order_x(const FewArgs& a) {
  const int n = a.T * (a.d / 8);  // uint4s
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
    const uint32_t* from = reinterpret_cast<const uint32_t*>(a.x) + (i >> 2) * 16 + (i & 3);
    reinterpret_cast<uint4*>(a.xf)[i] = make_uint4(load_x(from), load_x(from + 4), load_x(from + 8), load_x(from + 12));
  }
}

// Where a warp is in its K steps of gate/up: the CTA's i-th unit (expert, 64 channels, a part of K), step s of it.
// Of units that lie side by side in memory (channels) the numbers follow one another.
struct UpUnit {
  int seg, fb, q;
  __device__ UpUnit(int u, int nfb, int parts) {
    const int r = u / nfb;
    fb = u - r * nfb;
    seg = r / parts;
    q = r - seg * parts;
  }
};
template <int NT, int W>
struct UpFeed {
  const FewArgs& a;
  const FewMaps& maps;
  const Plan& p;
  const Units& units;
  int slice, lane, mat, i, s, kend, channel, matrix;
  const CUtensorMap* map;
  const uint4* x[NT];
  uint32_t bytes[NT];
  bool more;

  __device__ UpFeed(const FewArgs& a_, const FewMaps& m_, const Plan& p_, const Units& u_, int warp, int lane_)
      : a(a_), maps(m_), p(p_), units(u_), slice(warp >> 1), lane(lane_), mat(warp & 1), i(-1), s(0), kend(0),
        more(true) {
    settle();
  }
  // To the next unit in which this warp has a step.
  __device__ void settle() {
    while (s >= kend) {
      const int u = units.number(p, ++i);
      if (u >= units.total) {
        more = false;
        return;
      }
      const UpUnit at(u, a.f / 64, units.parts);
      s = units.begin(at.q) + slice;
      kend = units.begin(at.q + 1);
      const int e = p.seg_e[at.seg];
      map = e < a.E ? (mat ? &maps.up : &maps.gate) : (mat ? &maps.sh_up : &maps.sh_gate);
      matrix = e < a.E ? e : e - a.E;
      channel = at.fb * 64;
      const int g = lane >> 2, q = lane & 3, base = p.seg_base[at.seg], cnt = p.seg_base[at.seg + 1] - base;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bool there = g + 8 * n < cnt;
        bytes[n] = there ? 16 : 0;
        x[n] = reinterpret_cast<const uint4*>(a.xf) + (there ? p.tok[base + g + 8 * n] : 0) * (a.d / 8) + q;
      }
    }
  }
  __device__ __forceinline__ void issue(Ring<NT>& r, int slot) {
    if (more) {
      if (lane == 0) r.ask(slot, map, channel, s * 32, matrix);
      ++r.out;
#pragma unroll
      for (int n = 0; n < NT; ++n) cp_async16(r.piece(slot) + 1024 * n, x[n] + s * 4, bytes[n]);
      s += W / 2;
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

// Channels 2 k and 2 k + 1 of H in a column's row: 32 channels are 128 bytes, the values of the four q as above,
// then the remainders.
__device__ __forceinline__ void store_h(uint32_t* row, int k, float g0, float g1, float u0, float u1) {
  const float gv[2] = {g0, g1}, uv[2] = {u0, u1};
  uint32_t hi[2], lo[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float h = gv[i] / (1.f + expf(-gv[i])) * uv[i];
    const __nv_bfloat16 b = __float2bfloat16_rn(h);
    const float back = __bfloat162float(b);
    hi[i] = __bfloat16_as_ushort(b);
    // an infinite or NaN value has no remainder
    lo[i] = isfinite(back) ? __bfloat16_as_ushort(__float2bfloat16_rn(h - back)) : 0;
  }
  uint32_t* to = row + (k >> 4) * 32 + (k & 3) * 4 + (k >> 2 & 3);
  to[0] = hi[0] | hi[1] << 16;
  to[16] = lo[0] | lo[1] << 16;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }

// Sums of a gate/up unit in the workspace: [part][gate, up][column][channel].
__device__ __forceinline__ float2* up_part(const FewArgs& a, int columns, int part, int mat, int column,
                                           int channel) {
  return reinterpret_cast<float2*>(a.part + ((size_t)(part * 2 + mat) * columns + column) * a.f + channel);
}

template <int NT, int W>
__device__ void gate_up(const FewArgs& a, const FewMaps& maps, Plan& p, const Units& units, float* acc_s,
                        Ring<NT>& ring, int warp, int lane) {
  const int nfb = a.f / 64, columns = p.seg_base[p.n_seg], slice = warp >> 1;
  UpFeed<NT, W> feed(a, maps, p, units, warp, lane);
#pragma unroll
  for (int i = 0; i < Ring<NT>::kStages; ++i) feed.issue(ring, ring.later(i));
  for (int i = 0;; ++i) {
    const int u = units.number(p, i);
    if (u >= units.total) break;
    const UpUnit at(u, nfb, units.parts);
    const int base = p.seg_base[at.seg], cnt = p.seg_base[at.seg + 1] - base;
    const int k1 = units.begin(at.q + 1);
    float acc[NT][4][4] = {};
    for (int s = units.begin(at.q) + slice; s < k1; s += W / 2) {
      if (!ring.wait(a, p)) feed.more = false;
      const uint32_t tile = ring.tile(ring.slot);
      uint32_t f[2][4][4];
      fragments(tile, lane, f[0]);
      fragments(tile + 2048, lane, f[1]);
      uint4 b[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) b[n] = lds16(ring.piece(ring.slot) + 1024 * n);
      __syncwarp();
      const int slot = ring.slot;
      ring.next();
      feed.issue(ring, slot);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n == 0 || cnt > 8) {
#pragma unroll
          for (int m = 0; m < 4; ++m) mma(acc[n][m], f[0][m], b[n].x, b[n].y);
#pragma unroll
          for (int m = 0; m < 4; ++m) mma(acc[n][m], f[1][m], b[n].z, b[n].w);
        }
    }
    store_sums<NT>(acc_s + warp * (8 * NT) * kAccLd, acc, cnt, lane);
    workers_sync<W>();
    for (int k = threadIdx.x; k < cnt * 32; k += workers(W)) {
      const int c = k >> 5, pair = k & 31;
      float2 g = make_float2(0.f, 0.f), v = g;
#pragma unroll
      for (int w = 0; w < W; w += 2) {
        const float* row = acc_s + (w * (8 * NT) + c) * kAccLd + 2 * pair;
        g = add2(g, *reinterpret_cast<const float2*>(row));
        v = add2(v, *reinterpret_cast<const float2*>(row + (8 * NT) * kAccLd));
      }
      if (units.parts == 1) {
        store_h(a.h + (size_t)(base + c) * a.f, at.fb * 32 + pair, g.x, g.y, v.x, v.y);
      } else {
        *up_part(a, columns, at.q, 0, base + c, at.fb * 64 + 2 * pair) = g;
        *up_part(a, columns, at.q, 1, base + c, at.fb * 64 + 2 * pair) = v;
      }
    }
    unit_done<W>(a, p, units, i);
  }
  ring.drain(a, p, lane);
}

// The parts of a column of a tile of gate/up added up, a lane two channels.
__device__ __forceinline__ void join_up(const FewArgs& a, const Plan& p, const Units& units, int fb, int c,
                                        int lane) {
  const int columns = p.seg_base[p.n_seg];
  float2 g = make_float2(0.f, 0.f), u = g;
#pragma unroll 8
  for (int q = 0; q < units.parts; ++q) {
    g = add2(g, __ldcg(up_part(a, columns, q, 0, c, fb * 64 + 2 * lane)));
    u = add2(u, __ldcg(up_part(a, columns, q, 1, c, fb * 64 + 2 * lane)));
  }
  store_h(a.h + (size_t)c * a.f, fb * 32 + lane, g.x, g.y, u.x, u.y);
}

// Where a warp is in its K steps of down: the CTA's i-th unit (64 channels, a part of all experts' channels in a
// row), step s of it.
template <int NT, int W>
struct DownFeed {
  const FewArgs& a;
  const FewMaps& maps;
  const Plan& p;
  const Units& units;
  int slice, lane, fs, i, s, kend, seg, channel, matrix;
  const CUtensorMap* map;
  const uint4* h[NT];
  uint32_t bytes[NT];
  bool more;

  __device__ DownFeed(const FewArgs& a_, const FewMaps& m_, const Plan& p_, const Units& u_, int warp, int lane_)
      : a(a_), maps(m_), p(p_), units(u_), slice(warp), lane(lane_), fs(a_.f / 32), i(-1), s(0), kend(0),
        more(true) {
    settle();
  }
  __device__ void expert() {
    seg = s / fs;
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
      const int u = units.number(p, ++i);
      if (u >= units.total) {
        more = false;
        return;
      }
      const int q = u / units.tiles;
      channel = (u - q * units.tiles) * 64;
      s = units.begin(q) + slice;
      kend = units.begin(q + 1);
    }
    expert();
  }
  __device__ __forceinline__ void issue_w(Ring<NT>& r, int slot) const {
    if (!more) return;
    if (lane == 0) r.ask(slot, map, channel, (s - seg * fs) * 32, matrix);
    ++r.out;
  }
  __device__ __forceinline__ void issue_h(const Ring<NT>& r, int slot) const {
    if (more) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        cp_async16(r.piece(slot) + 1024 * n, h[n] + (s - seg * fs) * 8, bytes[n]);
        cp_async16(r.piece(slot) + 1024 * n + 512, h[n] + (s - seg * fs) * 8 + 4, bytes[n]);
      }
    }
    cp_commit();
  }
  __device__ __forceinline__ void next() {
    if (!more) return;
    s += W;
    if (s >= kend)
      settle();
    else if (s >= (seg + 1) * fs)
      expert();
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

__device__ __forceinline__ uint32_t bf16x2(float2 v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void store_out(const FewArgs& a, int t, int channel, float2 v) {
  *reinterpret_cast<uint32_t*>(a.out + (size_t)t * a.d + channel) = bf16x2(v);
}
// Sums of a down unit in the workspace: [part][token][channel].
__device__ __forceinline__ float2* down_part(const FewArgs& a, int part, int t, int channel) {
  return reinterpret_cast<float2*>(a.part + ((size_t)part * a.T + t) * a.d + channel);
}

// The first weights, which need nothing of the other CTAs: they are on their way while those finish H.
template <int NT, int W>
__device__ void down_ahead(const DownFeed<NT, W>& feed, Ring<NT>& ring) {
  DownFeed<NT, W> ahead = feed;
#pragma unroll
  for (int i = 0; i < Ring<NT>::kStages; ++i) {
    ahead.issue_w(ring, ring.later(i));
    ahead.next();
  }
}

template <int NT, int W>
__device__ void down(const FewArgs& a, Plan& p, const Units& units, DownFeed<NT, W>& feed, float* acc_s,
                     Ring<NT>& ring, int warp, int lane) {
  const int fs = a.f / 32;
  float* mine = acc_s + warp * (8 * NT) * kAccLd;
#pragma unroll
  for (int i = 0; i < Ring<NT>::kStages; ++i) {
    feed.issue_h(ring, ring.later(i));
    feed.next();
  }
  for (int i = 0;; ++i) {
    const int u = units.number(p, i);
    if (u >= units.total) break;
    const int q = u / units.tiles, channel = (u - q * units.tiles) * 64, k1 = units.begin(q + 1);
    for (int k = lane; k < a.T * kAccLd; k += 32) mine[k] = 0.f;
    __syncwarp();
    float acc[NT][4][4] = {};
    int seg = 0, cnt = 0, seg_end = 0;
    for (int s = units.begin(q) + warp; s < k1; s += W) {
      if (s >= seg_end) {
        if (seg_end > 0) add_sums<NT>(mine, acc, p, seg, lane);
        seg = s / fs;
        seg_end = (seg + 1) * fs;
        cnt = p.seg_base[seg + 1] - p.seg_base[seg];
      }
      if (!ring.wait(a, p)) feed.more = false;
      const uint32_t tile = ring.tile(ring.slot);
      uint32_t f[2][4][4];
      fragments(tile, lane, f[0]);
      fragments(tile + 2048, lane, f[1]);
      uint4 b[NT], lo[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        b[n] = lds16(ring.piece(ring.slot) + 1024 * n);
        lo[n] = lds16(ring.piece(ring.slot) + 1024 * n + 512);
      }
      __syncwarp();
      const int slot = ring.slot;
      ring.next();
      feed.issue_w(ring, slot);
      feed.issue_h(ring, slot);
      feed.next();
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n == 0 || cnt > 8) {
#pragma unroll
          for (int m = 0; m < 4; ++m) mma(acc[n][m], f[0][m], b[n].x, b[n].y);
#pragma unroll
          for (int m = 0; m < 4; ++m) mma(acc[n][m], f[1][m], b[n].z, b[n].w);
#pragma unroll
          for (int m = 0; m < 4; ++m) mma(acc[n][m], f[0][m], lo[n].x, lo[n].y);
#pragma unroll
          for (int m = 0; m < 4; ++m) mma(acc[n][m], f[1][m], lo[n].z, lo[n].w);
        }
    }
    if (seg_end > 0) add_sums<NT>(mine, acc, p, seg, lane);
    workers_sync<W>();
    for (int k = threadIdx.x; k < a.T * 32; k += workers(W)) {
      const int t = k >> 5, pair = k & 31;
      float2 v = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w)
        v = add2(v, *reinterpret_cast<const float2*>(acc_s + (w * (8 * NT) + t) * kAccLd + 2 * pair));
      if (units.parts == 1)
        store_out(a, t, channel + 2 * pair, v);
      else
        *down_part(a, q, t, channel + 2 * pair) = v;
    }
    unit_done<W>(a, p, units, i);
  }
  ring.drain(a, p, lane);
}

// The parts of a token's channels of a tile of down added up, a lane two.
__device__ __forceinline__ void join_down(const FewArgs& a, const Units& units, int tile, int t, int lane) {
  float2 v = make_float2(0.f, 0.f);
#pragma unroll 8
  for (int q = 0; q < units.parts; ++q) v = add2(v, __ldcg(down_part(a, q, t, tile * 64 + 2 * lane)));
  store_out(a, t, tile * 64 + 2 * lane, v);
}

template <int NT, int W>
constexpr int ring_bytes() {
  return W * Ring<NT>::kStages * (Ring<NT>::kTile + Ring<NT>::kPiece);
}
template <int NT, int W>
constexpr int smem_bytes() {
  return 1024 + ring_bytes<NT, W>() + W * 8 * NT * kAccLd * 4;  // 1024: swizzled tiles' alignment
}

template <int NT, int W>
__global__ void __launch_bounds__(threads(W), 1)
    few_kernel(const __grid_constant__ FewArgs a, const __grid_constant__ FewMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Plan p;
  __shared__ __align__(8) uint64_t bars[W][Ring<NT>::kStages];
  uint8_t* smem = smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Scratch& sc = *reinterpret_cast<Scratch*>(smem);
  static_assert(sizeof(Scratch) <= ring_bytes<NT, W>(), "it lies in the ring");
  float* acc_s = reinterpret_cast<float*>(smem + ring_bytes<NT, W>());
  Ring<NT> ring;
  ring.w = ptx::smem_u32(smem) + warp * Ring<NT>::kStages * ring.kTile;
  ring.b = ptx::smem_u32(smem) + W * Ring<NT>::kStages * ring.kTile + warp * Ring<NT>::kStages * ring.kPiece + lane * 16;
  ring.bar = ptx::smem_u32(&bars[warp][0]);
  ring.slot = 0;
  ring.phase = 0;
  ring.out = 0;
  if (warp < W && lane == 0) {
    for (int i = 0; i < Ring<NT>::kStages; ++i)
      ptx::mbar_init(ring.bar + 8 * i, a.withheld && i + warp + blockIdx.x == 0 ? 2 : 1);
    ptx::fence_mbarrier_init();
  }
  if (threadIdx.x == threads(W) - 1) {
    ptx::prefetch_tmap(&maps.gate);
    ptx::prefetch_tmap(&maps.up);
    ptx::prefetch_tmap(&maps.down);
    if (a.S > 0) {
      ptx::prefetch_tmap(&maps.sh_gate);
      ptx::prefetch_tmap(&maps.sh_up);
      ptx::prefetch_tmap(&maps.sh_down);
    }
  }
  if (threadIdx.x == 0) p.fail = 0;
  // the units' counters: work and brought of gate/up, then of down
  constexpr int kMostTiles = kFewUnits * kFewMaxCtas / 8;
  for (int i = blockIdx.x * threads(W) + threadIdx.x; i < 2 * (1 + kMostTiles); i += gridDim.x * threads(W))
    a.count[i] = 0;
  order_x(a);
  if (a.W_g_t != nullptr) {
    router<W>(a, sc, warp, lane);
    barrier_arrive(a, p);
    if (!barrier_wait(a, p)) return;
    for (int t = warp; t < a.T; t += threads(W) / 32) choose(a, p, sc.score[t], t, lane);
  } else {
    barrier_arrive(a, p);
    for (int i = threadIdx.x; i < a.T * a.k; i += threads(W)) {
      p.idx[i] = __ldg(a.idx_in + i);
      p.w[i] = a.w_in != nullptr ? __ldg(a.w_in + i) : 1.f;
    }
  }
  __syncthreads();
  const moe_route_out& ro = a.ro;
  if (a.T * a.k <= 32 && !(ro.counts || ro.offsets || ro.perm_slot || ro.slot_pos)) {
    if (warp == 0) {
      plan_warp(a, p, lane);
    } else if (warp == 1 && blockIdx.x == 0 && lane < a.T * a.k) {
      if (ro.topk_idx) ro.topk_idx[lane] = p.idx[lane];
      if (ro.topk_w) ro.topk_w[lane] = p.w[lane];
    }
    __syncthreads();
  } else {
    make_plan(a, p, sc, warp, lane);
  }
  if (a.W_g_t == nullptr && !barrier_wait(a, p)) return;
  if (p.n_seg == 0) {  // not one sound index
    for (int i = blockIdx.x * threads(W) + threadIdx.x; i < a.T * a.d / 4; i += gridDim.x * threads(W))
      reinterpret_cast<uint2*>(a.out)[i] = make_uint2(0u, 0u);
    return;
  }
  ptx::fence_proxy_async_smem();  // the scratch gives way to tiles that TMA writes
  const Units up(a.d / 32, p.n_seg * (a.f / 64), W / 2, Ring<NT>::kStages);
  if (threadIdx.x == 0) up.start(p);
  __syncthreads();
  {
    const int nfb = a.f / 64;
    const auto rows = [&](int tile) {
      const int seg = tile / nfb;
      return make_int2(p.seg_base[seg], p.seg_base[seg + 1]);
    };
    const auto join = [&](int tile, int c, int l) { join_up(a, p, up, tile % nfb, c, l); };
    if (warp < W)
      gate_up<NT, W>(a, maps, p, up, acc_s, ring, warp, lane);
    else if (warp == W)
      deal_units(a, p, up, a.count, lane);
    else
      join_units(a, p, up, a.count + 1, lane,
                 [&](int u) {
                   const UpUnit at(u, nfb, up.parts);
                   return at.seg * nfb + at.fb;
                 },
                 rows, join);
    __syncthreads();
    join_list(p, warp, lane, rows, join);
    __syncthreads();
  }
  const Units dn(p.n_seg * (a.f / 32), a.d / 64, W, Ring<NT>::kStages);
  if (threadIdx.x == 0) dn.start(p);
  barrier_arrive(a, p);
  int* count = a.count + 1 + kMostTiles;
  const auto rows = [&](int) { return make_int2(0, a.T); };
  const auto join = [&](int tile, int t, int l) { join_down(a, dn, tile, t, l); };
  // Where a wait of this CTA has given up before, or does so here, the workers take the copies under way and that is
  // all.
  if (warp < W) {
    DownFeed<NT, W> feed(a, maps, p, dn, warp, lane);
    if (__any_sync(kFull, p.fail)) feed.more = false;
    down_ahead(feed, ring);
    if (barrier_wait(a, p))
      down<NT, W>(a, p, dn, feed, acc_s, ring, warp, lane);
    else
      ring.drain(a, p, lane);
  } else if (barrier_wait(a, p)) {
    if (warp == W)
      deal_units(a, p, dn, count, lane);
    else
      join_units(a, p, dn, count + 1, lane, [&](int u) { return u % dn.tiles; }, rows, join);
  }
  __syncthreads();
  join_list(p, warp, lane, rows, join);
}

template <int NT, int W>
cudaError_t launch(const FewArgs& a, const FewMaps& maps, cudaStream_t st) {
  constexpr int smem = smem_bytes<NT, W>();
  cudaError_t e = cudaFuncSetAttribute(few_kernel<NT, W>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms() < kFewMaxCtas ? num_sms() : kFewMaxCtas);
  cfg.blockDim = dim3(threads(W));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_kernel<NT, W>, a, maps);
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
  L.xf = take(2ull * s.T * s.d);
  L.h = take(4ull * s.T * (s.k + s.S) * s.f);
  // counters of units, and the parts of cut tiles. A tile is cut into at most one part more than the most units
  // are times the number of tiles: of gate/up one for 64 channels of an expert, of down for 64 of d
  constexpr size_t units = kFewUnits * kFewMaxCtas / 8;
  L.count = take(4 * 2 * (1 + units));
  const size_t up = 2 * (64 * units * s.T + (size_t)s.T * (s.k + s.S) * s.f);
  const size_t down = s.T * (64 * units + s.d);
  L.part = take(4 * (up > down ? up : down));
  L.wg_t = take(2ull * s.d * s.E);
  L.total = o;
  return L;
}

cudaError_t launch_few(const FewArgs& a, cudaStream_t st) {
  FewMaps maps = {};
  const auto map = [&](CUtensorMap& m, const uint16_t* w, int n, int rows, int cols) {
    return make_tmap_3d(&m, w, n, rows, cols, 64, 32, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, false);
  };
  bool ok = map(maps.gate, a.gate, a.E, a.d, a.f) && map(maps.up, a.up, a.E, a.d, a.f) &&
            map(maps.down, a.down, a.E, a.f, a.d);
  if (a.S > 0)
    ok = ok && map(maps.sh_gate, a.sh_gate, a.S, a.d, a.f) && map(maps.sh_up, a.sh_up, a.S, a.d, a.f) &&
         map(maps.sh_down, a.sh_down, a.S, a.f, a.d);
  if (!ok) return cudaErrorInvalidValue;
  // Up to eight tokens an expert has one group of eight columns at most; a second one's slots of the ring leave room
  // for 12 workers. 16 workers and the two others would leave a thread 96 registers: it spilled, and one token of the
  // decode shape took 80 us instead of 66 with 14 or 12. With 14 nothing is spilled; the form for two groups, whose
  // sums are 32 registers, spills about 80 bytes of a thread with its 128 (16 tokens: HBM all the same).
  return a.T <= 8 ? launch<1, 14>(a, maps, st) : launch<2, 12>(a, maps, st);
}

}  // namespace moe
