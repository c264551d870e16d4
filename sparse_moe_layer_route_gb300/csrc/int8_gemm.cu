// Grouped products of 8-bit integers over row segments, with a scale per row and per output channel,
// on the 5th-generation tensor cores.
//
//   D[channel, row] = sum_k qw[channel, k] * xq[row, k],  out[row, channel] = D * sx[row] * sw[channel]
//
// sm_103a's 8-bit integer tensor rate is far below its 16-bit one, so the codes are multiplied as fp16:
// whole numbers up to 128 are exact there, their products are exact, and fp32 sums of them are exact
// below 2^24. The weights stay 8-bit in memory and in shared memory; they are widened on the way to the
// MMA, whose A operand they are (M = 256 output channels of a pair of CTAs) out of tensor memory. That costs
// no shared-memory writes and leaves the 16-bit B operand (the rows, widened once per call) as the only
// matrix the MMA reads from shared memory.
//
// With one CTA a tile's operand traffic through shared memory (weight codes in and out, rows in, and
// read by the MMA) takes longer than its MMAs: (64 / N + 0.75) of their time for two 128-channel tiles
// x N rows, 1.25 at N = 128. Here each CTA of a pair (a cluster of two) widens 128 channels into its own
// tensor memory but stages only half of the rows, which the MMA reads once for both: 40 KB per 64 k against
// 49 KB of shared-memory bandwidth in the 384 clk that N = 192 takes, and half the widening per MMA.
//
// Long segments are bound by the tensor cores or, in low tiles, by the widening; short ones by the weight
// bytes: 128 experts and a shared one of d 7168, d_ff 2048 for 64 tokens 492 to 536 us a call from run to run
// (7.4 to 6.8 TB/s; the two quantizations of rows are about 5 of it). 16384 rows of [4096 x 7168] in 482 us in short
// runs (2.0 PFLOP/s, 1.05 of the measured bf16 peak); a long run settles at the power cap: 535, 581 with the
// widening of the rows in front. A 64 k slot takes 2 clk of MMA a row; widening it takes one set of warps
// 776, so two sets keep up with 194 rows and three with 130: a lower tile is bound by the widening.
//
// A unit is 256 channels (SwiGLU pass: 128 channels of gate and up) x a row tile of one segment
// (int8_tile_height). Rank r of a pair holds channels [128 r, 128 r + 128) and rows [n / 2 * r, n / 2 *
// (r + 1)) of the n rows the MMA takes (the unit's rows rounded up to 32). SwiGLU pass: rank r holds 64
// channels; TMEM lanes 32 w + l, l < 16, hold the gate codes of channel 16 w + l and lanes 32 w + 16 + l the
// up codes, so that a warp's epilogue swaps halves by shuffles. Roles per CTA:
//   warp 0       TMA producer of codes: the CTA's 128 code rows x 128 B a step (128 k)
//   warp 1       MMA issuer (rank 0). It and the producers run in an elected lane: issued under `lane == 0`, an
//                MMA costs 75 clk, so 27
//   warp 2       TMEM allocator: ACOLS columns of accumulators, NSLOT 64-column slots of widened codes
//   warp 3       TMA producer of rows: two [n / 2 rows x 64 k] fp16 tiles a step, 32 rows a copy
//   warps 4-7    epilogue, overlapping the next unit's MMAs
//   warps 8-     widen, in SETS of four warps: the half-steps (64 k) of all units go to the sets in turn
// The MMA issuer's barrier operations are few, because one behind a commit costs it about 300 clk, with or
// without something to wait for: per 128 k it waits once (`ready`: both CTAs' rows have landed and the
// eight warps of each that widen the step have stored) and commits once (`done`, to both CTAs), and `done`
// frees the rows' stage and, with it, the slot of widened codes. (With a wait and a commit for each 64 k slot and each stage, a 64 k
// slot took 480 clk whatever its N.) The codes' stage is free once they are in registers (`taken`): they come
// from HBM and need the longer run-up (64 segments of 128 rows of [2048 x 2048] 83 us with four stages of
// both together, 77 apart).
// The accumulators of consecutive units begin at opposite ends of the ACOLS columns, so two tiles whose
// rows add up to ACOLS overlap fully. Where they add up to more, the second one's MMAs wait (`inner`) until
// the epilogue has read the columns that they share, which it does first.
// Three sets (640 threads: 96 registers each at launch, then 80 for the widening warps and 144 for the
// epilogue) against two: 48 tokens an expert, 148 against 154 us for the experts of d 2048, d_ff 1408;
// 16384 rows of [4096 x 7168] 1 to 3 % less. The slot pass of tall tiles keeps two: its units are short (11
// steps at K = 1408), its epilogue nearly as long as its MMAs, and a third set takes issue slots from it (132
// against 139 us).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "int8.cuh"
#include "int8_units.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kABytes = kInt8Ch * kInt8StageK;  // 16 KB of codes
constexpr int kBoxRows = 32;                    // rows of one copy

// Tiles of up to NT rows; two accumulators in ACOLS TMEM columns, NSLOT slots of 64 for widened codes; SA
// and SB stages of codes and of rows; SETS of four widening warps.
template <int NT_, int ACOLS_, int NSLOT_, int SA_, int SB_, int SETS_>
struct Cfg {
  static constexpr int SETS = SETS_, kThreads = 256 + 128 * SETS;
  static constexpr int NT = NT_, ACOLS = ACOLS_, NSLOT = NSLOT_, SA = SA_, SB = SB_;
  static constexpr int kBSub = NT / 2 * 128;  // one [NT / 2 rows x 64 k] fp16 tile
  static constexpr int kRows = SA * kABytes;  // where the rows' stages begin
  static constexpr int kPipeBytes = kRows + SB * 2 * kBSub;
  static constexpr int kSlotCol = ACOLS;  // first TMEM column of the widened codes
  static constexpr int kBars = 2 * SA + 2 * SB + 6, kBarBytes = 512;
  static constexpr int kSmemBytes =
      kPipeBytes + 2 * kInt8StepBytes + 1024 /*align*/ + kBarBytes;
  static_assert(kSlotCol + NSLOT * 64 <= 512, "TMEM columns");
  static_assert(SA >= NSLOT + 2 && SB >= 2, "a set that passes over steps finds each phase");
  static_assert(NSLOT <= SB, "a slot's last step is known by its rows' stage's barrier");
  static_assert(kBSub % 1024 == 0 && NT % (2 * kBoxRows) == 0, "swizzle atoms; whole copies");
  static_assert(NT <= 256 && ACOLS >= NT, "N of an MMA; a tile's accumulator");
  static_assert(8 * kBars + 8 <= kBarBytes, "barrier block");
};

template <int PASS, int OUT, typename C>
__global__ void __launch_bounds__(C::kThreads, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tmB,
                          const __grid_constant__ CUtensorMap tmA,
                          const __grid_constant__ CUtensorMap tmA2,
                          const __grid_constant__ CUtensorMap tmShA,
                          const __grid_constant__ CUtensorMap tmShA2, const Int8Gemm g) {
  constexpr bool GLU = PASS == kInt8SwiGLU;
  constexpr int UCH = GLU ? 128 : 256;  // output channels per unit
  constexpr int kNT = C::NT, kSA = C::SA, kSB = C::SB, kBSub = C::kBSub;

  extern __shared__ uint8_t smem_raw[];
  __shared__ SegTable segs;
  __shared__ __align__(16) float unit_sx[2][kNT];  // row scales, output rows of the epilogue's unit
  __shared__ int unit_orow[2][kNT];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  uint8_t* const stage_out = gbase + C::kPipeBytes;  // the epilogue's two steps
  const uint32_t bar0 = base + C::kPipeBytes + 2 * kInt8StepBytes;
  auto codes_bar = [&](int s) { return bar0 + 8u * s; };                   // own codes have landed
  auto taken_bar = [&](int s) { return bar0 + 8u * (kSA + s); };           // and are in registers
  auto ready_bar = [&](int s) { return bar0 + 8u * (2 * kSA + s); };       // rank 0: see above
  auto done_bar = [&](int s) { return bar0 + 8u * (2 * kSA + kSB + s); };  // the step's MMAs are done
  const uint32_t bar1 = bar0 + 8u * (2 * kSA + 2 * kSB);
  auto dfull_bar = [&](int b) { return bar1 + 8u * b; };
  auto dempty_bar = [&](int b) { return bar1 + 8u * (2 + b); };  // rank 0
  const uint32_t inner_bar = bar1 + 8u * 4;                      // rank 0: see above
  const uint32_t mma_done_bar = bar0 + 8u * (C::kBars - 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(stage_out + 2 * kInt8StepBytes + 8 * C::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_rank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSA; ++s) {
      ptx::mbar_init(codes_bar(s), 1);
      ptx::mbar_init(taken_bar(s), 8);  // the step's widening warps
    }
    for (int s = 0; s < kSB; ++s) {
      ptx::mbar_init(ready_bar(s), 17);  // rows (with their bytes), eight widening warps of each CTA
      ptx::mbar_init(done_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(dfull_bar(b), 1);
      ptx::mbar_init(dempty_bar(b), 8);  // four epilogue warps of each CTA
    }
    ptx::mbar_init(inner_bar, 8);
    ptx::mbar_init(mma_done_bar, 1);
    *abort_flag = 0;
    ptx::fence_mbarrier_init();
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
    if (GLU) ptx::prefetch_tmap(&tmA2);
  }
  if (warp == 2) {
    ptx::tmem_alloc_cg2(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish_cg2();
  }
  griddep_wait();  // everything above touched only shared memory, TMEM and parameters
  build_segments<PASS>(segs, g, min(g.tile_rows, kNT));
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // the peer's barriers are initialised
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int n_ct = (g.N + UCH - 1) / UCH;
  const int n_sub = (g.K + 63) / 64;
  const int n_step = (n_sub + 1) / 2;
  // partial pass: a unit is done in pieces, each some of its steps
  const int splits = PASS == kInt8Partial ? g.splits : 1;
  const long long total = (long long)segs.first[g.n_mat + g.S] * n_ct * splits;
  auto unit_of = [&](long long w) {
    return find_unit<GLU>(segs, g, n_ct, PASS == kInt8Partial ? w / splits : w);
  };
  auto first_step = [&](long long w) {
    return PASS == kInt8Partial ? (int)(w % splits) * n_step / splits : 0;
  };
  auto end_step = [&](long long w) {
    return PASS == kInt8Partial ? ((int)(w % splits) + 1) * n_step / splits : n_step;
  };
  const long long pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  auto mma_rows = [](const Unit& u) { return (u.rows + 31) & ~31; };
  // first column of the accumulator of a unit: even ones begin at the low end, odd ones end at the high
  auto acc_col = [](int acc, int n) { return acc == 0 ? 0 : C::ACOLS - n; };
  // columns that a unit shares with the one before it (a multiple of 32)
  auto shared_cols = [](int n, int n_before) { return max(0, n + n_before - C::ACOLS); };

  if (warp == 0) {
    if (ptx::elect_one()) {
      // ---------------------------------------------------------------- TMA producer of codes (both)
      int stage = 0;
      uint32_t phase = 0, issued = 0, last_parity = 0;  // per stage: ever issued, its parity
      bool ok = true;
      for (long long w = pair; w < total && ok; w += n_pairs) {
        const Unit u = unit_of(w);
        const bool sh = u.seg >= g.n_mat;
        const int ex = sh ? u.seg - g.n_mat : u.seg;
        const CUtensorMap* a0 = sh ? &tmShA : &tmA;
        const CUtensorMap* a1 = GLU ? (sh ? &tmShA2 : &tmA2) : a0;
        const int ch0 = u.ct * UCH + (int)rank * (UCH / 2), ch1 = GLU ? ch0 : ch0 + 64;
        const int i1 = end_step(w);
        for (int i = first_step(w); i < i1; ++i) {
          if (!ptx::mbar_wait_bounded(taken_bar(stage), phase ^ 1u, abort_flag, g.status,
                                      MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs)) {
            ok = false;
            break;
          }
          const uint32_t sA = base + stage * kABytes, cb = codes_bar(stage);
          ptx::mbar_arrive_expect_tx(cb, kABytes);
          ptx::tma_load_3d(sA, a0, cb, i * kInt8StageK, ch0, ex);
          ptx::tma_load_3d(sA + kABytes / 2, a1, cb, i * kInt8StageK, ch1, ex);
          issued |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == kSA) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // never leave while a copy into this CTA's shared memory may still be in flight
      for (int s = 0; s < kSA; ++s)
        if (issued & (1u << s)) {
          volatile int no_abort = 0;
          ptx::mbar_wait_bounded(codes_bar(s), (last_parity >> s) & 1u, &no_abort, g.status,
                                 MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs / 4);
        }
    }
    __syncwarp();
  } else if (warp == 3) {
    if (ptx::elect_one()) {
      // ---------------------------------------------------------------- TMA producer of rows (both)
      int stage = 0;
      uint32_t phase = 0, issued = 0, last_parity = 0;
      bool ok = true;
      for (long long w = pair; w < total && ok; w += n_pairs) {
        const Unit u = unit_of(w);
        const int half_rows = mma_rows(u) / 2;  // of each CTA
        const int brow = u.brow0 + (int)rank * half_rows;
        const int boxes = (half_rows + kBoxRows - 1) / kBoxRows;
        const int i1 = end_step(w);
        for (int i = first_step(w); i < i1; ++i) {
          if (!ptx::mbar_wait_bounded(done_bar(stage), phase ^ 1u, abort_flag, g.status,
                                      MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs)) {
            ok = false;
            break;
          }
          const uint32_t sB = base + C::kRows + stage * (2 * kBSub);
          const uint32_t rb = leader ? ready_bar(stage) : ptx::mapa_shared(ready_bar(stage), 0);
          const bool half = 2 * i + 1 < n_sub;  // the step's second 64 k hold something
          if (leader) ptx::mbar_arrive_expect_tx(rb, (half ? 4 : 2) * boxes * (kBoxRows * 128));
          for (int b = 0; b < boxes; ++b) {
            const uint32_t to = sB + b * (kBoxRows * 128);
            ptx::tma_load_2d_cg2(to, &tmB, rb, i * kInt8StageK, brow + b * kBoxRows);
            if (half)
              ptx::tma_load_2d_cg2(to + kBSub, &tmB, rb, i * kInt8StageK + 64, brow + b * kBoxRows);
          }
          issued |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == kSB) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // the same for the rows. Their barrier also counts the widening warps, so after an abort it may not
      // complete: then the wait runs out
      for (int s = 0; s < kSB; ++s)
        if (issued & (1u << s)) {
          volatile int no_abort = 0;
          ptx::mbar_wait_bounded(done_bar(s), (last_parity >> s) & 1u, &no_abort, g.status,
                                 MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs / 4);
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader && ptx::elect_one()) {
      // ---------------------------------------------------------------- MMA issuer (rank 0)
      int stage = 0, slot = 0, acc = 0, n_before = 0;
      uint32_t phase = 0, acc_phase = 0, inner_phase = 0;
      bool ok = true;
      for (long long w = pair; w < total && ok; w += n_pairs) {
        const int n = mma_rows(unit_of(w));
        const uint32_t idesc = ptx::idesc_f16kind_f32(256, (uint32_t)n, 0, 0, 0u);
        if (!ptx::mbar_wait_bounded(dempty_bar(acc), acc_phase ^ 1u, abort_flag, g.status,
                                    MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs))
          break;
        if (shared_cols(n, n_before) > 0) {
          if (!ptx::mbar_wait_bounded(inner_bar, inner_phase, abort_flag, g.status,
                                      MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs))
            break;
          inner_phase ^= 1u;
        }
        n_before = n;
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)acc_col(acc, n);
        const int i0 = first_step(w), i1 = end_step(w);
        for (int i = i0; i < i1; ++i) {
          if (!ptx::mbar_wait_bounded(ready_bar(stage), phase, abort_flag, g.status,
                                      MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t a = tmem_base + C::kSlotCol + slot * 64;
          // rows: K-major, 128 B each, 8-row groups 1024 B apart; a K step of 16 = +32 B
          const uint64_t bd =
              ptx::smem_desc_sw128(base + C::kRows + stage * (2 * kBSub), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::umma_f16_ta_cg2(d, a + kk * 8, bd + (uint64_t)(kk * 2), idesc,
                                 ((i - i0) | kk) != 0 ? 1u : 0u);
          if (2 * i + 1 < n_sub) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              ptx::umma_f16_ta_cg2(d, a + 32 + kk * 8, bd + (uint64_t)((kBSub >> 4) + kk * 2),
                                   idesc, 1u);
          }
          ptx::umma_commit_cg2(done_bar(stage), 0x3);
          if (++slot == C::NSLOT) slot = 0;
          if (++stage == kSB) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::umma_commit_cg2(dfull_bar(acc), 0x3);
        acc_phase ^= (uint32_t)acc;
        acc ^= 1;
      }
      // all MMAs issued by this thread have finished before TMEM is released
      ptx::umma_commit_cg2(mma_done_bar, 0x1);
      volatile int no_abort = 0;
      ptx::mbar_wait_bounded(mma_done_bar, 0, &no_abort, g.status,
                                     MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs / 4);
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ widening warps (both)
    const int set = (warp - 8) >> 2, q = warp & 3;  // TMEM lanes [32 q, 32 q + 32)
    const int row = GLU ? 16 * q + (lane & 15) + 64 * (lane >> 4) : 32 * q + lane;
    if constexpr (C::SETS == 3) ptx::setmaxnreg_dec<80>();
    // half-steps of 64 k, numbered through all units, go to the sets in turn. A set passes over steps of the
    // others, but each barrier's earlier phase is over when it looks: its last step, at most two before this
    // one, had all but NSLOT of the steps before it done, and SA >= NSLOT + 2
    uint32_t step = 0;           // step of this set's half-step, and of it:
    int h = set;                 // the half
    int stage = 0, slot = 0;     // the stage of the codes; the slot of the widened ones
    int bstage = 0, dstage = 0;  // the rows' stage, and that of the step NSLOT before it
    uint32_t phase = 0, dphase = 0;
    long long w = pair;
    int i = w < total ? first_step(w) : 0, i1 = w < total ? end_step(w) : 0;
    auto next_step = [&] {
      if (++slot == C::NSLOT) slot = 0;
      if (++bstage == kSB) bstage = 0;
      if (++stage == kSA) {
        stage = 0;
        phase ^= 1u;
      }
      if (step >= (uint32_t)C::NSLOT && ++dstage == kSB) {
        dstage = 0;
        dphase ^= 1u;
      }
      ++step;
      if (++i == i1) {
        w += n_pairs;
        if (w < total) {
          i = first_step(w);
          i1 = end_step(w);
        }
      }
    };
    if (C::SETS == 3 && h == 2) {
      if (w < total) next_step();
      h = 0;
    }
    while (w < total) {
      if (!ptx::mbar_wait_bounded_warp(codes_bar(stage), phase, abort_flag, g.status,
                                       MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs))
        break;
      const bool on = 2 * i + h < n_sub;
      uint32_t r[32];
      if (on) {
        const uint8_t* src = gbase + stage * kABytes + row * kInt8StageK;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          // 16-byte piece 4 h + c of the row sits at piece (4 h + c) ^ (row mod 8)
          const uint4 v = *reinterpret_cast<const uint4*>(src + (((4 * h + c) ^ (row & 7)) << 4));
          widen4(v.x, r[8 * c], r[8 * c + 1]);
          widen4(v.y, r[8 * c + 2], r[8 * c + 3]);
          widen4(v.z, r[8 * c + 4], r[8 * c + 5]);
          widen4(v.w, r[8 * c + 6], r[8 * c + 7]);
        }
      }
      // the MMAs that read this slot last are done
      if (step >= (uint32_t)C::NSLOT &&
          !ptx::mbar_wait_bounded_warp(done_bar(dstage), dphase, abort_flag, g.status,
                                       MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs))
        break;
      if (on) {
        ptx::tc_fence_after();
        ptx::tmem_st_32x32b_x32(tmem_base + ((uint32_t)(32 * q) << 16) +
                                    (uint32_t)(C::kSlotCol + slot * 64 + h * 32),
                                r);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(taken_bar(stage));
        if (leader)
          ptx::mbar_arrive(ready_bar(bstage));
        else
          ptx::mbar_arrive_remote(ptx::mapa_shared(ready_bar(bstage), 0));
      }
      // SETS half-steps on
      next_step();
      if (C::SETS == 3) {
        if (h == 1 && w < total) next_step();
        h ^= 1;
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ epilogue (both)
    if constexpr (C::SETS == 3) ptx::setmaxnreg_inc<144>();
    using P = Panel<PASS, OUT, GLU ? 64 : 128>;
    const int q = warp - 4, t = threadIdx.x - 128;
    const int up = GLU ? lane >> 4 : 0;  // this lane's accumulators belong to the up projection
    const int chl = GLU ? 16 * q + (lane & 15) : 32 * q + lane;  // channel of the CTA's panel
    int acc = 0, ub = 0, sb = 0;  // accumulator; buffers of the unit's rows and of the step
    uint32_t acc_phase = 0, clamp = 0u;
    Unit u = {}, ahead = {};
    if (pair < total) ahead = unit_of(pair);
    for (long long w = pair; w < total; w += n_pairs) {
      u = ahead;
      const int n = mma_rows(u);
      int inner_steps = 0;  // steps that free the columns of the next unit
      if (w + n_pairs < total) {
        ahead = unit_of(w + n_pairs);
        inner_steps = shared_cols(mma_rows(ahead), n) / 32;
      }
      const bool sh = u.seg >= g.n_mat;
      const long long ex = sh ? u.seg - g.n_mat : u.seg;
      const int ch0 = u.ct * UCH + (int)rank * (UCH / 2);
      const bool in = ch0 + chl < g.N;
      float wc = 1.0f;
      if (PASS != kInt8Partial) {
        const float* sw = (up ? (sh ? g.sh_sw2 : g.sw2) : (sh ? g.sh_sw : g.sw)) + ex * g.N;
        wc = in ? sw[ch0 + chl] : 0.0f;
      }
      // partial pass: this piece's plane of the output
      uint8_t* out = static_cast<uint8_t*>(g.out);
      const int cols = PASS == kInt8Partial ? int8_part_cols(g.N) : g.N;
      if (PASS == kInt8Partial) out += (w % splits) * 4ll * g.rows * cols;
      float* usx = unit_sx[ub];
      int* orow = unit_orow[ub];
      ub ^= 1;
      for (int r = t; r < kNT; r += 128) unit_row<PASS>(g, u, r, orow[r], usx[r]);
      if (!epilogue_all(ptx::mbar_wait_bounded_warp(dfull_bar(acc), acc_phase, abort_flag,
                                                    g.status, MOE_DEVFAULT_PIPELINE_TIMEOUT,
                                                    kInt8WaitNs)))
        break;
      ptx::tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)acc_col(acc, n);
#pragma unroll 1
      for (int k = 0; k * 32 < n; ++k) {
        const int c = acc == 0 ? n / 32 - 1 - k : k;  // the columns next to the other accumulator first
        uint32_t v[32];
        float sx[32];
        ptx::tmem_ld_32x32b_x32(taddr + c * 32, v);
        load_scales(usx + c * 32, sx);
        // PASS slot: bit j, row c * 32 + j is written
        const uint32_t rows_on =
            PASS == kInt8Slot ? __ballot_sync(0xffffffffu, in && orow[c * 32 + lane] >= 0) : 0u;
        ptx::tmem_wait_ld();
        const bool last = (k + 1) * 32 >= n, inner = k + 1 == inner_steps;
        if (last || inner) {  // the accumulator, or those columns of it, are in registers
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            auto arrive = [&](uint32_t bar) {
              if (leader)
                ptx::mbar_arrive(bar);
              else
                ptx::mbar_arrive_remote(ptx::mapa_shared(bar, 0));
            };
            if (inner) arrive(inner_bar);
            if (last) arrive(dempty_bar(acc));
          }
        }
        if constexpr (GLU) {
          // gate lanes finish columns 0-15, up lanes columns 16-31: each sends the other half over
          uint8_t* buf = stage_out + sb * kInt8StepBytes;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float x = __uint_as_float(v[j]) * wc, y = __uint_as_float(v[16 + j]) * wc;
            const float got = __shfl_xor_sync(0xffffffffu, up ? x : y, 16);
            const int col = j + 16 * up;
            const float s = up ? sx[16 + j] : sx[j];
            const float gv = (up ? got : x) * s, uv = (up ? y : got) * s;
            P::put(buf, col, chl, swiglu(gv, uv));
          }
          epilogue_barrier();
          P::flush(out, cols, buf, orow + c * 32, ch0, t);
          sb ^= 1;
        } else {
#pragma unroll
          for (int j0 = 0; j0 < 32; j0 += P::kCols) {
            uint8_t* buf = stage_out + sb * kInt8StepBytes;
#pragma unroll
            for (int j = 0; j < P::kCols; ++j) {
              const float y = __uint_as_float(v[j0 + j]) * sx[j0 + j] * wc;
              P::put(buf, j, chl, y);
              if (PASS == kInt8Slot && ((rows_on >> (j0 + j)) & 1u))
                clamp = max(clamp, mag_bits(y));
            }
            epilogue_barrier();
            P::flush(out, cols, buf, orow + c * 32 + j0, ch0, t);
            sb ^= 1;
          }
        }
      }
      acc_phase ^= (uint32_t)acc;
      acc ^= 1;
    }
    if (PASS == kInt8Slot && __any_sync(0xffffffffu, clamp >= kInt8F16Clamp) && lane == 0)
      atomicOr(g.status, MOE_DEVFAULT_FP16_RANGE);
  }

  // every copy into either CTA has landed and every MMA has finished once the producers and rank 0's
  // MMA thread are here; neither CTA leaves (nor frees TMEM) before both are
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_cg2(tmem_base, 512);
  }
}

template <int PASS, int OUT, typename C>
cudaError_t launch_one(const Int8Gemm& g, cudaStream_t st) {
  constexpr CUtensorMapDataType kCode = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUtensorMap b, a, a2, sa, sa2;
  bool ok = make_tmap_2d(&b, g.xq, g.x_rows, g.K, 64, kBoxRows, CU_TENSOR_MAP_DATA_TYPE_FLOAT16) &&
            make_tmap_3d(&a, g.qw, g.n_mat, g.N, g.K, kInt8StageK, 64, kCode, 1);
  a2 = a;
  if (ok && PASS == kInt8SwiGLU)
    ok = make_tmap_3d(&a2, g.qw2, g.n_mat, g.N, g.K, kInt8StageK, 64, kCode, 1);
  sa = a;
  sa2 = a2;
  if (ok && g.S > 0) {
    ok = make_tmap_3d(&sa, g.sh_qw, g.S, g.N, g.K, kInt8StageK, 64, kCode, 1);
    if (ok && PASS == kInt8SwiGLU)
      ok = make_tmap_3d(&sa2, g.sh_qw2, g.S, g.N, g.K, kInt8StageK, 64, kCode, 1);
  }
  if (!ok) return cudaErrorInvalidValue;
  auto kern = int8_gemm_kernel<PASS, OUT, C>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms() / 2 * 2);  // persistent: one CTA pair per two SMs
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, b, a, a2, sa, sa2, g);
}

template <int PASS, int OUT>
cudaError_t launch_pass(const Int8Gemm& g, cudaStream_t st) {
  const int mean = g.rows / g.n_mat, pairs = num_sms() / 2, ch = PASS == kInt8SwiGLU ? 128 : 256;
  // units with tiles of at most `tile` rows, of an even spread of the rows over the segments
  auto units = [&](int tile) {
    return ((long long)((mean + tile - 1) / tile) * g.n_mat +
            (long long)((g.T + tile - 1) / tile) * g.S) *
           ((g.N + ch - 1) / ch);
  };
  // where one round of the pairs holds all units, the lowest tiles for which it does: the round takes as
  // long as one unit (pieces of K fill the pairs already)
  auto one_round = [&](int tile) { return PASS != kInt8Partial && units(tile) <= pairs; };
  Int8Gemm t = g;
  // decode: deeper stages, for the weights' sake, where tiles of 64 rows hold every segment (64 tokens, 128 + 1
  // experts of d 7168, d_ff 2048 502 against 514 us in turn; with a shared expert's 512 rows in tiles of 64 541
  // against 524)
  t.tile_rows = 64;
  if ((mean <= kInt8Mean64 && (g.S == 0 || g.T <= 64)) || one_round(64))
    return launch_one<PASS, OUT, Cfg<64, 128, 4, 9, 6, 3>>(t, st);
  // a tile costs about the same whatever its rows, so tiles of 128, with more slots and stages, are for
  // segments that they hold (64 segments of [2048 x 2048], 96 rows each: 69 against 72 us; 128 rows each,
  // half of them longer: 93 against 77)
  t.tile_rows = 128;
  if (mean <= kInt8Mean128 || one_round(128))
    return launch_one<PASS, OUT, Cfg<128, 256, 4, 6, 6, 3>>(t, st);
  // tall tiles (int8_tile_height) where there are units for more than one round of the pairs without them
  // (8 segments of 210 rows of [2048 x 2048] 21.6 against 25.9 us; 4 segments 18 against 16.4)
  t.tile_rows = PASS != kInt8Partial && units(192) > pairs ? 256 : 192;
  return launch_one<PASS, OUT, Cfg<256, 384, 2, 4, 4, PASS == kInt8Slot ? 2 : 3>>(t, st);
}

}  // namespace

cudaError_t launch_int8_gemm(Int8Pass pass, const Int8Gemm& g, cudaStream_t st) {
  switch (pass) {
    case kInt8Partial: return launch_pass<kInt8Partial, MOE_DTYPE_F32>(g, st);
    case kInt8SwiGLU: return launch_pass<kInt8SwiGLU, MOE_DTYPE_F32>(g, st);
    case kInt8Slot: return launch_pass<kInt8Slot, MOE_DTYPE_F16>(g, st);
    default: break;
  }
  switch (g.out_dtype) {
    case MOE_DTYPE_F32: return launch_pass<kInt8Matrix, MOE_DTYPE_F32>(g, st);
    case MOE_DTYPE_BF16: return launch_pass<kInt8Matrix, MOE_DTYPE_BF16>(g, st);
    default: return launch_pass<kInt8Matrix, MOE_DTYPE_F16>(g, st);
  }
}

}  // namespace moe
