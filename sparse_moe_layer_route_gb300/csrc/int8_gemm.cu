// Grouped products of 8-bit integers over row segments, with a scale per row and per output channel,
// on the 5th-generation tensor cores: the kernel for short segments (decode), the products in pieces
// of K, and the choice between this kernel and int8_gemm_pair.cu's.
//
//   D[channel, row] = sum_k qw[channel, k] * xq[row, k],  out[row, channel] = D * sx[row] * sw[channel]
//
// sm_103a's 8-bit integer tensor rate is far below its 16-bit one, so the codes are multiplied as fp16:
// whole numbers up to 128 are exact there, their products are exact, and fp32 sums of them are exact
// below 2^24. The weights stay 8-bit in memory and in shared memory; they are widened on the way to the
// MMA, whose A operand they are (M = 128 output channels) out of tensor memory. That costs the tile no
// shared-memory writes and leaves the 16-bit B operand (the rows, widened once per call) as the only
// matrix the MMA reads from shared memory.
//
// Bound by the weight bytes: 128 experts and a shared one of [2048 x 7168], 64 tokens, gate and up in
// 329 us and down in 184, 0.96 to 1.0 of the measured copy bandwidth.
//
// One persistent CTA per SM, a unit = two 128-channel tiles (SwiGLU pass: the gate and the up projection
// of the same channels) x up to NT rows of one segment:
//   warp 0       TMA producer, 128 k per stage: two [128 channels x 128 B] code tiles and two
//                [NT rows x 64 k] fp16 tiles, all 128-byte swizzled
//   warp 1       MMA issuer: M = 128, N = the unit's rows rounded up to 16, K = 16. It and the producer
//                run in an elected lane: issued under `lane == 0`, an MMA costs 75 clk, so 27 (decode
//                experts 755 against 531 us)
//   warp 2       TMEM allocator
//   warps 4-7    epilogue: scales, SwiGLU or gate weight, stores (32 channels of a row per warp)
//   warps 8-15   widen the codes, four warps per channel tile: 64 codes of a thread's channel from
//                shared memory to 32 TMEM columns (a slot of 64 k for both tiles is 64 columns)
// Units go segment by segment (find_unit), so CTAs that run together share weights and rows through L2.
// Every wait is bounded (MOE_DEVFAULT_PIPELINE_TIMEOUT on expiry).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "int8.cuh"
#include "int8_units.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kABytes = kInt8Ch * kInt8StageK;   // 16 KB per channel tile

// NB accumulator buffers of 2 NT columns, SA slots of widened weights of 64 columns.
template <int NT, int NB, int SA>
struct Cfg {
  static constexpr int kBBytes = NT * kInt8StageK * 2;
  static constexpr int kStageBytes = 2 * kABytes + kBBytes;
  static constexpr int kStages = 204 * 1024 / kStageBytes > 6 ? 6 : 204 * 1024 / kStageBytes;
  static constexpr int kSmemBytes =
      kStages * kStageBytes + 2 * kInt8StepBytes + 1024 /*align*/ + 256 /*barriers*/;
  static constexpr int kACol = NB * 2 * NT;  // first column of the weight slots
  static_assert(kACol + SA * 64 <= 512, "TMEM columns");
  static_assert(NT % 32 == 0, "epilogue steps; B sub-tiles stay 1024-byte aligned");
};

template <int PASS, int OUT, int NT, int NB, int SA>
__global__ void __launch_bounds__(kInt8Threads, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ CUtensorMap tmA2,
                     const __grid_constant__ CUtensorMap tmShA,
                     const __grid_constant__ CUtensorMap tmShA2, const Int8Gemm g) {
  using C = Cfg<NT, NB, SA>;
  constexpr bool PAIR = PASS == kInt8SwiGLU;
  constexpr int STAGES = C::kStages;
  constexpr int UCH = PAIR ? kInt8Ch : 2 * kInt8Ch;  // output channels per unit

  extern __shared__ uint8_t smem_raw[];
  __shared__ SegTable segs;
  __shared__ __align__(16) float unit_sx[2][NT];  // row scales, output rows of the epilogue's unit
  __shared__ int unit_orow[2][NT];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  uint8_t* const stage_out = gbase + STAGES * C::kStageBytes;  // the epilogue's two steps
  const uint32_t bar0 = base + STAGES * C::kStageBytes + 2 * kInt8StepBytes;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto afull_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };
  auto aempty_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + SA + s); };
  auto dfull_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + 2 * SA + b); };
  auto dempty_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + 2 * SA + NB + b); };
  constexpr int kBars = 2 * STAGES + 2 * SA + 2 * NB;
  const uint32_t mma_done_bar = bar0 + 8u * kBars;
  static_assert(8 * (kBars + 1) + 8 <= 256, "barrier block");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(stage_out + 2 * kInt8StepBytes + 8 * (kBars + 1));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 9);  // eight widening warps and the MMAs
    }
    for (int s = 0; s < SA; ++s) {
      ptx::mbar_init(afull_bar(s), 8);
      ptx::mbar_init(aempty_bar(s), 1);
    }
    for (int b = 0; b < NB; ++b) {
      ptx::mbar_init(dfull_bar(b), 1);
      ptx::mbar_init(dempty_bar(b), 4);
    }
    ptx::mbar_init(mma_done_bar, 1);
    *abort_flag = 0;
    ptx::fence_mbarrier_init();
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
    if (PAIR) ptx::prefetch_tmap(&tmA2);
  }
  if (warp == 2) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  griddep_wait();  // everything above touched only shared memory, TMEM and parameters
  build_segments(segs, g, NT);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int n_ct = (g.N + UCH - 1) / UCH;
  const int n_sub = (g.K + 63) / 64;           // 64-k slots per unit
  const int n_stage = (n_sub + 1) / 2;         // 128-k stages per unit
  // partial pass: a unit is done in pieces, each some of its stages
  const int splits = PASS == kInt8Partial ? g.splits : 1;
  const long long total = (long long)segs.first[g.n_mat + g.S] * n_ct * splits;
  auto unit_of = [&](long long w) {
    return find_unit<PAIR>(segs, g, n_ct, PASS == kInt8Partial ? w / splits : w);
  };
  auto first_stage = [&](long long w) {
    return PASS == kInt8Partial ? (int)(w % splits) * n_stage / splits : 0;
  };
  auto end_stage = [&](long long w) {
    return PASS == kInt8Partial ? ((int)(w % splits) + 1) * n_stage / splits : n_stage;
  };

  if (warp == 0) {
    if (ptx::elect_one()) {
      // ---------------------------------------------------------------- TMA producer
      int stage = 0;
      uint32_t phase = 0, issued = 0, last_parity = 0;  // per stage: ever issued, its parity
      bool ok = true;
      for (long long w = blockIdx.x; w < total && ok; w += gridDim.x) {
        const Unit u = unit_of(w);
        const bool sh = u.seg >= g.n_mat;
        const int ex = sh ? u.seg - g.n_mat : u.seg;
        const CUtensorMap* a0 = sh ? &tmShA : &tmA;
        const CUtensorMap* a1 = PAIR ? (sh ? &tmShA2 : &tmA2) : a0;
        const int ch0 = u.ct * UCH, ch1 = PAIR ? ch0 : ch0 + kInt8Ch;
        const bool two = ch1 < g.N;
        const int i1 = end_stage(w);
        for (int i = first_stage(w); i < i1; ++i) {
          if (!ptx::mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag, g.status,
                                      MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs)) {
            ok = false;
            break;
          }
          const uint32_t sA = base + stage * C::kStageBytes, sB = sA + 2 * kABytes;
          const uint32_t fb = full_bar(stage);
          const bool half = 2 * i + 1 < n_sub;  // the stage's second 64 k hold something
          ptx::mbar_arrive_expect_tx(
              fb, (two ? 2 : 1) * kABytes + (half ? C::kBBytes : C::kBBytes / 2));
          ptx::tma_load_3d(sA, a0, fb, i * kInt8StageK, ch0, ex);
          if (two) ptx::tma_load_3d(sA + kABytes, a1, fb, i * kInt8StageK, ch1, ex);
          ptx::tma_load_2d(sB, &tmB, fb, i * kInt8StageK, u.brow0);
          if (half) ptx::tma_load_2d(sB + C::kBBytes / 2, &tmB, fb, i * kInt8StageK + 64, u.brow0);
          issued |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // never leave while a copy into this CTA's shared memory may still be in flight
      for (int s = 0; s < STAGES; ++s)
        if (issued & (1u << s)) {
          volatile int no_abort = 0;
          ptx::mbar_wait_bounded(full_bar(s), (last_parity >> s) & 1u, &no_abort, g.status,
                                 MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs / 4);
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (ptx::elect_one()) {
      // ---------------------------------------------------------------- MMA issuer
      int stage = 0, slot = 0, acc = 0;
      uint32_t phase = 0, slot_phase = 0, acc_phase = 0;
      bool ok = true;
      for (long long w = blockIdx.x; w < total && ok; w += gridDim.x) {
        const Unit u = unit_of(w);
        const bool two = PAIR || u.ct * UCH + kInt8Ch < g.N;
        const uint32_t idesc =
            ptx::idesc_f16kind_f32(kInt8Ch, (uint32_t)((u.rows + 15) & ~15), 0, 0, 0u);
        if (!ptx::mbar_wait_bounded(dempty_bar(acc), acc_phase ^ 1u, abort_flag, g.status,
                                    MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs))
          break;
        ptx::tc_fence_after();
        const uint32_t d0 = tmem_base + (uint32_t)(acc * 2 * NT), d1 = d0 + NT;
        const int i0 = first_stage(w), i1 = end_stage(w);
        for (int i = i0; i < i1 && ok; ++i) {
          if (!ptx::mbar_wait_bounded(full_bar(stage), phase, abort_flag, g.status,
                                      MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs)) {
            ok = false;
            break;
          }
          const uint32_t sB = base + stage * C::kStageBytes + 2 * kABytes;
          for (int h = 0; h < 2 && 2 * i + h < n_sub; ++h) {
            if (!ptx::mbar_wait_bounded(afull_bar(slot), slot_phase, abort_flag, g.status,
                                        MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            const uint32_t a0 = tmem_base + C::kACol + slot * 64;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              // B: K-major, 128 B rows, 8-row groups 1024 B apart; a K step of 16 = +32 B
              const uint64_t bdesc =
                  ptx::smem_desc_sw128(sB + h * (C::kBBytes / 2) + kk * 32, 16, 1024);
              const uint32_t more = ((i - i0) | h | kk) != 0 ? 1u : 0u;
              ptx::umma_f16_ta(d0, a0 + kk * 8, bdesc, idesc, more);
              if (two) ptx::umma_f16_ta(d1, a0 + 32 + kk * 8, bdesc, idesc, more);
            }
            ptx::umma_commit(aempty_bar(slot));
            if (++slot == SA) {
              slot = 0;
              slot_phase ^= 1u;
            }
          }
          if (!ok) break;
          ptx::umma_commit(empty_bar(stage));
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::umma_commit(dfull_bar(acc));
        if (++acc == NB) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      // all MMAs issued by this thread have finished before TMEM is released
      ptx::umma_commit(mma_done_bar);
      volatile int no_abort = 0;
      ptx::mbar_wait_bounded(mma_done_bar, 0, &no_abort, g.status, MOE_DEVFAULT_PIPELINE_TIMEOUT,
                             kInt8WaitNs / 4);
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ widening warps
    const int tile = (warp - 8) >> 2, q = warp & 3;  // channel tile; TMEM lanes [32 q, 32 q + 32)
    const int row = 32 * q + lane;
    int stage = 0, slot = 0;
    uint32_t phase = 0, slot_phase = 0;
    bool ok = true;
    for (long long w = blockIdx.x; w < total && ok; w += gridDim.x) {
      const Unit u = unit_of(w);
      const bool on = PAIR || tile == 0 || u.ct * UCH + kInt8Ch < g.N;
      const int i1 = end_stage(w);
      for (int i = first_stage(w); i < i1 && ok; ++i) {
        if (!ptx::mbar_wait_bounded_warp(full_bar(stage), phase, abort_flag, g.status,
                                         MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs)) {
          ok = false;
          break;
        }
        const uint8_t* src = gbase + stage * C::kStageBytes + tile * kABytes + row * kInt8StageK;
        for (int h = 0; h < 2 && 2 * i + h < n_sub; ++h) {
          uint32_t r[32];
          if (on) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              // 16-byte piece 4 h + c of the row sits at piece (4 h + c) ^ (row mod 8)
              const uint4 v =
                  *reinterpret_cast<const uint4*>(src + (((4 * h + c) ^ (row & 7)) << 4));
              widen4(v.x, r[8 * c], r[8 * c + 1]);
              widen4(v.y, r[8 * c + 2], r[8 * c + 3]);
              widen4(v.z, r[8 * c + 4], r[8 * c + 5]);
              widen4(v.w, r[8 * c + 6], r[8 * c + 7]);
            }
          }
          if (h == 1 || 2 * i + 1 == n_sub) {  // the stage's codes are in registers
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(empty_bar(stage));
          }
          if (!ptx::mbar_wait_bounded_warp(aempty_bar(slot), slot_phase ^ 1u, abort_flag, g.status,
                                           MOE_DEVFAULT_PIPELINE_TIMEOUT, kInt8WaitNs)) {
            ok = false;
            break;
          }
          if (on) {
            ptx::tc_fence_after();
            ptx::tmem_st_32x32b_x32(tmem_base + ((uint32_t)(32 * q) << 16) +
                                        (uint32_t)(C::kACol + slot * 64 + tile * 32),
                                    r);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(afull_bar(slot));
          if (++slot == SA) {
            slot = 0;
            slot_phase ^= 1u;
          }
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ epilogue
    using P = Panel<PASS, OUT, kInt8Ch>;
    const int q = warp - 4, t = threadIdx.x - 128, chl = 32 * q + lane;
    int acc = 0, ub = 0, sb = 0;  // accumulator; buffers of the unit's rows and of the step
    uint32_t acc_phase = 0, clamp = 0u;
    for (long long w = blockIdx.x; w < total; w += gridDim.x) {
      const Unit u = unit_of(w);
      const bool sh = u.seg >= g.n_mat;
      const long long ex = sh ? u.seg - g.n_mat : u.seg;
      const int ch0 = u.ct * UCH, ch1 = PAIR ? ch0 : ch0 + kInt8Ch;
      const bool in0 = ch0 + chl < g.N, in1 = ch1 + chl < g.N, two = ch1 < g.N;
      float w0 = 1.0f, w1 = 1.0f;
      if (PASS != kInt8Partial) {
        const float* sw = (sh ? g.sh_sw : g.sw) + ex * g.N;
        const float* sw2 = PAIR ? (sh ? g.sh_sw2 : g.sw2) + ex * g.N : sw;
        w0 = in0 ? sw[ch0 + chl] : 0.0f;
        w1 = in1 ? sw2[ch1 + chl] : 0.0f;
      }
      // partial pass: this piece's plane of the output
      uint8_t* out = static_cast<uint8_t*>(g.out);
      if (PASS == kInt8Partial) out += (w % splits) * 4ll * g.rows * g.N;
      float* usx = unit_sx[ub];
      int* orow = unit_orow[ub];
      ub ^= 1;
      for (int r = t; r < NT; r += 128) unit_row<PASS>(g, u, r, orow[r], usx[r]);
      if (!epilogue_all(ptx::mbar_wait_bounded_warp(dfull_bar(acc), acc_phase, abort_flag,
                                                    g.status, MOE_DEVFAULT_PIPELINE_TIMEOUT,
                                                    kInt8WaitNs)))
        break;
      ptx::tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(32 * q) << 16) + (uint32_t)(acc * 2 * NT);
      // one panel of staged steps: value(j) is this thread's channel of row c * 32 + j; slot pass:
      // bit j of rows_on, that row is written
      auto steps = [&](int c, int ch, bool in, uint32_t rows_on, auto value) {
#pragma unroll
        for (int j0 = 0; j0 < 32; j0 += P::kCols) {
          uint8_t* buf = stage_out + sb * kInt8StepBytes;
#pragma unroll
          for (int j = 0; j < P::kCols; ++j) {
            const float y = value(j0 + j);
            P::put(buf, j, chl, y);
            if (PASS == kInt8Slot && in && ((rows_on >> (j0 + j)) & 1u))
              clamp = max(clamp, mag_bits(y));
          }
          epilogue_barrier();
          P::flush(out, g.N, buf, orow + c * 32 + j0, ch, t);
          sb ^= 1;
        }
      };
#pragma unroll 1
      for (int c = 0; c * 32 < u.rows; ++c) {
        uint32_t v0[32], v1[32];
        float sx[32];
        ptx::tmem_ld_32x32b_x32(taddr + c * 32, v0);
        ptx::tmem_ld_32x32b_x32(taddr + NT + c * 32, v1);
        load_scales(usx + c * 32, sx);
        const uint32_t rows_on =
            PASS == kInt8Slot ? __ballot_sync(0xffffffffu, orow[c * 32 + lane] >= 0) : 0u;
        ptx::tmem_wait_ld();
        if ((c + 1) * 32 >= u.rows) {  // the accumulators are in registers
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(dempty_bar(acc));
        }
        if constexpr (PAIR) {
          steps(c, ch0, in0, rows_on, [&](int j) {
            const float gv = __uint_as_float(v0[j]) * (sx[j] * w0);
            return swiglu(gv, __uint_as_float(v1[j]) * (sx[j] * w1));
          });
        } else {
          steps(c, ch0, in0, rows_on, [&](int j) { return __uint_as_float(v0[j]) * (sx[j] * w0); });
          if (two)
            steps(c, ch1, in1, rows_on,
                  [&](int j) { return __uint_as_float(v1[j]) * (sx[j] * w1); });
        }
      }
      if (++acc == NB) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (PASS == kInt8Slot && __any_sync(0xffffffffu, clamp >= kInt8F16Clamp) && lane == 0)
      atomicOr(g.status, MOE_DEVFAULT_FP16_RANGE);
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, 512);
  }
}

template <int PASS, int OUT, int NT, int NB, int SA>
cudaError_t launch_one(const Int8Gemm& g, cudaStream_t st) {
  using C = Cfg<NT, NB, SA>;
  constexpr CUtensorMapDataType kCode = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUtensorMap b, a, a2, sa, sa2;
  bool ok = make_tmap_2d(&b, g.xq, g.x_rows, g.K, 64, NT, CU_TENSOR_MAP_DATA_TYPE_FLOAT16) &&
            make_tmap_3d(&a, g.qw, g.n_mat, g.N, g.K, kInt8StageK, kInt8Ch, kCode, 1);
  a2 = a;
  if (ok && PASS == kInt8SwiGLU)
    ok = make_tmap_3d(&a2, g.qw2, g.n_mat, g.N, g.K, kInt8StageK, kInt8Ch, kCode, 1);
  sa = a;
  sa2 = a2;
  if (ok && g.S > 0) {
    ok = make_tmap_3d(&sa, g.sh_qw, g.S, g.N, g.K, kInt8StageK, kInt8Ch, kCode, 1);
    if (ok && PASS == kInt8SwiGLU)
      ok = make_tmap_3d(&sa2, g.sh_qw2, g.S, g.N, g.K, kInt8StageK, kInt8Ch, kCode, 1);
  }
  if (!ok) return cudaErrorInvalidValue;
  auto kern = int8_gemm_kernel<PASS, OUT, NT, NB, SA>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3(num_sms()), dim3(kInt8Threads), C::kSmemBytes, st, b, a, a2, sa, sa2, g);
}

// y = (sum of the pieces, in their order) * row scale * channel scale; rows past the last segment are left.
template <typename YT>
__global__ void __launch_bounds__(256) join_splits_kernel(const float* __restrict__ part,
                                                          const Int8Gemm g) {
  griddep_wait();
  const int row = blockIdx.x;
  int seg = 0;
  if (g.offsets != nullptr) {
    // the last segment that begins at or before the row and reaches it (bad offsets were reported by
    // the product, which left their rows out)
    int lo = 0, hi = g.n_mat;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (g.offsets[mid] <= row)
        lo = mid;
      else
        hi = mid;
    }
    seg = lo;
    const int r0 = g.offsets[seg], r1 = g.offsets[seg + 1];
    if (r0 < 0 || r1 > g.rows || row < r0 || row >= r1) return;
  }
  const int n = blockIdx.y * 256 + threadIdx.x;
  if (n >= g.N) return;
  const long long at = (long long)row * g.N + n, plane = (long long)g.rows * g.N;
  const float scale = g.sx[row] * g.sw[(long long)seg * g.N + n];
  float sum = 0.0f;
  for (int i = 0; i < g.splits; i += 8) {  // eight loads in flight, added in the pieces' order
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j < g.splits ? part[(i + j) * plane + at] : 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += v[j];
  }
  sum *= scale;
  if constexpr (sizeof(YT) == 4)
    static_cast<float*>(g.out)[at] = sum;
  else if constexpr (std::is_same<YT, __nv_bfloat16>::value)
    static_cast<__nv_bfloat16*>(g.out)[at] = __float2bfloat16(sum);
  else
    static_cast<__half*>(g.out)[at] = __float2half(sum);
}

}  // namespace

int int8_splits(long long rows, int K, int N, int n_mat) {
  const long long mean = rows / n_mat;
  const bool pair = mean > kInt8MeanSingle;
  const long long at_once = pair ? 76 : 152;  // units that run at the same time
  const long long tile = !pair ? 32 : mean <= kInt8Mean128 ? 128 : 192;
  const long long units = std::max(1ll, (mean + tile - 1) / tile) * n_mat * ((N + 255) / 256);
  if (units * 2 > at_once || N > 65535 * 256) return 1;
  // at least four 128-k steps a piece: shorter ones spend their time on filling the pipeline
  return (int)std::max(1ll, std::min(at_once / units, (long long)(K / kInt8StageK / 4)));
}

cudaError_t launch_int8_split(const Int8Gemm& g, float* part, cudaStream_t st) {
  Int8Gemm p = g;
  p.splits = int8_splits(g.rows, g.K, g.N, g.n_mat);
  p.out = part;
  cudaError_t e = g.rows / g.n_mat > kInt8MeanSingle
                      ? launch_int8_gemm_pair(kInt8Partial, p, st)
                      : launch_one<kInt8Partial, MOE_DTYPE_F32, 32, 2, 6>(p, st);
  if (e != cudaSuccess) return e;
  p.out = g.out;
  const dim3 grid(g.rows, (g.N + 255) / 256), block(256);
  switch (g.out_dtype) {
    case MOE_DTYPE_F32: return launch_k(join_splits_kernel<float>, grid, block, 0, st, part, p);
    case MOE_DTYPE_BF16:
      return launch_k(join_splits_kernel<__nv_bfloat16>, grid, block, 0, st, part, p);
    default: return launch_k(join_splits_kernel<__half>, grid, block, 0, st, part, p);
  }
}

cudaError_t launch_int8_gemm(Int8Pass pass, const Int8Gemm& g, cudaStream_t st) {
  // by the rows per segment of an even spread. Decode's short segments are bound by the weights, which
  // single CTAs of 32-row tiles stream better (decode experts, 1 row a segment, 330 against 358 us for
  // gate and up); from 16 rows on the pairs' cheaper tiles win (64 segments of [2048 x 2048], 24 rows
  // each: 59 against 63 us)
  if (g.rows / g.n_mat > kInt8MeanSingle) return launch_int8_gemm_pair(pass, g, st);
  switch (pass) {
    case kInt8SwiGLU: return launch_one<kInt8SwiGLU, MOE_DTYPE_F32, 32, 2, 6>(g, st);
    case kInt8Slot: return launch_one<kInt8Slot, MOE_DTYPE_F16, 32, 2, 6>(g, st);
    default: break;
  }
  switch (g.out_dtype) {
    case MOE_DTYPE_F32: return launch_one<kInt8Matrix, MOE_DTYPE_F32, 32, 2, 6>(g, st);
    case MOE_DTYPE_BF16: return launch_one<kInt8Matrix, MOE_DTYPE_BF16, 32, 2, 6>(g, st);
    default: return launch_one<kInt8Matrix, MOE_DTYPE_F16, 32, 2, 6>(g, st);
  }
}

}  // namespace moe
