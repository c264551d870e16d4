// What the 8-bit product kernels share: the work units of a grouped product and its stores.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "int8.cuh"

namespace moe {

constexpr int kInt8Ch = 128;                       // channels per MMA tile of one CTA (TMEM lanes)
constexpr uint64_t kInt8WaitNs = 2000000000ull;    // 2 s per wait
constexpr int kMaxSegs = 256 + 4;
// Channel tiles per block of units. A prefill product of 16384 x 7168 rows: with 16 tiles in a row of row
// tiles each wave read all 235 MB of rows again, 634 us; blocks of 8 read them twice.
constexpr int kCtBlock = 8;

__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
constexpr uint32_t kInt8F16Clamp = 0x477FF000u;  // 65520.0f: the first value past fp16's range

__device__ __forceinline__ uint16_t f16_sat(float v) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.0f), "f"(v));
  return (uint16_t)r;
}

// silu(g) * u. The quotient is the reciprocal's (2 ulp): an exact division branches, which kept the
// epilogue's elements from overlapping (180 clk each).
__device__ __forceinline__ float swiglu(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

struct Unit {
  int seg;      // expert, or n_mat + shared expert
  int ct;       // channel tile
  int row0;     // first position
  int rows;     // 1..the segment's tile height
  int brow0;    // first row of the activations
  bool mixed;   // some segments are unsound: others may share rows
};

// Row tiles before each segment (first[n_segs] = all of them) and the segments' first positions.
struct SegTable {
  int first[kMaxSegs + 1];
  int row0[kMaxSegs];
  int rows[kMaxSegs];
  int height[kMaxSegs];  // rows of a row tile (the last one may be lower)
  int warp_tot[32];
  int mixed;
};

// Rows that a segment can have. The experts' positions past the last offset are those of dropped slots: no codes
// are written there, so an expert that reaches past it is unsound.
template <int PASS>
__device__ __forceinline__ int rows_end(const Int8Gemm& g) {
  return PASS == kInt8SwiGLU || PASS == kInt8Slot ? min(g.rows, g.offsets[g.n_mat]) : g.rows;
}

// Called by every thread of a CTA (of at least kMaxSegs). NT: the tallest tile.
template <int PASS>
__device__ __forceinline__ void build_segments(SegTable& t, const Int8Gemm& g, int NT) {
  const int n = g.n_mat + g.S, i = threadIdx.x;
  const int lane = i & 31, warp = i >> 5;
  int r0 = 0, nr = 0;
  bool bad = false;
  if (i < g.n_mat) {
    int r1 = g.rows;
    if (g.offsets != nullptr) {
      r0 = g.offsets[i];
      r1 = g.offsets[i + 1];
      if (!segment_ok(r0, r1, rows_end<PASS>(g))) {
        atomicOr(g.status, MOE_DEVFAULT_BAD_TILE);
        bad = true;
        r0 = r1 = 0;
      }
    }
    nr = r1 - r0;
  } else if (i < n) {
    r0 = g.rows + (i - g.n_mat) * g.T;
    nr = g.T;
  }
  const int height = int8_tile_height(nr, NT);
  const int nt = (nr + height - 1) / height;
  int v = nt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) t.warp_tot[warp] = v;
  const int mixed = __syncthreads_or(bad);
  if (i == 0) t.mixed = mixed;
  int base = 0;
  for (int w = 0; w < warp; ++w) base += t.warp_tot[w];
  if (i < n) {
    t.first[i] = base + v - nt;
    t.row0[i] = r0;
    t.rows[i] = nr;
    t.height[i] = height;
    if (i == n - 1) t.first[n] = base + v;
  }
  __syncthreads();
}

// X_SHARED: the shared experts all read rows [rows, rows + T) of the activations (SwiGLU pass).
template <bool X_SHARED>
__device__ __forceinline__ Unit find_unit(const SegTable& t, const Int8Gemm& g, int n_ct,
                                          long long w) {
  int lo = 0, hi = g.n_mat + g.S;  // first[lo] * n_ct <= w < first[hi] * n_ct
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((long long)t.first[mid] * n_ct <= w)
      lo = mid;
    else
      hi = mid;
  }
  // a segment's units go in blocks of kCtBlock channel tiles, in a block by row tiles: CTAs that run
  // together share the weights of a block and read each row tile once per block
  const int local = (int)(w - (long long)t.first[lo] * n_ct);
  const int nt = t.first[lo + 1] - t.first[lo];
  const int blk = local / (nt * kCtBlock), in = local - blk * (nt * kCtBlock);
  const int wide = min(kCtBlock, n_ct - blk * kCtBlock);
  Unit u;
  u.seg = lo;
  u.ct = blk * kCtBlock + in % wide;
  const int off = in / wide * t.height[lo];
  u.row0 = t.row0[lo] + off;
  u.rows = min(t.height[lo], t.rows[lo] - off);
  u.brow0 = X_SHARED && lo >= g.n_mat ? g.rows + off : u.row0;
  u.mixed = t.mixed != 0;
  return u;
}

// Whether a sound segment before `seg` holds the row as well.
template <int PASS>
__device__ __forceinline__ bool row_taken(const Int8Gemm& g, int seg, int row) {
  const int end = rows_end<PASS>(g);
#pragma unroll 1
  for (int e = 0; e < seg; ++e) {
    const int r0 = g.offsets[e], r1 = g.offsets[e + 1];
    if (segment_ok(r0, r1, end) && row >= r0 && row < r1) return true;
  }
  return false;
}

// The output row and the row scale of position row0 + r of a unit: -1 past the unit's rows, where another
// segment has the row, or where the slot is out of range.
template <int PASS>
__device__ __forceinline__ void unit_row(const Int8Gemm& g, const Unit& u, int r, int& orow,
                                         float& sx) {
  sx = 0.0f;
  orow = -1;
  if (r >= u.rows) return;
  if (u.mixed && u.seg < g.n_mat && row_taken<PASS>(g, u.seg, u.row0 + r)) return;
  sx = PASS == kInt8Partial ? 1.0f : g.sx[u.brow0 + r];
  orow = u.row0 + r;
  if (PASS == kInt8Slot && u.seg < g.n_mat) {
    const int slot = g.perm_slot[u.row0 + r];
    const bool good = slot >= 0 && slot < g.rows;
    orow = good ? slot : -1;
    if (good && g.topk_w != nullptr) sx *= g.topk_w[slot];
  }
}

// ---------------------------------------------------------------------------- epilogue stores
// An accumulator row is one output channel, so a thread's values belong to as many output rows, two or
// four bytes in each. They pass through shared memory: a step stages kCols output rows of a panel of CH
// channels (8 KB), and the four epilogue warps write them back as 16-byte pieces of whole rows. Two
// buffers, so one barrier per step: a buffer is rewritten after the next step's barrier. (Stored
// straight from the accumulators, an epilogue took about 150 clk per column, longer than the MMAs of a
// unit with K = 1408.)
constexpr int kInt8StepBytes = 8192;

// The scales of 32 consecutive rows to registers, before the step's stores: the compiler keeps a shared
// load behind the shared stores in front of it, and 32 of those in turn cost 3000 clk a step.
__device__ __forceinline__ void load_scales(const float* usx, float (&s)[32]) {
#pragma unroll
  for (int j = 0; j < 32; j += 4)
    *reinterpret_cast<float4*>(s + j) = *reinterpret_cast<const float4*>(usx + j);
}

__device__ __forceinline__ void epilogue_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// A barrier that tells every epilogue thread whether `ok` held in all of them.
__device__ __forceinline__ bool epilogue_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

template <int PASS, int OUT, int CH>
struct Panel {
  static constexpr int kSize = OUT == MOE_DTYPE_F32 ? 4 : 2;
  static constexpr int kRowBytes = CH * kSize;
  static constexpr int kCols = kInt8StepBytes / kRowBytes;  // output rows per step

  static __device__ __forceinline__ void put(uint8_t* buf, int col, int ch, float y) {
    uint8_t* at = buf + col * kRowBytes + ch * kSize;
    if (OUT == MOE_DTYPE_F32)
      *reinterpret_cast<float*>(at) = y;
    else if (OUT == MOE_DTYPE_BF16)
      *reinterpret_cast<__nv_bfloat16*>(at) = __float2bfloat16(y);
    else if (PASS == kInt8Slot)
      *reinterpret_cast<uint16_t*>(at) = f16_sat(y);
    else
      *reinterpret_cast<__half*>(at) = __float2half(y);
  }

  // t: 0..127. The step's rows to the output: the first `bytes` of a row's panel at panel + row * row_bytes,
  // in pieces of VB bytes.
  template <int VB>
  static __device__ __forceinline__ void copy(uint8_t* panel, long long row_bytes, int bytes,
                                              const uint8_t* buf, const int* orow, int t) {
    using V = std::conditional_t<VB == 16, uint4,
                                 std::conditional_t<VB == 8, uint2,
                                                    std::conditional_t<VB == 4, uint32_t, uint16_t>>>;
    constexpr int kPer = kRowBytes / VB, kN = kInt8StepBytes / (128 * VB);
    V v[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = *reinterpret_cast<const V*>(buf + (i * 128 + t) * VB);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = (i * 128 + t) % kPer * VB, to = orow[(i * 128 + t) / kPer];
      if (to >= 0 && at < bytes) *reinterpret_cast<V*>(panel + to * row_bytes + at) = v[i];
    }
  }
  // Channels [ch0, ch0 + CH) of the output rows orow[0, kCols), in the widest pieces that the output's
  // address, its row length and the panel's channels allow.
  static __device__ __forceinline__ void flush(uint8_t* out, int N, const uint8_t* buf,
                                               const int* orow, int ch0, int t) {
    const int bytes = min(CH, N - ch0) * kSize;
    if (bytes <= 0) return;
    const long long row_bytes = (long long)N * kSize;
    uint8_t* panel = out + (long long)ch0 * kSize;
    const unsigned odd = (unsigned)(row_bytes | reinterpret_cast<long long>(out)) | (unsigned)bytes;
    if ((odd & 15u) == 0u)
      copy<16>(panel, row_bytes, bytes, buf, orow, t);
    else if ((odd & 7u) == 0u)
      copy<8>(panel, row_bytes, bytes, buf, orow, t);
    else if (kSize == 4 || (odd & 3u) == 0u)
      copy<4>(panel, row_bytes, bytes, buf, orow, t);
    else if constexpr (kSize == 2)
      copy<2>(panel, row_bytes, bytes, buf, orow, t);
  }
};

}  // namespace moe
