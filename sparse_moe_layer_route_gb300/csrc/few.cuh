// The MoE layer for a few tokens (few.cu): launch interface and workspace.
#pragma once
#include "internal.h"

namespace moe {

constexpr int kFewMaxCtas = 208;    // persistent CTAs at most
constexpr int kFewUnits = 5;        // units of work for eight CTAs, at least (see few.cu)
constexpr int kFewSteps = 2;        // tiles of a warp in a unit, at least, where tiles are cut
constexpr unsigned long long kFewWaitNs = 2000000000ull;  // the longest that a wait takes
constexpr int kFewMaxSize = 65536;  // d and d_ff: work is counted in 32 bits

// The grid barriers' count of arrivals, in the counter block that moe_workspace_init clears: a multiple of the
// number of CTAs after every call that completes. It lies behind what the layer of many tokens counts there.
struct FewMeta {
  unsigned others[16];
  unsigned long long arrived;
  unsigned pad[46];
};
static_assert(sizeof(FewMeta) == sizeof(Meta), "it takes the counter block's place");
static_assert(offsetof(FewMeta, arrived) >= offsetof(Meta, pad), "nothing else writes there");

struct FewArgs {
  const uint16_t* x;                                  // [T, d]
  const uint16_t* W_g_t;                              // [E, d], or nullptr: idx_in and w_in are the choice
  const uint16_t *gate, *up, *down;                   // [E, d, f], [E, d, f], [E, f, d]
  const uint16_t *sh_gate, *sh_up, *sh_down;          // the same for S
  const float *bias, *u;                              // BIAS_SELECT, GUMBEL
  const int32_t* idx_in;                              // [T, k]
  const float* w_in;                                  // [T, k] or nullptr (every gate 1)
  moe_route_out ro;                                   // optional results
  uint16_t* out;                                      // [T, d]
  float* logits;                                      // [T, E]
  uint16_t* xf;                                       // x in the order of MMA operands: see few.cu
  uint32_t* h;                                        // activations [columns, f]: see few.cu
  int* count;                                         // of units: see few.cu
  float* part;                                        // sums of tiles' parts
  int* status;
  FewMeta* meta;
  int T, d, E, k, f, S, mode, G, Gk, C;
  float tau;
  // of waits: the limit; in the check of them, CTAs that barriers wait for in vain, and whether a tile is not reported
  unsigned long long limit_ns;
  int absent, withheld;
};

// Tensor maps of the weights: tiles of 32 rows x 64 columns.
struct FewMaps {
  CUtensorMap gate, up, down, sh_gate, sh_up, sh_down;
};

struct FewLayout {
  size_t meta, logits, xf, h, count, part, wg_t, total;
};
FewLayout few_layout(const Shape& s);
cudaError_t launch_few(const FewArgs& a, cudaStream_t st);

}  // namespace moe
