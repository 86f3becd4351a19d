// cross_attn.cuh -- what the kernels of the attention to the encoder's states share.
#pragma once

#include <cuda_bf16.h>

#include "gdn_internal.h"

namespace gdn {

constexpr float kLowest = -3e38f;  // the running maximum of no scores: from it, p of a score of -inf is 0
constexpr int kFewRows = 16;  // query rows of a (b, key head) that cross_few.cu takes

struct CrossParams {
  int Tq, S, Hk, G, D;
  int tokens;            // query tokens per tile: 128 / G
  int gmul;              // r / G = r * gmul >> 16 for rows r < 128
  int qtiles, groups;    // query tiles of a (b, key head); units along them
  int ntiles;            // key tiles
  unsigned full;         // units that one CTA each takes whole; those behind them ...
  int nsplit, per_split; // ... are split along the keys: CTAs of a unit, tiles of each
  int most;              // key tiles of a CTA, at most
  int qb, kb, vb;        // batch coordinate factors: 0 for a broadcast batch
  const uint8_t* mask;
  long long mask_bs;
  float scale_log2;      // scale * log2(e)
  __nv_bfloat16* out;    // [B, Tq, Hq, D]
  float* lse;            // [B, Hq, Tq] or nullptr
  float* part_o;         // [split units][nsplit][rows of a unit][D] fp32
  float* part_lse;       // [split units][nsplit][rows of a unit]
  long long limit;
  unsigned* err;
};

// The kernel for at most kFewRows rows: CTAs of a (b, key head), and the launch.  Up
// to kFewCluster CTAs join by themselves, more leave parts as split units do.
constexpr int kFewCluster = 8;
int few_splits(int B, int Hk, int S);
cudaError_t launch_cross_few(const CrossCall& c, const CrossParams& P);

}  // namespace gdn
