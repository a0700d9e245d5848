// Arguments of the two product kernels for a few tokens.
#pragma once

#include "common.cuh"

namespace moe {

struct FewUpArgs {
  int T, K, E, n, cap;
  const int32_t* ids;   // [T, K]
  const float* topk_w;  // [T, K]
  bf16* act;            // [active experts][T][n]
  float* part;          // [2 pieces][T][256]
  uint32_t* arrived;    // [pieces], zero when the kernel starts
  // set by launch_few_up
  int kblocks, nt, npad, stages, stage_bytes;
  unsigned* status;
  unsigned long long limit_ns;
};

struct FewDownArgs {
  int T, K, E, cap;
  int kb;      // 64-wide k-blocks of one expert's matrix, or of the projection
  int d;       // output width
  const int32_t* ids;  // [T, K] (layer), or [T]: the adapter of each row (projection)
  bf16* out;           // [T, d]
  // projection only
  const float* low_part;  // [low_splits][T][rank]
  float* low;             // [T, rank]
  const bf16* b;          // [n_adapters, rank, d]
  const float* scale;     // [n_adapters]
  int rank, low_splits, n_adapters;
  // set by the launcher
  int split, stages, stage_bytes, ring_bytes;
  unsigned* status;
  unsigned long long limit_ns;
};

}  // namespace moe
