// Arguments of the product kernels for a few tokens.
#pragma once

#include "common.cuh"

namespace moe {

struct FewUpArgs {
  int T, K, E, n, cap;
  const int32_t* ids;   // [T, K]
  const float* topk_w;  // [T, K]
  bf16* act;            // [active experts][T][n]: row j is the expert's j-th token
  float* part;          // [2 pieces][T][256]
  uint32_t* arrived;    // [pieces], zero when the kernel starts
  // set by launch_few_up
  int kblocks, nt, npad, stages, stage_bytes;
  unsigned* status;
  unsigned long long limit_ns;
};

struct FewDownArgs {
  int T, K, E, cap, n, d;
  const int32_t* ids;  // [T, K]
  const bf16* act;     // [active experts][T][n]: row j is the expert's j-th token
  int rows;            // its rows: active experts (at most) times T
  bf16* out;           // [T, d]
  float* part;         // [2 pieces][T][128]: partials of cut tiles
  // set by the launcher
  int kb, nt;  // stages of one expert's matrix; 128-column tiles
  int ring_bytes;
  unsigned* status;
  unsigned long long limit_ns;
};

struct AdapterFewArgs {
  int T, d;                // d: output width
  const int32_t* ids;      // [T]
  const float* low_part;   // [low_splits][T][rank]
  float* low;              // [T, rank]
  const bf16* b;           // [n_adapters, rank, d]
  const float* scale;      // [n_adapters]
  int rank, low_splits, n_adapters;
  bf16* out;               // [T, d]
  // set by the launcher
  int kb, split, stages, stage_bytes, ring_bytes, low_bytes;
  unsigned* status;
  unsigned long long limit_ns;
};

}  // namespace moe
