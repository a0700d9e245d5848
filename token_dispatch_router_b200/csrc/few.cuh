// Arguments of the few-token product kernel (few.cu), shared by the decode layer and the
// adapter projection, and the layout of its control words.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kFewMaxTokens = 128;  // tokens on the MMA's N: two accumulators, double-buffered
constexpr int kFewMaxSplit = 16;
constexpr int kFewTarget = 1024;     // at most this many tiles are split over their contraction
constexpr int kFewMaxExperts = 256;

// Control words, zero when the kernel starts: the kernel that runs before it in the same call
// clears them.
constexpr int kFewTicket = 0;                            // next unit of work
constexpr int kFewDone = 1;                              // finished second-product units
constexpr int kFewExpert = 2;                            // + active expert: finished act tiles
constexpr int kFewTile = kFewExpert + kFewMaxExperts;    // + tile: arrived contraction splits
constexpr int kFewCtlWords = kFewTile + kFewTarget;

struct FewArgs {
  int T, K, E;
  int kb1, kb2;    // 64-wide k-blocks of the first and of the second product
  int n, nt1;      // width of the first product's output, its 128-column tiles
  int d, nt2;      // width of the second product's output, its 256-column tiles
  int smax1, smax2;  // contraction splits that the partial buffers have room for
  int cap;         // kept tokens per expert
  int npad;        // T rounded up to 16: the MMA's N
  int stages, stage_bytes;
  const int32_t* ids;   // [T, K] (layer), or [T] (projection: the adapter of each token)
  const float* topk_w;  // [T, K]
  uint32_t* ctl;
  bf16* act;     // [T * K, n]
  float* part1;  // [T * K][nt1][split][256]
  float* y32;    // [split][T * K][d]
  bf16* out;     // [T, d]
  // projection only
  const float* low_part;  // [low_splits][T][rank]
  float* low;             // [T, rank]
  const bf16* b;          // [n_adapters, rank, d]
  const float* scale;     // [n_adapters]
  int rank, low_splits, n_adapters;
  unsigned* status;
  unsigned long long limit_ns;
};

}  // namespace moe
