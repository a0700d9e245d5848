// Arguments shared by the single-CTA and CTA-pair grouped-GEMM kernels, and the host
// helper that encodes their TMA tensor maps.
#pragma once

#include "common.cuh"

namespace moe {

struct GemmArgs {
  const int32_t* offsets;  // [E + 1] expert-major row offsets
  const int32_t* p2a;      // gate/up: slot -> flat assignment (token = a / K)
  const uint8_t* x;        // gate/up: token rows gathered by cp.async
  long long x_row_bytes;
  bf16* out;
  int ld_out;    // elements per output row
  int n_out;     // valid output columns
  int out_tile;  // output columns per tile (128 gate/up, 256 down)
  int n_tiles;
  int kblocks;   // contraction / 64
  int kb_split;  // backward dX: k-blocks below it read the first B map, the rest the second
  int E, K, T;
  unsigned* status;
  unsigned long long limit_ns;
  bf16* h_out;  // gate/up, single CTA: if not NULL, also the pre-activations (g | u) per row
};

// bf16 tensor of `rank` dims (at most 5, innermost first), 128-byte swizzle, zero fill out of
// bounds; L2 fetches of 256 bytes (wide_fetch) or 64.
bool make_map(CUtensorMap* m, const void* ptr, int rank, const uint64_t* dims,
              const uint64_t* strides_bytes, const uint32_t* box, bool wide_fetch = true);

// Matrices [count][rows][cols] seen as 64-column pieces: dims (64, rows, cols / 64, count), so
// that one copy brings `piece_box` pieces of `row_box` rows one after another, each in the
// swizzled layout of a 64-wide operand tile (rows or pieces past the end are zeros).
// L2 fetches are 256 bytes where rows start on such a boundary; elsewhere a row's 256-byte piece
// would fetch twice its bytes (streaming 92160 rows, two pieces a copy: 2880 columns 4.9 TB/s
// with wide fetches, 5.9 without; 2048 columns 6.3 with, 5.3 without).
inline bool make_piece_map(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols,
                           uint64_t count, uint32_t row_box, uint32_t piece_box) {
  const uint64_t dims[4] = {64, rows, cols / 64, count};
  const uint64_t strides[3] = {cols * 2, 128, rows * cols * 2};
  const uint32_t box[4] = {64, row_box, piece_box, 1};
  return make_map(m, ptr, 4, dims, strides, box, cols * 2 % 256 == 0);
}

}  // namespace moe
