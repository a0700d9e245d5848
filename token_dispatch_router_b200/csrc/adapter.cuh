// Shared pieces of the adapter kernels: the table of adapters by row tile, predicated copies and
// the split of an fp32 value into bf16 terms.
#pragma once

#include "tc_ptx.cuh"

namespace moe {

// The adapters that have rows in a 256-row tile of the large product, and for each the rows
// (bit r % 32 of word r / 32) that are NOT its own.
constexpr int kAdapterTileRows = 256;
struct AdapterTile {
  int n;
  int pad[3];
  int id[kAdapterTileRows];
  uint32_t off[kAdapterTileRows][8];
};

// (a, b) as bf16 pairs hi + lo (+ what is left, returned in a and b): 8 bits of mantissa each.
__device__ __forceinline__ uint32_t take_bf16x2(float& a, float& b) {
  const uint32_t h = pack_bf16x2(a, b);
  a -= __uint_as_float(h << 16);
  b -= __uint_as_float(h & 0xffff0000u);
  return h;
}

}  // namespace moe
