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

// Tile w of the large product: kAdapterTileGroup row tiles at a time, all column tiles of the
// group (they share the W panels of a wave through L2).
constexpr int kAdapterTileCols = 256, kAdapterTileGroup = 8;
__device__ __forceinline__ void adapter_tile_of(int w, int mt, int nt, int& m, int& n) {
  const int per = kAdapterTileGroup * nt, grp = w / per, r = w % per;
  const int gm = min(kAdapterTileGroup, mt - grp * kAdapterTileGroup);
  m = grp * kAdapterTileGroup + r % gm;
  n = r / gm;
}

// What is left to add after the products. Tiles whole ... of the large product were split along
// the contraction: part [others][split][2 CTAs][64][128 rows][4].
struct AdapterTileSums {
  int T, n_out, mt, nt, whole, split, others;
  const float* part;
  bf16* out;
};
// Units of the gradients (256 columns of one adapter's matrix) that pieces end inside: cuts[c]
// holds for the first piece that begins inside a unit which unit it is and the last piece with a
// part of it (l = -1 for other pieces). part [2 pieces][256 r]: piece c's first part in place
// 2 c, its last in 2 c + 1.
constexpr int kAdapterUnitCols = 256;
struct AdapterCut {
  int l, p, c0, end;
};
struct AdapterUnitSums {
  int D[2], r, pieces;
  const AdapterCut* cuts;
  const float* part;
  float* out[2];
};

// (a, b) as bf16 pairs hi + lo (+ what is left, returned in a and b): 8 bits of mantissa each.
__device__ __forceinline__ uint32_t take_bf16x2(float& a, float& b) {
  const uint32_t h = pack_bf16x2(a, b);
  a -= __uint_as_float(h << 16);
  b -= __uint_as_float(h & 0xffff0000u);
  return h;
}

}  // namespace moe
