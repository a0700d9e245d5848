// Shared pieces of the adapter kernels: the table of adapters by row tile, predicated copies and
// the split of an fp32 value into bf16 terms.
#pragma once

#include <math.h>

#include "tc_ptx.cuh"

namespace moe {

// The table of the large product's 256-row tiles. For each: how many adapters have rows in it, which
// ones, and for each of them the rows (bit r % 32 of word r / 32) that are NOT its own. A tile has
// room for as many as there can be, so that 2^24 rows of one adapter take 10 MB and not 605.
constexpr int kAdapterTileRows = 256;
struct AdapterTiles {
  int32_t* at;
  int most;  // adapters of a tile at most, rounded up to 4: words of a tile stay 16-byte aligned
  __host__ __device__ static int most_of(int n_adapters) {
    return ((n_adapters < kAdapterTileRows ? n_adapters : kAdapterTileRows) + 3) / 4 * 4;
  }
  __host__ __device__ static size_t bytes(int n_tiles, int n_adapters) {
    return (size_t)n_tiles * (4 + 9 * most_of(n_adapters)) * 4;
  }
  __device__ __forceinline__ int32_t* count(int m) const {
    return at + (size_t)m * (4 + 9 * most);
  }
  __device__ __forceinline__ int32_t* ids(int m) const { return count(m) + 4; }
  __device__ __forceinline__ uint32_t* off(int m, int i) const {
    return reinterpret_cast<uint32_t*>(ids(m) + most + 8 * i);
  }
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

// A value as N bf16 terms that add up to it: N = 2 to 2^-16 of it, N = 3 exactly (both above
// 2^-100). Each term has the value's sign and none is zero unless the value is, so a product with
// an infinity comes out as the value's own would, term by term (rounded terms leave a rest of the
// other sign, or of zero: inf - inf, 0 inf). So bits are cut off rather than rounded, which leaves
// the largest finite values finite, too; where nothing is left for a term, it shares the one before
// (halves are exact); and an infinity or NaN is itself in every term.
template <int N>
__device__ __forceinline__ void bf16_terms(float v, float (&t)[N]) {
  float rest = v;
#pragma unroll
  for (int i = 0; i < N - 1; ++i) {
    t[i] = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
    rest -= t[i];
  }
  t[N - 1] = rest;  // rounded where it is packed
#pragma unroll
  for (int i = 1; i < N; ++i)
    if (t[i] == 0.f && fabsf(t[i - 1]) >= 0x1p-120f) t[i] = t[i - 1] *= 0.5f;
  if (!(fabsf(v) < INFINITY))
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = v;
}

// (a, b) as N packed pairs of such terms.
template <int N>
__device__ __forceinline__ void bf16x2_terms(float a, float b, uint32_t (&h)[N]) {
  float s[N], t[N];
  bf16_terms<N>(a, s);
  bf16_terms<N>(b, t);
#pragma unroll
  for (int i = 0; i < N; ++i) h[i] = pack_bf16x2(s[i], t[i]);
}

}  // namespace moe
