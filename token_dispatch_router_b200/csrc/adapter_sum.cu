// The partial sums that the adapter products leave, added in order (results repeat bit for bit):
// tiles of the large product split along the contraction, and units of the gradients that pieces
// of the line end inside. One launch for both: behind the gradients each would add about 5 us of
// start and end to the call (2049 rows, 2880 x 2880: 84.6 us with two launches, 82.9 with one).
// Bound by reading the partials, which lie in L2.
#include "adapter.cuh"

namespace moe {

namespace {

constexpr int THREADS = 256;
constexpr int TILE_BLOCKS = kAdapterTileRows * kAdapterTileCols / 8 / THREADS;
constexpr int UNIT_PIECE = 2 * 4 * THREADS;  // values of a unit a CTA

// Eight columns of a row a thread.
__device__ __forceinline__ void sum_tile(const AdapterTileSums& g, int block) {
  const int other = block / TILE_BLOCKS;
  const int i = block % TILE_BLOCKS * THREADS + (int)threadIdx.x;
  const int lr = i % 128, c8 = i / 128 % (kAdapterTileCols / 8), half = i / 128 / (kAdapterTileCols / 8);
  int m, n;
  adapter_tile_of(g.whole + other, g.mt, g.nt, m, n);
  const int r = m * kAdapterTileRows + half * 128 + lr, col = n * kAdapterTileCols + c8 * 8;
  if (r >= g.T || col >= g.n_out) return;
  const float4* p0 = reinterpret_cast<const float4*>(g.part) +
                     ((size_t)other * g.split * 2 + half) * (kAdapterTileCols / 4) * 128 +
                     (size_t)c8 * 2 * 128 + lr;
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int s = 0; s < g.split; ++s) {
    const float4* pp = p0 + (size_t)s * 2 * (kAdapterTileCols / 4) * 128;
    const float4 u = __ldcg(pp), v = __ldcg(pp + 128);
    f[0] += u.x; f[1] += u.y; f[2] += u.z; f[3] += u.w;
    f[4] += v.x; f[5] += v.y; f[6] += v.z; f[7] += v.w;
  }
  *reinterpret_cast<uint4*>(g.out + (size_t)r * g.n_out + col) = pack16(f, bf16());
}

__device__ __forceinline__ void sum_unit(const AdapterUnitSums& g, int block) {
  const int size = kAdapterUnitCols * g.r, per = (size + UNIT_PIECE - 1) / UNIT_PIECE;
  const int c = block / per + 1;
  const AdapterCut cut = g.cuts[c];
  if (cut.l < 0) return;
  const int D = g.D[cut.p];
  float* out = g.out[cut.p] + (size_t)cut.l * D * g.r + (size_t)cut.c0 * (cut.p ? 1 : g.r);
  const float* p0 = g.part + (size_t)(2 * c - 1) * size;  // piece c - 1 ends here, c ... go on
  float4 v[2];
  int at[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    at[i] = block % per * UNIT_PIECE + (i * THREADS + (int)threadIdx.x) * 4;
    if (at[i] < size) v[i] = __ldcg(reinterpret_cast<const float4*>(p0 + at[i]));
  }
#pragma unroll 4
  for (int q = c; q <= cut.end; ++q)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (at[i] < size) {
        const float4 u =
            __ldcg(reinterpret_cast<const float4*>(g.part + (size_t)(2 * q) * size + at[i]));
        v[i].x += u.x; v[i].y += u.y; v[i].z += u.z; v[i].w += u.w;
      }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (at[i] >= size) continue;
    // [column][r] or [r][256 columns]; columns behind the last were not written
    const int col = cut.p ? at[i] % kAdapterUnitCols : at[i] / g.r;
    if (cut.c0 + col >= D) continue;
    *reinterpret_cast<float4*>(
        cut.p ? out + (size_t)(at[i] / kAdapterUnitCols) * D + col : out + at[i]) = v[i];
  }
}

__global__ void __launch_bounds__(THREADS)
    adapter_sum_kernel(const AdapterTileSums a, const AdapterUnitSums b, int tile_blocks) {
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();
  if ((int)blockIdx.x < tile_blocks) sum_tile(a, blockIdx.x);
  else sum_unit(b, (int)blockIdx.x - tile_blocks);
}

}  // namespace

moe_status launch_adapter_sum(const AdapterTileSums& a, const AdapterUnitSums& b,
                              cudaStream_t st) {
  const int tiles = a.others * TILE_BLOCKS;
  const int per = (kAdapterUnitCols * b.r + UNIT_PIECE - 1) / UNIT_PIECE;
  const int units = b.pieces > 1 ? (b.pieces - 1) * per : 0;
  if (tiles + units == 0) return MOE_OK;
  launch_begin(K_ADAPTER_SUM, st);
  launch_kernel(adapter_sum_kernel, dim3((unsigned)(tiles + units)), dim3(THREADS), 0, st, 1, a, b,
                tiles);
  return launch_end(K_ADAPTER_SUM, st);
}

}  // namespace moe
