// Host side of the adapter products: workspace layouts and launch sequences.
//
//   forward,  few rows:         low partials -> product with the adapter term (two launches)
//   forward,  more rows:        group rows by adapter -> low -> product with the adapter term
//   backward:                   group -> d_low -> d_x product with the adapter term
//                               -> outer products d_A, d_B
// Grouping is the layer's stable permutation with one "expert" an adapter and K = 1; a row
// with id -1 belongs to none.
#include "adapter.cuh"
#include "few.cuh"
#include "few_args.cuh"

namespace moe {

size_t permute_scratch_bytes(const moe_shape& s);
moe_status launch_permute(const moe_shape& s, const int32_t* ids, int32_t* counts,
                          int32_t* offsets, int32_t* a2p, int32_t* p2a, const void* x,
                          void* x_perm, void* scratch, cudaStream_t st);
moe_status launch_adapter_few(const AdapterFewArgs& a, int d_in, const void* x, const void* w,
                              cudaStream_t st);
moe_status launch_adapter_low_few(int T, int D, int r, int L, int splits, const void* x,
                                  const void* a, const int32_t* ids, float* part,
                                  cudaStream_t st);
moe_status launch_adapter_low(bool trans, int T, int D, int r, int L, const void* in,
                              const void* m, const int32_t* ids, const int32_t* offsets,
                              const int32_t* rows, const float* scale, float* low, void* planes,
                              const float* low2, void* planes2, void* terms,
                              AdapterTiles tiles, cudaStream_t st);
moe_status launch_adapter_gemm(bool bwd, int T, int d_in, int d_out, int n_adapters, int rank,
                               const void* in, const void* w, AdapterTiles tiles,
                               const void* low, const void* m, void* out, float* part,
                               cudaStream_t st);
AdapterTileSums adapter_gemm_sums(int T, int k_dim, int n_out, void* out, const float* part);
size_t adapter_gemm_part_bytes(int T, int k_dim, int n_out);
size_t adapter_outer_part_bytes(int T, int r);
moe_status launch_adapter_outer(int T, int d_in, int d_out, int r, int L, const void* x,
                                const void* d_y, const void* planes_d_low,
                                const void* planes_low, const int32_t* offsets,
                                const int32_t* rows, float* d_a, float* d_b, float* part,
                                bool early, cudaStream_t st);
AdapterUnitSums adapter_outer_sums(int T, int d_in, int d_out, int r, float* d_a, float* d_b,
                                   const float* part);
moe_status launch_adapter_sum(const AdapterTileSums& a, const AdapterUnitSums& b,
                              cudaStream_t st);

namespace {

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Whether the forward takes the kernels for few rows. Their adapter terms are sums of a row at a
// time: their time grows with rows times rank, whoever's rows they are. The grouped kernels pay for
// every adapter that a tile's rows have (about 1 us, 2 at rank 128) and for three launches. How many
// there are is not known here: as many as there can be. Measured, few rows / grouped, us, and the
// limit's side (512 -> 3584, 2048 -> 2880, 4096 -> 4096):
//   64 rows of rank 64, 4 adapters    30 / 20    28 / 27    35 / 30   grouped
//   64 rows of rank 64, 32            30 / 50    29 / 59    36 / 69   few
//   128 rows of rank 16, 1            20 / 18    19 / 22    24 / 25   few
//   128 rows of rank 32, 16           31 / 31    30 / 38    37 / 45   few
//   128 rows of rank 64, 32           51 / 53    49 / 60    64 / 70   grouped
//   128 rows of rank 64, 128          67 / 166   60 / 193   95 / 203  few
//   128 rows of rank 128, 128        147 / 334  135 / 359  177 / 372  few
bool few_rows(const moe_adapter_shape& s) {
  if (s.T > kFewMaxTokens) return false;
  const int most = s.n_adapters < s.T ? s.n_adapters : s.T;
  return s.T * s.rank <= 2048 + 128 * most;
}

// Splits of the few-row low sums: two CTAs an SM over all rows, at least 64 of d_in each, 16 at most.
int low_few_splits(const moe_adapter_shape& s) {
  int n = 2 * sm_count() / (s.T > 0 ? s.T : 1);
  if (n > s.d_in / 64) n = s.d_in / 64;
  return n < 1 ? 1 : n > 16 ? 16 : n;
}

moe_shape group_shape(const moe_adapter_shape& s) {
  moe_shape g = {};
  g.T = s.T;
  g.d = 64;
  g.E = s.n_adapters;
  g.K = 1;
  g.dtype = MOE_BF16;
  return g;
}

struct Layout {
  size_t counts, offsets, a2p, rows, scratch;                    // grouping
  size_t tiles, terms, gemm_part;                                // for the large product
  size_t d_low, planes_d, planes_l, part, total_fwd, total;  // backward
};
Layout layout(const moe_adapter_shape& s) {
  Layout L;
  const size_t T = s.T, r = s.rank;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = up256(o + bytes);
    return at;
  };
  L.counts = take((size_t)s.n_adapters * 4);
  L.offsets = take(((size_t)s.n_adapters + 1) * 4);
  L.a2p = take(T * 4);
  L.rows = take(T * 4);
  L.scratch = take(permute_scratch_bytes(group_shape(s)));
  L.tiles = take(AdapterTiles::bytes((s.T + kAdapterTileRows - 1) / kAdapterTileRows, s.n_adapters));
  L.terms = take(2 * T * r * 2);
  const size_t pf = adapter_gemm_part_bytes(s.T, s.d_in, s.d_out);
  const size_t pb = adapter_gemm_part_bytes(s.T, s.d_out, s.d_in);
  L.gemm_part = take(pf > pb ? pf : pb);
  L.total_fwd = o;
  L.d_low = take(T * r * 4);
  L.planes_d = take(3 * T * r * 2);
  L.planes_l = take(3 * T * r * 2);
  L.part = take(adapter_outer_part_bytes(s.T, s.rank));
  L.total = o;
  return L;
}

AdapterTiles tiles_at(const moe_adapter_shape& s, const Layout& L, uint8_t* ws) {
  return AdapterTiles{(int32_t*)(ws + L.tiles), AdapterTiles::most_of(s.n_adapters)};
}

moe_status group(const moe_adapter_shape& s, const int32_t* ids, const Layout& L, uint8_t* ws,
                 cudaStream_t st) {
  return launch_permute(group_shape(s), ids, (int32_t*)(ws + L.counts),
                        (int32_t*)(ws + L.offsets), (int32_t*)(ws + L.a2p),
                        (int32_t*)(ws + L.rows), nullptr, nullptr, ws + L.scratch, st);
}

}  // namespace

size_t adapter_forward_bytes(const moe_adapter_shape& s) {
  return few_rows(s) ? up256((size_t)low_few_splits(s) * s.T * s.rank * 4)
                              : layout(s).total_fwd;
}
size_t adapter_backward_bytes(const moe_adapter_shape& s) { return layout(s).total; }

moe_status launch_adapter_forward(const moe_adapter_shape& s, const void* x, const void* w,
                                  const void* a, const void* b, const int32_t* ids,
                                  const float* scale, float* low, void* y, uint8_t* ws,
                                  cudaStream_t st) {
  moe_status r;
  if (few_rows(s)) {
    AdapterFewArgs f = {};
    f.T = s.T;
    f.d = s.d_out;
    f.ids = ids;
    f.out = (bf16*)y;
    f.low_part = (const float*)ws;
    f.low = low;
    f.b = (const bf16*)b;
    f.scale = scale;
    f.rank = s.rank;
    f.low_splits = low_few_splits(s);
    f.n_adapters = s.n_adapters;
    if ((r = launch_adapter_low_few(s.T, s.d_in, s.rank, s.n_adapters, f.low_splits, x, a, ids,
                                    (float*)ws, st)) != MOE_OK)
      return r;
    return launch_adapter_few(f, s.d_in, x, w, st);
  }
  const Layout L = layout(s);
  if ((r = group(s, ids, L, ws, st)) != MOE_OK) return r;
  if ((r = launch_adapter_low(false, s.T, s.d_in, s.rank, s.n_adapters, x, a, ids,
                              (const int32_t*)(ws + L.offsets), (const int32_t*)(ws + L.rows),
                              scale, low, nullptr, nullptr, nullptr, ws + L.terms,
                              tiles_at(s, L, ws), st)) != MOE_OK)
    return r;
  float* part = (float*)(ws + L.gemm_part);
  if ((r = launch_adapter_gemm(false, s.T, s.d_in, s.d_out, s.n_adapters, s.rank, x, w,
                               tiles_at(s, L, ws), ws + L.terms, b, y, part,
                               st)) != MOE_OK)
    return r;
  return launch_adapter_sum(adapter_gemm_sums(s.T, s.d_in, s.d_out, y, part), AdapterUnitSums{},
                            st);
}

moe_status launch_adapter_backward(const moe_adapter_shape& s, const void* d_y, const void* x,
                                   const void* w, const void* a, const void* b,
                                   const int32_t* ids, const float* scale, const float* low,
                                   void* d_x, float* d_a, float* d_b, uint8_t* ws,
                                   cudaStream_t st) {
  const Layout L = layout(s);
  const int32_t* offsets = (const int32_t*)(ws + L.offsets);
  const int32_t* rows = (const int32_t*)(ws + L.rows);
  float* d_low = (float*)(ws + L.d_low);
  moe_status r;
  if ((r = group(s, ids, L, ws, st)) != MOE_OK) return r;
  if ((r = launch_adapter_low(
           true, s.T, s.d_out, s.rank, s.n_adapters, d_y, b, ids, offsets, rows, scale, d_low,
           ws + L.planes_d, low, ws + L.planes_l, ws + L.terms, tiles_at(s, L, ws),
           st)) != MOE_OK)
    return r;
  float* gemm_part = (float*)(ws + L.gemm_part);
  float* part = (float*)(ws + L.part);
  if (d_x != nullptr &&
      (r = launch_adapter_gemm(true, s.T, s.d_in, s.d_out, s.n_adapters, s.rank, d_y, w,
                               tiles_at(s, L, ws), ws + L.terms, a, d_x,
                               gemm_part, st)) != MOE_OK)
    return r;
  // the outer products start as the large product's CTAs leave; what both leave is added last
  if ((r = launch_adapter_outer(s.T, s.d_in, s.d_out, s.rank, s.n_adapters, x, d_y,
                                ws + L.planes_d, ws + L.planes_l, offsets, rows, d_a, d_b, part,
                                d_x != nullptr, st)) != MOE_OK)
    return r;
  return launch_adapter_sum(d_x != nullptr ? adapter_gemm_sums(s.T, s.d_out, s.d_in, d_x, gemm_part)
                                           : AdapterTileSums{},
                            adapter_outer_sums(s.T, s.d_in, s.d_out, s.rank, d_a, d_b, part), st);
}

}  // namespace moe
