// The low-rank halves of the adapter products:
//
//   grouped:  low[t] = scale_l in[t] M_l, l = ids[t], for rows grouped by adapter
//             (forward: in = x, M = A_l [d_in, r]; backward: in = d_y, M = B_l^T, B_l [r, d_out])
//   few:      partial sums of x[t] A_l for at most 128 rows, and the control words of the
//             kernel that follows
//   outer:    dA_l = sum_t x[t]^T d_low[t],  dB_l = sum_t low[t]^T d_y[t], t over l's rows
//
// All are bound by reading the wide rows (r is 8 ... 128, the rows are thousands wide), so they
// use the warp-level MMA (16 x 8 tiles fit the rank) fed by cp.async. Rows are grouped by
// adapter with the layer's stable permutation, so a tile never mixes adapters.
#include "adapter.cuh"
#include "few.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int THREADS = 128;
constexpr int ROWS = 64;   // rows of a grouped tile: 16 a warp
constexpr int KC = 64;     // contraction per stage
constexpr int STAGES = 4;
constexpr int SPLIT = 4;   // CTAs of a cluster that split the contraction

// ------------------------------------------------------------------ grouped
struct LowArgs {
  const bf16* in;   // [T, D]
  const bf16* m;    // [L, D, r], or [L, r, D] (TRANS)
  const int32_t* ids;
  const int32_t* offsets;  // [L + 1]
  const int32_t* rows;     // slot -> row
  const float* scale;
  float* low;      // [T, r]
  bf16* planes;    // NULL, or low in slot order as three bf16 terms: [3][T][r]
  const float* low2;  // with planes: another [T, r] ...
  bf16* planes2;      // ... put into slot order the same way
  bf16* terms;        // [2][T][r]: low as two bf16 terms
  AdapterTile* tiles; // [ceil(T / 256)]
  int tile_clusters;  // clusters up to here make low, those behind the table of tiles
  uint32_t* clear;    // words to zero for the kernel that follows (or none)
  int n_clear;
  int T, D, r, L;
};

// Where the 16-byte piece c of row r lies in a tile of NT pieces a row, so that the eight rows
// that one ldmatrix phase reads fall on distinct banks.
template <int NT>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  const int x = NT >= 8 ? r & 7 : NT == 4 ? (r >> 1) & 3 : (r >> 2) & 1;
  return (uint32_t)(r * (NT * 16) + ((c ^ x) << 4));
}

// Adapter l and first slot of row tile `tile` (ROWS rows); l = -1 past the last tile.
__device__ __forceinline__ void find_tile(const int32_t* offsets, int L, int tile, int rows,
                                          int* s_l, int* s_first) {
  const int lane = threadIdx.x & 31;
  int run = 0;
  for (int l0 = 0; l0 < L; l0 += 32) {
    const int l = l0 + lane;
    const int lo = l < L ? offsets[l] : 0, hi = l < L ? offsets[l + 1] : 0;
    const int n = (hi - lo + rows - 1) / rows;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int mine = run + incl - n;
    if (n > 0 && tile >= mine && tile < mine + n) {
      *s_l = l;
      *s_first = lo + (tile - mine) * rows;
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// Entry `m` of the table of tiles: which adapters have rows in 256 m ..., and which rows.
__device__ __forceinline__ void make_tile(int m, const LowArgs& g, uint8_t* smem) {
  const int r0 = m * kAdapterTileRows, tid = threadIdx.x, lane = tid & 31;
  if (r0 >= g.T) return;
  uint32_t* own = reinterpret_cast<uint32_t*>(smem);  // [L][8]
  for (int i = tid; i < g.L * 8; i += THREADS) own[i] = 0u;
  __syncthreads();
  for (int r = tid; r < kAdapterTileRows && r0 + r < g.T; r += THREADS) {
    const int l = g.ids[r0 + r];
    if (l >= 0 && l < g.L) atomicOr(&own[l * 8 + (r >> 5)], 1u << (r & 31));
  }
  __syncthreads();
  if (tid >= 32) return;
  AdapterTile* t = g.tiles + m;
  int n = 0;
  for (int l0 = 0; l0 < g.L; l0 += 32) {
    const int l = l0 + lane;
    uint32_t any = 0;
    if (l < g.L)
#pragma unroll
      for (int i = 0; i < 8; ++i) any |= own[l * 8 + i];
    const unsigned has = __ballot_sync(0xffffffffu, any != 0u);
    if (any != 0u) {
      const int at = n + __popc(has & lanemask_lt());
      t->id[at] = l;
#pragma unroll
      for (int i = 0; i < 8; ++i) t->off[at][i] = ~own[l * 8 + i];
    }
    n += __popc(has);
  }
  if (lane == 0) t->n = n;
}

// NT: 8-column blocks of the rank, rounded up to 2, 4, 8 or 16.
template <bool TRANS, int NT>
__global__ void __launch_bounds__(THREADS) adapter_low_kernel(const LowArgs g) {
  constexpr int X_BYTES = ROWS * KC * 2, M_BYTES = KC * NT * 8 * 2, ST = X_BYTES + M_BYTES;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_l, s_first, s_row[ROWS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank();
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();
  for (int i = blockIdx.x * THREADS + tid; i < g.n_clear; i += gridDim.x * THREADS) g.clear[i] = 0u;
  if ((int)cluster_id_x() >= g.tile_clusters) {
    make_tile(((int)cluster_id_x() - g.tile_clusters) * SPLIT + rank, g, smem);
    return;  // the whole cluster
  }
  // rows without an adapter
  for (int t = blockIdx.x * THREADS + tid; t < g.T; t += gridDim.x * THREADS) {
    const int l = g.ids[t];
    if (l < 0 || l >= g.L)
      for (int j = 0; j < g.r; j += 4)
        *reinterpret_cast<float4*>(g.low + (size_t)t * g.r + j) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (tid == 0) s_l = -1;
  __syncthreads();
  if (warp == 0) find_tile(g.offsets, g.L, (int)cluster_id_x(), ROWS, &s_l, &s_first);
  __syncthreads();
  const int l = s_l;
  if (l < 0) return;  // the whole cluster: past the last tile
  const int first = s_first, n = min(ROWS, g.offsets[l + 1] - first);
  if (tid < ROWS) s_row[tid] = tid < n ? g.rows[first + tid] : -1;
  __syncthreads();

  const int kblocks = g.D / KC;
  const int kb0 = rank * kblocks / SPLIT, kb1 = (rank + 1) * kblocks / SPLIT;
  const uint32_t sb = saddr(smem);
  // this thread's pieces of the x tile: rows tid / 8 + 16 i, 16-byte piece tid % 8
  const int pc = tid & 7, pr = tid >> 3;
  const bf16* src[4];
  uint32_t dst[4];
  bool on[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = pr + 16 * i, t = s_row[r];
    on[i] = t >= 0;
    src[i] = g.in + (size_t)(on[i] ? t : 0) * g.D + pc * 8;
    dst[i] = (uint32_t)(r * 128 + ((pc ^ (r & 7)) << 4));
  }
  const bf16* ml = g.m + (size_t)l * g.D * g.r;
  auto load = [&](int kb, int stage) {
    const uint32_t xs = sb + stage * ST, ms = xs + X_BYTES;
#pragma unroll
    for (int i = 0; i < 4; ++i) cp_async16_if(xs + dst[i], src[i] + (size_t)kb * KC, on[i]);
    if (TRANS) {  // [NT * 8 rank rows][KC], swizzled
      for (int i = tid; i < NT * 8 * 8; i += THREADS) {
        const int j = i >> 3, c = i & 7;
        const bool real = j < g.r;
        cp_async16_if(ms + j * 128 + ((c ^ (j & 7)) << 4),
                      ml + (size_t)(real ? j : 0) * g.D + kb * KC + c * 8, real);
      }
    } else {  // [KC][NT * 8]
      for (int i = tid; i < KC * NT; i += THREADS) {
        const int k = i / NT, c = i % NT;
        const bool real = c * 8 < g.r;
        cp_async16_if(ms + piece<NT>(k, c),
                      ml + (size_t)(kb * KC + k) * g.r + (real ? c * 8 : 0), real);
      }
    }
  };
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) {
    if (kb0 + s < kb1) load(kb0 + s, s);
    cp_async_commit();
  }
  for (int kb = kb0; kb < kb1; ++kb) {
    cp_async_wait<STAGES - 2>();
    __syncthreads();  // the stage has landed for every thread; the one before is free
    if (kb + STAGES - 1 < kb1) load(kb + STAGES - 1, (kb - kb0 + STAGES - 1) % STAGES);
    cp_async_commit();
    const uint32_t xs = sb + ((kb - kb0) % STAGES) * ST, ms = xs + X_BYTES;
#pragma unroll
    for (int kk = 0; kk < KC / 16; ++kk) {
      uint32_t a[4];
      {
        const int r = warp * 16 + (lane & 15), c = kk * 2 + (lane >> 4);
        ldmatrix4(a, xs + r * 128 + ((c ^ (r & 7)) << 4));
      }
#pragma unroll
      for (int i = 0; i < NT; i += 2) {
        uint32_t b[4];
        if (TRANS) {
          const int j = i * 8 + (lane & 7) + ((lane >> 4) << 3), c = kk * 2 + ((lane >> 3) & 1);
          ldmatrix4(b, ms + j * 128 + ((c ^ (j & 7)) << 4));
        } else {
          const int k = kk * 16 + (lane & 15), c = i + (lane >> 4);
          ldmatrix4t(b, ms + piece<NT>(k, c));
        }
        mma16816(acc[i], a, b[0], b[1]);
        mma16816(acc[i + 1], a, b[2], b[3]);
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);  // [ROWS][NT * 8]
  {
    const int r = warp * 16 + (lane >> 2), c = 2 * (lane & 3);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      *reinterpret_cast<float2*>(part + r * (NT * 8) + i * 8 + c) = make_float2(acc[i][0], acc[i][1]);
      *reinterpret_cast<float2*>(part + (r + 8) * (NT * 8) + i * 8 + c) =
          make_float2(acc[i][2], acc[i][3]);
    }
  }
  cluster_sync();
  // this rank's share of the rows: the four partials in rank order
  const float sc = g.scale[l];
  uint32_t peer[SPLIT];
#pragma unroll
  for (int q = 0; q < SPLIT; ++q) peer[q] = map_rank(sb, (uint32_t)q);
  for (int i = tid; i < ROWS / SPLIT * (g.r / 2); i += THREADS) {
    const int r = rank * (ROWS / SPLIT) + i / (g.r / 2), j = (i % (g.r / 2)) * 2;
    if (r >= n) continue;
    const uint32_t at = (uint32_t)((r * (NT * 8) + j) * 4);
    float v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int q = 0; q < SPLIT; ++q) {
      v0 += ld_dsmem_f32(peer[q] + at);
      v1 += ld_dsmem_f32(peer[q] + at + 4);
    }
    v0 *= sc;
    v1 *= sc;
    const size_t o = (size_t)s_row[r] * g.r + j;
    *reinterpret_cast<float2*>(g.low + o) = make_float2(v0, v1);
    {
      float a0 = v0, a1 = v1;
      *reinterpret_cast<uint32_t*>(g.terms + o) = take_bf16x2(a0, a1);
      *reinterpret_cast<uint32_t*>(g.terms + (size_t)g.T * g.r + o) = pack_bf16x2(a0, a1);
    }
    if (g.planes != nullptr) {
      const size_t slot = (size_t)(first + r) * g.r + j, plane = (size_t)g.T * g.r;
      float2 w = *reinterpret_cast<const float2*>(g.low2 + o);
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        *reinterpret_cast<uint32_t*>(g.planes + p * plane + slot) = take_bf16x2(v0, v1);
        *reinterpret_cast<uint32_t*>(g.planes2 + p * plane + slot) = take_bf16x2(w.x, w.y);
      }
    }
  }
  __syncwarp();
  cluster_sync();  // no rank leaves while its partial may be read
}

template <bool TRANS, int NT>
moe_status run_low(LowArgs a, cudaStream_t st) {
  auto kern = adapter_low_kernel<TRANS, NT>;
  const int smem = STAGES * (ROWS * KC * 2 + KC * NT * 16);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return MOE_ERR_CUDA;
  // at most T / ROWS whole tiles and one ragged tile an adapter (or a row)
  const int ragged = a.L < a.T ? a.L : a.T;
  a.tile_clusters = a.T / ROWS + ragged;
  const int table = (a.T + SPLIT * kAdapterTileRows - 1) / (SPLIT * kAdapterTileRows);
  launch_begin(K_ADAPTER_LOW, st);
  launch_kernel(kern, dim3((unsigned)(SPLIT * (a.tile_clusters + table))), dim3(THREADS),
                (size_t)smem, st, SPLIT, a);
  return launch_end(K_ADAPTER_LOW, st);
}

template <bool TRANS>
moe_status run_low_nt(const LowArgs& a, cudaStream_t st) {
  if (a.r <= 16) return run_low<TRANS, 2>(a, st);
  if (a.r <= 32) return run_low<TRANS, 4>(a, st);
  if (a.r <= 64) return run_low<TRANS, 8>(a, st);
  return run_low<TRANS, 16>(a, st);
}

// ------------------------------------------------------------------ few rows
struct LowFewArgs {
  const bf16* x;
  const bf16* a;
  const int32_t* ids;
  float* part;  // [splits][T][r]
  uint32_t* clear;
  int n_clear;
  int T, D, r, L, splits;
  unsigned* status;
};

// CTA (row t, split s): eight rank values a thread, the contraction over the threads.
__global__ void __launch_bounds__(THREADS) adapter_low_few_kernel(const LowFewArgs g) {
  __shared__ float xs[1024];
  __shared__ float red[THREADS * 8];
  const int tid = threadIdx.x, t = blockIdx.x, s = blockIdx.y;
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();
  const int bid = blockIdx.y * gridDim.x + blockIdx.x, nb = gridDim.x * gridDim.y;
  for (int i = bid * THREADS + tid; i < g.n_clear; i += nb * THREADS) g.clear[i] = 0u;
  const int l = g.ids[t];
  if (l < 0 || l >= g.L) {
    if (l != -1 && tid == 0 && s == 0) report(g.status, MOE_ERR_DEVICE_INDEX);
    return;  // nobody reads this row's partials
  }
  const int rc = g.r / 8, step = THREADS / rc;
  const int c = tid % rc, k_t = tid / rc;
  const int k0 = (int)((long long)s * (g.D / 8) / g.splits) * 8;
  const int k1 = (int)((long long)(s + 1) * (g.D / 8) / g.splits) * 8;
  const bf16* al = g.a + (size_t)l * g.D * g.r;
  float acc[8];
#pragma unroll
  for (int v = 0; v < 8; ++v) acc[v] = 0.f;
  for (int kc = k0; kc < k1; kc += 1024) {
    const int nk = min(1024, k1 - kc);
    __syncthreads();
    for (int i = tid * 8; i < nk; i += THREADS * 8) {
      float f[8];
      unpack16(*reinterpret_cast<const uint4*>(g.x + (size_t)t * g.D + kc + i), f, bf16());
#pragma unroll
      for (int v = 0; v < 8; ++v) xs[i + v] = f[v];
    }
    __syncthreads();
    if (k_t < step) {
#pragma unroll 4
      for (int k = k_t; k < nk; k += step) {
        float f[8];
        unpack16(*reinterpret_cast<const uint4*>(al + (size_t)(kc + k) * g.r + c * 8), f, bf16());
#pragma unroll
        for (int v = 0; v < 8; ++v) acc[v] = fmaf(xs[k], f[v], acc[v]);
      }
    }
  }
  if (k_t < step)
#pragma unroll
    for (int v = 0; v < 8; ++v) red[k_t * g.r + c * 8 + v] = acc[v];
  __syncthreads();
  for (int j = tid; j < g.r; j += THREADS) {
    float sum = 0.f;
    for (int q = 0; q < step; ++q) sum += red[q * g.r + j];
    g.part[((size_t)s * g.T + t) * g.r + j] = sum;
  }
}

// ------------------------------------------------------------------ outer products
constexpr int OC = 128;   // columns of a unit: 32 a warp
constexpr int OT = 32;    // rows per stage
constexpr int OSTAGES = 3;

struct OuterArgs {
  const bf16* big[2];     // x [T, D0], d_y [T, D1]
  const bf16* planes[2];  // [3][T][r] in slot order
  float* out[2];          // dA [L, D0, r], dB [L, r, D1]
  int D[2], tiles[2];     // widths and their 128-column tiles
  const int32_t* offsets;
  const int32_t* rows;
  float* part;        // [chunk][D0 + D1][r]: adapters of several chunks
  uint32_t* arrived;  // [L][tiles0 + tiles1], zero when the kernel starts
  int T, r, L, chunk;
};

template <int NT>
__global__ void __launch_bounds__(THREADS) adapter_outer_kernel(const OuterArgs g) {
  constexpr int B_BYTES = OT * OC * 2, P_BYTES = OT * NT * 16, ST = B_BYTES + 3 * P_BYTES;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_l, s_i, s_n, s_base, s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();
  const int nct = g.tiles[0] + g.tiles[1];
  const int cg = blockIdx.x / nct, ct = blockIdx.x % nct;  // chunk, column tile
  if (tid == 0) s_l = -1;
  __syncthreads();
  if (warp == 0) {  // chunk cg: adapter, index in it, its chunks, first partial slot
    int run = 0, mrun = 0;
    for (int l0 = 0; l0 < g.L; l0 += 32) {
      const int l = l0 + lane;
      const int c = l < g.L ? g.offsets[l + 1] - g.offsets[l] : 0;
      const int n = l < g.L ? max(1, (c + g.chunk - 1) / g.chunk) : 0;
      const int m = n > 1 ? n : 0;
      int incl = n, mincl = m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        const int w = __shfl_up_sync(0xffffffffu, mincl, o);
        if (lane >= o) {
          incl += v;
          mincl += w;
        }
      }
      const int mine = run + incl - n;
      if (cg >= mine && cg < mine + n) {
        s_l = l;
        s_i = cg - mine;
        s_n = n;
        s_base = mrun + mincl - m;
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
      mrun += __shfl_sync(0xffffffffu, mincl, 31);
    }
  }
  __syncthreads();
  const int l = s_l;
  if (l < 0) return;
  const int p = ct >= g.tiles[0] ? 1 : 0;
  const int c0 = (ct - (p ? g.tiles[0] : 0)) * OC, D = g.D[p];
  const int lo = g.offsets[l] + s_i * g.chunk;
  const int n = max(0, min(g.chunk, g.offsets[l + 1] - lo));
  const bf16* big = g.big[p];
  const bf16* planes = g.planes[p];
  const size_t plane = (size_t)g.T * g.r;
  const uint32_t sb = saddr(smem);
  const int cc = tid & 15, cr = tid >> 4;  // 16-byte piece of a row, rows cr + 8 i
  const bool col_on = c0 + cc * 8 < D;
  auto load = [&](int r0, int stage) {
    const uint32_t bs = sb + stage * ST, ps = bs + B_BYTES;
#pragma unroll
    for (int i = 0; i < OT / 8; ++i) {
      const int r = cr + 8 * i;
      const bool on = r0 + r < n && col_on;
      const int t = on ? g.rows[lo + r0 + r] : 0;
      cp_async16_if(bs + r * 256 + ((cc ^ (r & 7)) << 4),
                    big + (size_t)t * D + (on ? c0 + cc * 8 : 0), on);
    }
    for (int i = tid; i < 3 * OT * NT; i += THREADS) {
      const int q = i / (OT * NT), r = i / NT % OT, c = i % NT;
      const bool on = r0 + r < n && c * 8 < g.r;
      cp_async16_if(ps + q * P_BYTES + piece<NT>(r, c),
                    planes + q * plane + (on ? (size_t)(lo + r0 + r) * g.r + c * 8 : 0), on);
    }
  };
  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][i][j] = 0.f;
  const int steps = (n + OT - 1) / OT;
#pragma unroll
  for (int s = 0; s < OSTAGES - 1; ++s) {
    if (s < steps) load(s * OT, s);
    cp_async_commit();
  }
  for (int s = 0; s < steps; ++s) {
    cp_async_wait<OSTAGES - 2>();
    __syncthreads();
    if (s + OSTAGES - 1 < steps) load((s + OSTAGES - 1) * OT, (s + OSTAGES - 1) % OSTAGES);
    cp_async_commit();
    const uint32_t bs = sb + (s % OSTAGES) * ST, ps = bs + B_BYTES;
#pragma unroll
    for (int kk = 0; kk < OT / 16; ++kk) {
      uint32_t a[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int k = kk * 16 + (lane & 7) + ((lane >> 4) << 3);
        const int c = warp * 4 + m * 2 + ((lane >> 3) & 1);
        ldmatrix4t(a[m], bs + k * 256 + ((c ^ (k & 7)) << 4));
      }
#pragma unroll
      for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int i = 0; i < NT; i += 2) {
          uint32_t b[4];
          ldmatrix4t(b, ps + q * P_BYTES + piece<NT>(kk * 16 + (lane & 15), i + (lane >> 4)));
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            mma16816(acc[m][i], a[m], b[0], b[1]);
            mma16816(acc[m][i + 1], a[m], b[2], b[3]);
          }
        }
    }
  }
  cp_async_wait<0>();
  // rows of the accumulators are columns of `big`: c = c0 + 32 warp + 16 m + lane / 4 (+ 8)
  const size_t wide = (size_t)(g.D[0] + g.D[1]);
  const bool direct = s_n == 1;
  float* part = direct ? nullptr
                       : g.part + ((size_t)(s_base + s_i) * wide + (p ? g.D[0] : 0)) * g.r;
  float* out = g.out[p] + (size_t)l * D * g.r;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + warp * 32 + m * 16 + (lane >> 2) + 8 * h;
      if (c >= D) continue;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int j = i * 8 + 2 * (lane & 3);
        if (j >= g.r) continue;
        const float v0 = acc[m][i][2 * h], v1 = acc[m][i][2 * h + 1];
        if (!direct) {
          *reinterpret_cast<float2*>(part + (size_t)c * g.r + j) = make_float2(v0, v1);
        } else if (p == 0) {
          *reinterpret_cast<float2*>(out + (size_t)c * g.r + j) = make_float2(v0, v1);
        } else {
          out[(size_t)j * D + c] = v0;
          out[(size_t)(j + 1) * D + c] = v1;
        }
      }
    }
  if (direct) return;
  // the adapter's last chunk to arrive adds them up, in chunk order
  __threadfence();
  __syncthreads();
  if (tid == 0)
    s_last = atomicAdd(g.arrived + (size_t)l * nct + ct, 1u) == (unsigned)(s_n - 1);
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const float* p0 = g.part + ((size_t)s_base * wide + (p ? g.D[0] : 0)) * g.r;
  const int w = min(OC, D - c0);
  for (int i = tid; i < w * g.r; i += THREADS) {
    // consecutive threads on consecutive outputs
    const int c = c0 + (p == 0 ? i / g.r : i % w), j = p == 0 ? i % g.r : i / w;
    float v = 0.f;
    for (int q = 0; q < s_n; ++q) v += __ldcg(p0 + (size_t)q * wide * g.r + (size_t)c * g.r + j);
    out[p == 0 ? (size_t)c * g.r + j : (size_t)j * D + c] = v;
  }
}

template <int NT>
moe_status run_outer(const OuterArgs& a, cudaStream_t st) {
  auto kern = adapter_outer_kernel<NT>;
  const int smem = OSTAGES * (OT * OC * 2 + 3 * OT * NT * 16);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return MOE_ERR_CUDA;
  launch_begin(K_ADAPTER_OUTER, st);
  launch_kernel(kern, dim3((unsigned)((a.T / a.chunk + a.L) * (a.tiles[0] + a.tiles[1]))),
                dim3(THREADS), (size_t)smem, st, 1, a);
  return launch_end(K_ADAPTER_OUTER, st);
}

}  // namespace

// Rows of an outer-product unit: enough units for four a SM, at least 512 rows each.
static int outer_chunk(int T, int d_in, int d_out) {
  const long long tiles = (d_in + OC - 1) / OC + (d_out + OC - 1) / OC;
  long long c = (long long)T * tiles / (4 * 148);
  c = (c + 63) / 64 * 64;
  return (int)(c < 512 ? 512 : c);
}

// Partial sums of adapters with more than one chunk: at most 2 T / chunk chunks.
size_t adapter_outer_part_bytes(int T, int d_in, int d_out, int r) {
  const size_t chunks = 2 * (size_t)(T / outer_chunk(T, d_in, d_out));
  return chunks * (size_t)(d_in + d_out) * r * 4;
}
size_t adapter_outer_arrived_words(int d_in, int d_out, int L) {
  return (size_t)L * ((d_in + OC - 1) / OC + (d_out + OC - 1) / OC);
}

moe_status launch_adapter_low(bool trans, int T, int D, int r, int L, const void* in,
                              const void* m, const int32_t* ids, const int32_t* offsets,
                              const int32_t* rows, const float* scale, float* low, void* planes,
                              const float* low2, void* planes2, void* terms,
                              AdapterTile* tiles, uint32_t* clear, int n_clear,
                              cudaStream_t st) {
  const LowArgs a{(const bf16*)in, (const bf16*)m,  ids,          offsets, rows, scale, low,
                  (bf16*)planes,   low2,            (bf16*)planes2, (bf16*)terms, tiles, 0,
                  clear,           n_clear,         T,            D,       r,    L};
  return trans ? run_low_nt<true>(a, st) : run_low_nt<false>(a, st);
}

moe_status launch_adapter_low_few(int T, int D, int r, int L, int splits, const void* x,
                                  const void* a, const int32_t* ids, float* part,
                                  uint32_t* clear, int n_clear, cudaStream_t st) {
  const LowFewArgs f{(const bf16*)x, (const bf16*)a, ids, part, clear, n_clear, T, D, r, L,
                     splits, device_status_ptr()};
  launch_begin(K_ADAPTER_LOW_FEW, st);
  launch_kernel(adapter_low_few_kernel, dim3((unsigned)T, (unsigned)splits), dim3(THREADS), 0, st,
                1, f);
  return launch_end(K_ADAPTER_LOW_FEW, st);
}

moe_status launch_adapter_outer(int T, int d_in, int d_out, int r, int L, const void* x,
                                const void* d_y, const void* planes_d_low,
                                const void* planes_low, const int32_t* offsets,
                                const int32_t* rows, float* d_a, float* d_b, float* part,
                                uint32_t* arrived, cudaStream_t st) {
  OuterArgs a = {};
  a.big[0] = (const bf16*)x;
  a.big[1] = (const bf16*)d_y;
  a.planes[0] = (const bf16*)planes_d_low;
  a.planes[1] = (const bf16*)planes_low;
  a.out[0] = d_a;
  a.out[1] = d_b;
  a.D[0] = d_in;
  a.D[1] = d_out;
  a.tiles[0] = (d_in + OC - 1) / OC;
  a.tiles[1] = (d_out + OC - 1) / OC;
  a.offsets = offsets;
  a.rows = rows;
  a.part = part;
  a.arrived = arrived;
  a.T = T;
  a.r = r;
  a.L = L;
  a.chunk = outer_chunk(T, d_in, d_out);
  if (r <= 16) return run_outer<2>(a, st);
  if (r <= 32) return run_outer<4>(a, st);
  if (r <= 64) return run_outer<8>(a, st);
  return run_outer<16>(a, st);
}

}  // namespace moe
