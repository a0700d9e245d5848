// The low-rank halves of the adapter products:
//
//   grouped:  low[t] = scale_l in[t] M_l, l = ids[t], for rows grouped by adapter
//             (forward: in = x, M = A_l [d_in, r]; backward: in = d_y, M = B_l^T, B_l [r, d_out])
//   few:      partial sums of x[t] A_l for at most 128 rows
//
// Bound by reading the wide rows once. The grouped form gives a cluster of four CTAs up to 128
// rows of one adapter (grouping is the layer's stable permutation, so a tile never mixes
// adapters) and splits the contraction over them: enough bytes in flight from few rows. Rows
// are gathered by cp.async, the adapter's matrix comes by TMA as it lies, the product runs on
// the tensor cores (M = rows, N = rank), and the four partials are added in rank order through
// distributed shared memory.
#include "adapter.cuh"
#include "few.cuh"
#include "ffn_args.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int ROWS = 128;  // rows of a grouped tile
constexpr int KC = 64;     // contraction per stage
constexpr int STAGES = 4;
constexpr int SPLIT = 4;   // CTAs of a cluster that split the contraction
constexpr int LOADERS = 128, THREADS = 192;  // four gather / store warps, MMA warp, TMA warp
constexpr int X_BYTES = ROWS * KC * 2;       // 16 KB
constexpr int M_CHUNK = 8192;                // 64 x 64 of the adapter's matrix

// ------------------------------------------------------------------ grouped
struct LowArgs {
  const bf16* in;   // [T, D]
  const int32_t* ids;
  const int32_t* offsets;  // [L + 1]
  const int32_t* rows;     // slot -> row
  const float* scale;
  float* low;      // [T, r]
  bf16* planes;    // NULL, or low in slot order as three bf16 terms: [3][T][r]
  const float* low2;  // with planes: another [T, r] ...
  bf16* planes2;      // ... put into slot order the same way
  bf16* terms;        // [2][T][r]: low as two bf16 terms
  AdapterTiles tiles; // [ceil(T / 256)]
  int tile_clusters;  // clusters up to here make low, those behind the table of tiles
  int T, D, r, L;
  int n_mma, nc;      // the rank rounded up to 16; its 64-wide pieces
  unsigned* status;
  unsigned long long limit_ns;
};

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
  int32_t* ids = g.tiles.ids(m);
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
      ids[at] = l;
      uint32_t* off = g.tiles.off(m, at);
#pragma unroll
      for (int i = 0; i < 8; ++i) off[i] = ~own[l * 8 + i];
    }
    n += __popc(has);
  }
  if (lane == 0) *g.tiles.count(m) = n;
}

// TRANS: the adapter's matrix is [r, D] (the backward's B_l), else [D, r].
template <bool TRANS>
__global__ void __launch_bounds__(THREADS)
    adapter_low_kernel(const __grid_constant__ CUtensorMap tmM, const LowArgs g) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[STAGES], empty[STAGES], done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_l, s_first, s_abort, s_row[ROWS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank();
  uint8_t* base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = saddr(base);
  const int st_bytes = X_BYTES + g.nc * M_CHUNK;
  volatile int* abort_flag = &s_abort;
  // The tensor core cuts what it adds to an accumulator off rather than rounding it: the k steps
  // go round four accumulators (two of a rank above 64), which are added in fp32, so that the
  // fp32 result stays near that of a rounded sum.
  const int accs = g.nc == 1 ? 4 : 2;
  uint32_t tcols = 32;
  while ((int)tcols < accs * g.n_mma) tcols *= 2;
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(saddr(&full[s]), LOADERS + 1);
      mbar_init(saddr(&empty[s]), 1);
    }
    mbar_init(saddr(&done), 1);
    s_abort = 0;
    s_l = -1;
    mbar_init_fence();
  }
  __syncthreads();
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();
  if ((int)cluster_id_x() >= g.tile_clusters) {
    make_tile(((int)cluster_id_x() - g.tile_clusters) * SPLIT + rank, g, base);
    return;  // the whole cluster
  }
  // rows without an adapter
  for (int t = blockIdx.x * THREADS + tid; t < g.T; t += SPLIT * g.tile_clusters * THREADS) {
    const int l = g.ids[t];
    if (l < 0 || l >= g.L)
      for (int j = 0; j < g.r; j += 4)
        *reinterpret_cast<float4*>(g.low + (size_t)t * g.r + j) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (warp == 0) find_tile(g.offsets, g.L, (int)cluster_id_x(), ROWS, &s_l, &s_first);
  __syncthreads();
  const int l = s_l;
  if (l < 0) return;  // the whole cluster: past the last tile
  if (warp == 4) tmem_alloc<1>(saddr(&s_tmem), tcols);
  const int first = s_first, n = min(ROWS, g.offsets[l + 1] - first);
  if (tid < ROWS) s_row[tid] = tid < n ? g.rows[first + tid] : -1;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int kblocks = g.D / KC;
  const int kb0 = rank * kblocks / SPLIT, kb1 = (rank + 1) * kblocks / SPLIT;
  const uint64_t limit = g.limit_ns;
  bool ok = true;

  if (warp < 4) {
    // ------------------------------------------------------------ gather
    // 16-byte piece tid % 8 of rows tid / 8 + 16 i: a warp copies whole 128-byte lines
    const int pc = tid & 7, pr = tid >> 3;
    const bf16* src[8];
    unsigned on = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = s_row[pr + 16 * i];
      if (t >= 0) on |= 1u << i;
      src[i] = g.in + (size_t)max(t, 0) * g.D + pc * 8;
    }
    const uint32_t dst0 = (uint32_t)(pr * 128 + ((pc ^ (pr & 7)) << 4));  // rows 16 apart: + 2 KB
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_warp(saddr(&empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) {
        ok = false;
        break;
      }
      const uint32_t xs = sb + stage * st_bytes + dst0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        cp_async16_if(xs + i * 2048, src[i] + (size_t)kb * KC, (on >> i & 1u) != 0);
      cp_async_arrive_noinc(saddr(&full[stage]));
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    cp_async_wait_all();
  } else if (warp == 4) {
    // ------------------------------------------------------------ MMA issuer
    // D fp32, A (rows) K-major bf16, B bf16: MN-major [k][r] or K-major [r][k] (TRANS)
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (TRANS ? 0u : 1u << 16) |
                           ((uint32_t)(g.n_mma >> 3) << 17) | (8u << 24);
    const uint64_t xd0 = desc_sw128(sb, 16, 1024);
    const uint64_t md0 = TRANS ? desc_sw128(sb + X_BYTES, 16, 1024)
                               : desc_sw128(sb + X_BYTES, M_CHUNK, 1024);
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_warp(saddr(&full[stage]), phase, abort_flag, g.status, limit)) break;
      fence_proxy_async_smem();  // the gathered rows (cp.async) -> MMA reads
      tc_fence_after();
      if (elect_one()) {
        const uint64_t so = (uint64_t)((stage * st_bytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < KC / 16; ++kk)
          tc_mma<1>(tmem + (uint32_t)((kk & (accs - 1)) * g.n_mma), xd0 + so + (uint64_t)(kk * 2),
                    md0 + so + (uint64_t)(kk * (TRANS ? 2 : 128)), idesc,
                    (kb > kb0 || kk >= accs) ? 1u : 0u);
        tc_commit<1>(saddr(&empty[stage]));
      }
      __syncwarp();
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (elect_one()) tc_commit<1>(saddr(&done));
  } else if (lane == 0) {
    // ------------------------------------------------------------ the adapter's matrix (TMA)
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_par = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(saddr(&empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) break;
      const uint32_t fb = saddr(&full[stage]), ms = sb + stage * st_bytes + X_BYTES;
      mbar_expect_tx(fb, (uint32_t)(g.nc * M_CHUNK));
      for (int c = 0; c < g.nc; ++c) {
        if (TRANS) tma_load_3d(ms + c * M_CHUNK, &tmM, kb * KC, 64 * c, l, fb);
        else tma_load_3d(ms + c * M_CHUNK, &tmM, 64 * c, kb * KC, l, fb);
      }
      issued_mask |= 1u << stage;
      issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    for (int s = 0; s < STAGES; ++s) {  // nothing of ours is in flight after this (bounded)
      if (!(issued_mask & (1u << s))) continue;
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try(saddr(&full[s]), (issued_par >> s) & 1u) && globaltimer_ns() - t0 < limit) {
      }
    }
  }
  __syncwarp();
  int w_ok = 0;
  if (lane == 0) w_ok = mbar_wait(saddr(&done), 0, nullptr, g.status, limit);
  ok = __shfl_sync(0xffffffffu, w_ok, 0) && ok;
  tc_fence_before();
  __syncthreads();  // every copy and MMA is done: the ring is free
  tc_fence_after();
  ok = ok && !*abort_flag;
  // the partial in shared memory: [row][pitch], a thread its row
  const int pitch = g.r + 4;
  float* part = reinterpret_cast<float*>(base);
  if (warp < 4) {
    for (int j = 0; j < g.r; j += 8) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.f;
      if (kb0 < kb1)  // else no k-block for this rank (d < 256)
        for (int c = 0; c < accs; ++c) {
          uint32_t v[8];
          tmem_ld8(tmem + (uint32_t)(c * g.n_mma + j) + ((uint32_t)(warp * 32) << 16), v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] += __uint_as_float(v[i]);
        }
      float4* o = reinterpret_cast<float4*>(part + (size_t)tid * pitch + j);
      o[0] = make_float4(f[0], f[1], f[2], f[3]);
      o[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
  // TMEM is given back before the peers are waited for: one of them may be waiting for TMEM itself,
  // beside another call's CTA that waits for a peer of its own
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, tcols);
  }
  __syncwarp();
  cluster_sync();
  // this rank's share of the rows: the four partials in rank order
  const float sc = g.scale[l];
  uint32_t peer[SPLIT];
#pragma unroll
  for (int q = 0; q < SPLIT; ++q) peer[q] = map_rank(sb, (uint32_t)q);
  for (int i = tid; ok && i < ROWS / SPLIT * (g.r / 2); i += THREADS) {
    const int r = rank * (ROWS / SPLIT) + i / (g.r / 2), j = (i % (g.r / 2)) * 2;
    if (r >= n) continue;
    const uint32_t at = (uint32_t)((r * pitch + j) * 4);
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
    uint32_t h[2];
    bf16x2_terms<2>(v0, v1, h);
    *reinterpret_cast<uint32_t*>(g.terms + o) = h[0];
    *reinterpret_cast<uint32_t*>(g.terms + (size_t)g.T * g.r + o) = h[1];
    if (g.planes != nullptr) {
      const size_t slot = (size_t)(first + r) * g.r + j, plane = (size_t)g.T * g.r;
      const float2 w = *reinterpret_cast<const float2*>(g.low2 + o);
      uint32_t hv[3], hw[3];
      bf16x2_terms<3>(v0, v1, hv);
      bf16x2_terms<3>(w.x, w.y, hw);
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        *reinterpret_cast<uint32_t*>(g.planes + p * plane + slot) = hv[p];
        *reinterpret_cast<uint32_t*>(g.planes2 + p * plane + slot) = hw[p];
      }
    }
  }
  __syncwarp();
  cluster_sync();  // no rank leaves while its partial may be read
}

template <bool TRANS>
moe_status run_low(LowArgs a, const void* m, cudaStream_t st) {
  auto kern = adapter_low_kernel<TRANS>;
  a.n_mma = (a.r + 15) / 16 * 16;
  a.nc = (a.r + 63) / 64;
  a.status = device_status_ptr();
  a.limit_ns = kWaitLimitNs;
  CUtensorMap mm;
  const uint64_t r = a.r, D = a.D, L = a.L;
  const uint64_t md[3] = {TRANS ? D : r, TRANS ? r : D, L}, ms[2] = {md[0] * 2, D * r * 2};
  const uint32_t mbox[3] = {64, 64, 1};
  if (!make_map(&mm, m, 3, md, ms, mbox)) return MOE_ERR_CUDA;
  int smem = STAGES * (X_BYTES + a.nc * M_CHUNK);
  if (smem < ROWS * (a.r + 4) * 4) smem = ROWS * (a.r + 4) * 4;  // the partial
  smem += 1024;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  // at most T / ROWS whole tiles and one ragged tile an adapter (or a row)
  const int ragged = a.L < a.T ? a.L : a.T;
  a.tile_clusters = a.T / ROWS + ragged;
  const int table = (a.T + SPLIT * kAdapterTileRows - 1) / (SPLIT * kAdapterTileRows);
  launch_begin(K_ADAPTER_LOW, st);
  launch_kernel(kern, dim3((unsigned)(SPLIT * (a.tile_clusters + table))), dim3(THREADS),
                (size_t)smem, st, SPLIT, mm, a);
  return launch_end(K_ADAPTER_LOW, st);
}

// ------------------------------------------------------------------ few rows
constexpr int FEW_THREADS = 128;

struct LowFewArgs {
  const bf16* x;
  const bf16* a;
  const int32_t* ids;
  float* part;  // [splits][T][r]
  int T, D, r, L, splits;
  unsigned* status;
};

// CTA (row t, split s): eight rank values a thread, the contraction over the threads.
__global__ void __launch_bounds__(FEW_THREADS) adapter_low_few_kernel(const LowFewArgs g) {
  __shared__ float xs[1024];
  __shared__ float red[FEW_THREADS * 8];
  const int tid = threadIdx.x, t = blockIdx.x, s = blockIdx.y;
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();
  const int l = g.ids[t];
  if (l < 0 || l >= g.L) {
    if (l != -1 && tid == 0 && s == 0) report(g.status, MOE_ERR_DEVICE_INDEX);
    return;  // nobody reads this row's partials
  }
  const int rc = g.r / 8, step = FEW_THREADS / rc;
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
    for (int i = tid * 8; i < nk; i += FEW_THREADS * 8) {
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
  for (int j = tid; j < g.r; j += FEW_THREADS) {
    float sum = 0.f;
    for (int q = 0; q < step; ++q) sum += red[q * g.r + j];
    g.part[((size_t)s * g.T + t) * g.r + j] = sum;
  }
}

}  // namespace

moe_status launch_adapter_low(bool trans, int T, int D, int r, int L, const void* in,
                              const void* m, const int32_t* ids, const int32_t* offsets,
                              const int32_t* rows, const float* scale, float* low, void* planes,
                              const float* low2, void* planes2, void* terms,
                              AdapterTiles tiles, cudaStream_t st) {
  LowArgs a = {};
  a.in = (const bf16*)in;
  a.ids = ids;
  a.offsets = offsets;
  a.rows = rows;
  a.scale = scale;
  a.low = low;
  a.planes = (bf16*)planes;
  a.low2 = low2;
  a.planes2 = (bf16*)planes2;
  a.terms = (bf16*)terms;
  a.tiles = tiles;
  a.T = T;
  a.D = D;
  a.r = r;
  a.L = L;
  return trans ? run_low<true>(a, m, st) : run_low<false>(a, m, st);
}

moe_status launch_adapter_low_few(int T, int D, int r, int L, int splits, const void* x,
                                  const void* a, const int32_t* ids, float* part,
                                  cudaStream_t st) {
  const LowFewArgs f{(const bf16*)x, (const bf16*)a, ids, part, T, D, r, L, splits,
                     device_status_ptr()};
  launch_begin(K_ADAPTER_LOW_FEW, st);
  launch_kernel(adapter_low_few_kernel, dim3((unsigned)T, (unsigned)splits), dim3(FEW_THREADS), 0, st,
                1, f);
  return launch_end(K_ADAPTER_LOW_FEW, st);
}

}  // namespace moe
