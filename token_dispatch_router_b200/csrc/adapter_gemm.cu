// The shared projection with per-row low-rank adapters for many rows:
//
//   forward:      y[t]   = x[t] W     + low[t] B[ids[t]]       W [d_in, d_out], B [L, r, d_out]
//   backward dX:  d_x[t] = d_y[t] W^T + d_low[t] A[ids[t]]^T   A [L, d_in, r]
//
// The large product runs on CTA pairs (tcgen05.mma.cta_group::2, 256 x 256 tiles, TMA-fed,
// accumulators double-buffered in TMEM); W is read as it lies, MN-major forward and K-major
// backward. Bound by the tensor pipe while a tile's rows have few adapters.
//
// The adapter term is a few more k-blocks of the same accumulation: after a tile's product, for
// each adapter that has rows in the tile, low (A operand) times the adapter's matrix (B operand),
// with the MMA's lane mask (disable-output-lane) keeping it out of the other rows. Rows of one
// tile may so belong to any adapters in any order, nothing is multiplied by zero (an infinity
// or NaN in one adapter stays in its own rows), and the epilogue only stores. low is fp32: it
// enters as two bf16 terms (bf16_terms, error 2^-16), far inside the rounding of the output. The
// adapters of each 256-row tile and their masks come from a table built with low. Every adapter of a
// tile costs a stage and its MMAs over all of the tile's rows, and the low of every four (two above
// rank 64) is loaded again: rows with an adapter each are bound by that (forward, 4096 -> 4096, rank
// 16, one adapter and one a row: 129 rows 31 and 157 us, 256 rows 39 and 286, 512 rows 46 and 287).
#include "adapter.cuh"
#include "ffn_args.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int BM = 128, PAIR_M = kAdapterTileRows, BK = 64, BN = kAdapterTileCols, STAGES = 6;
constexpr int A_BYTES = BM * BK * 2;
constexpr int B_CHUNK = BK * 64 * 2;
constexpr int B_HALF = 2 * B_CHUNK;
constexpr int STAGE_BYTES = A_BYTES + B_HALF;  // 32 KB a CTA
constexpr int THREADS = 192;                   // producer, MMA, 4 epilogue warps
constexpr uint32_t TMEM_COLS = 512;
constexpr int SMEM_TAIL = 512;
// All that a CTA can have: it holds all of TMEM while it waits for the kernel before it, so no
// CTA of another call that wants TMEM may come beside it.
constexpr int SMEM_BYTES = 227 * 1024;
static_assert(1024 + STAGES * STAGE_BYTES + SMEM_TAIL <= SMEM_BYTES, "ring and barriers");

struct AdapterGemmArgs {
  int T, n_out, kblocks, mt, nt, rank;
  int whole, split;          // tiles made whole; pairs that share the contraction of the others
  float* part;               // [others][split][2 CTAs][64][128 rows][4]
  AdapterTiles tiles;        // [mt]
  bf16* out;                 // [T, n_out]
  unsigned* status;
  unsigned long long limit_ns;
};

// D += A B in the rows whose bit in `off` is clear (rows 32 i ... of the pair in off[i]).
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, const uint32_t (&off)[8]) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.b32 p, %3, %3;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7, %8, %9, %10, %11}, "
      "p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]),
      "r"(off[4]), "r"(off[5]), "r"(off[6]), "r"(off[7])
      : "memory");
}

// Work item w: a whole tile, or split `s` of one of the tiles behind the whole ones.
struct Item {
  int tile, s, k0, k1;
  bool whole, adapters;  // the adapter term belongs to the last split
};
__device__ __forceinline__ Item item_of(int w, const AdapterGemmArgs& g) {
  if (w < g.whole) return Item{w, 0, 0, g.kblocks, true, true};
  const int v = w - g.whole, s = v % g.split;
  return Item{g.whole + v / g.split, s, s * g.kblocks / g.split, (s + 1) * g.kblocks / g.split,
              false, s == g.split - 1};
}

template <bool BWD>
__global__ void __launch_bounds__(THREADS, 1)
    adapter_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmLow,
                        const __grid_constant__ CUtensorMap tmM, const AdapterGemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = (uint64_t*)(base + STAGES * STAGE_BYTES);  // leader: both CTAs' bytes landed
  uint64_t* empty = full + STAGES;    // both: the MMAs reading the stage completed
  uint64_t* tfull = empty + STAGES;   // both: accumulator b complete
  uint64_t* tempty = tfull + 2;       // leader: both CTAs drained accumulator b
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = (uint32_t*)(done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* epi_flag = (volatile int*)(tmem_slot + 2);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = (int)cluster_id_x(), npairs = (int)num_clusters_x();
  const int total = g.whole + (g.mt * g.nt - g.whole) * g.split;
  const uint64_t limit = g.limit_ns;
  // Ring stages after a tile's k-blocks: for each group of its adapters, low (nl stages, both
  // terms) and then nl stages an adapter; low's stages are freed with the group, so a group and
  // its low fit the ring together.
  const int nl = (g.rank + 63) / 64, group = nl == 1 ? 4 : 2;

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(saddr(&full[s]), 1);
      mbar_init(saddr(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(saddr(&tfull[b]), 1);
      mbar_init(saddr(&tempty[b]), 8);  // 4 epilogue warps x 2 CTAs
    }
    mbar_init(saddr(done), 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<2>(saddr(tmem_slot), TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any cross-CTA arrival
  tc_fence_after();
  // low and the table of tiles come from the kernel before this one; x, d_y, W and the adapters
  // are older (that kernel lets this one start only once all before it is complete). So only the
  // adapter term waits for it (backward, 300 rows: 23.7 us with the wait here, 19.8
  // without).
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_par = 0;
      bool ok = true, waited = false;
      // the next stage, when it is free: its full barrier (the leader's) expecting `bytes` a CTA
      auto begin = [&](uint32_t bytes, uint32_t& fb, uint32_t& a) {
        if (!mbar_wait<true>(saddr(&empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) {
          ok = false;
          return false;
        }
        fb = map_rank(saddr(&full[stage]), 0);
        a = saddr(base + stage * STAGE_BYTES);
        if (leader) mbar_expect_tx(saddr(&full[stage]), 2 * bytes);
        issued_mask |= 1u << stage;
        issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        return true;
      };
      for (int w = pair; w < total && ok; w += npairs) {
        const Item it = item_of(w, g);
        int m, n;
        adapter_tile_of(it.tile, g.mt, g.nt, m, n);
        const int m0 = m * PAIR_M + (int)rank * BM, n0 = n * BN + (int)rank * 128;
        uint32_t fb, a;
        for (int kb = it.k0; kb < it.k1; ++kb) {
          if (!begin(STAGE_BYTES, fb, a)) break;
          const uint32_t b = a + A_BYTES;
          tma_load_2d_pair(a, &tmA, kb * BK, m0, fb);
          if (BWD) {
            tma_load_2d_pair(b, &tmB, kb * BK, n0, fb);
          } else {
            tma_load_2d_pair(b, &tmB, n0, kb * BK, fb);
            tma_load_2d_pair(b + B_CHUNK, &tmB, n0 + 64, kb * BK, fb);
          }
        }
        if (!waited) {
          pdl_wait();  // the previous kernel in the stream has completed
          pdl_trigger();
          waited = true;
        }
        const int n_ad = it.adapters ? *g.tiles.count(m) : 0;
        for (int i = 0; i < n_ad && ok; ++i) {
          if (i % group == 0)
            for (int j = 0; j < nl; ++j) {
              if (!begin(STAGE_BYTES, fb, a)) break;
              tma_load_3d_pair(a, &tmLow, 64 * j, m0, 0, fb);
              tma_load_3d_pair(a + A_BYTES, &tmLow, 64 * j, m0, 1, fb);
            }
          const int l = g.tiles.ids(m)[i];
          for (int j = 0; j < nl && ok; ++j) {
            if (!begin(B_HALF, fb, a)) break;
            const uint32_t b = a + A_BYTES;
            if (BWD) {
              tma_load_3d_pair(b, &tmM, 64 * j, n0, l, fb);
            } else {
              tma_load_3d_pair(b, &tmM, n0, 64 * j, l, fb);
              tma_load_3d_pair(b + B_CHUNK, &tmM, n0 + 64, 64 * j, l, fb);
            }
          }
        }
      }
      // the leader's barriers count both CTAs' bytes: no load is in flight after this (bounded);
      // the peer waits for it at the final cluster barrier
      if (leader)
        for (int s = 0; s < STAGES; ++s) {
          if (!(issued_mask & (1u << s))) continue;
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_cluster(saddr(&full[s]), (issued_par >> s) & 1u) &&
                 globaltimer_ns() - t0 < limit) {
          }
        }
    }
  } else if (warp == 1) {
    if (leader && lane == 0) {
      // ---------------------------------------------------------- MMA issuer (leader)
      const uint32_t idesc = idesc_bf16(PAIR_M, BN) & ~(BWD ? 1u << 16 : 0u);
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true, waited = false;
      // the next stage's index, once both CTAs' halves have landed; -1 when the wait ran out
      auto next = [&]() {
        if (!mbar_wait<true>(saddr(&full[stage]), phase, abort_flag, g.status, limit)) {
          ok = false;
          return -1;
        }
        tc_fence_after();
        const int s = stage;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        return s;
      };
      auto release = [&](int s) {
        tc_commit<2>(saddr(&empty[s]));
        tc_commit<2>(map_rank(saddr(&empty[s]), 1));
      };
      for (int w = pair; w < total && ok; w += npairs, ++it) {
        const Item wi = item_of(w, g);
        int m, n;
        adapter_tile_of(wi.tile, g.mt, g.nt, m, n);
        const int buf = it & 1;
        const uint32_t use = (uint32_t)(it >> 1);
        if (!mbar_wait<true>(saddr(&tempty[buf]), (use & 1u) ^ 1u, abort_flag, g.status, limit))
          break;
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(buf * BN);
        for (int kb = wi.k0; kb < wi.k1; ++kb) {
          const int s = next();
          if (s < 0) break;
          const uint32_t a = saddr(base + s * STAGE_BYTES), b = a + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            tc_mma<2>(d, desc_sw128(a + kk * 32, 16, 1024),
                      BWD ? desc_sw128(b + kk * 32, 16, 1024)
                          : desc_sw128(b + kk * 2048, B_CHUNK, 1024),
                      idesc, (kb > wi.k0 || kk > 0) ? 1u : 0u);
          release(s);
        }
        if (!waited) pdl_wait();  // the previous kernel in the stream has completed
        waited = true;
        const int n_ad = wi.adapters ? *g.tiles.count(m) : 0;
        int low[2] = {0, 0};
        for (int i = 0; i < n_ad && ok; ++i) {
          uint32_t off[8];
          {
            const uint4* mp = reinterpret_cast<const uint4*>(g.tiles.off(m, i));
            const uint4 u = mp[0], v = mp[1];
            off[0] = u.x; off[1] = u.y; off[2] = u.z; off[3] = u.w;
            off[4] = v.x; off[5] = v.y; off[6] = v.z; off[7] = v.w;
          }
          if (i % group == 0)
            for (int j = 0; j < nl && ok; ++j) low[j] = next();
          for (int j = 0; j < nl && ok; ++j) {
            const int s = next();
            if (s < 0) break;
            const uint32_t a = saddr(base + low[j] * STAGE_BYTES);
            const uint32_t b = saddr(base + s * STAGE_BYTES) + A_BYTES;
            const int steps = min(4, (g.rank - 64 * j + 15) / 16);
            for (int kk = 0; kk < steps; ++kk) {
              const uint64_t bd = BWD ? desc_sw128(b + kk * 32, 16, 1024)
                                      : desc_sw128(b + kk * 2048, B_CHUNK, 1024);
              mma_rows(d, desc_sw128(a + kk * 32, 16, 1024), bd, idesc, off);
              mma_rows(d, desc_sw128(a + A_BYTES + kk * 32, 16, 1024), bd, idesc, off);
            }
            release(s);
          }
          if (ok && (i % group == group - 1 || i == n_ad - 1))
            for (int j = 0; j < nl; ++j) release(low[j]);
        }
        if (ok) {
          tc_commit<2>(saddr(&tfull[buf]));
          tc_commit<2>(map_rank(saddr(&tfull[buf]), 1));
        }
      }
      tc_commit<2>(saddr(done));  // every MMA of the pair completed before TMEM is freed
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try(saddr(done), 0) && globaltimer_ns() - t0 < limit) {
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    // One thread waits for all four warps, so that they leave a wait that ran out together.
    const int q = warp & 3;  // TMEM lanes 32 q ...
    const bool first = tid == 64;
    const uint32_t tempty_leader = map_rank(saddr(&tempty[0]), 0);
    int it = 0;
    for (int w = pair; w < total; w += npairs, ++it) {
      const Item wi = item_of(w, g);
      int m, n;
      adapter_tile_of(wi.tile, g.mt, g.nt, m, n);
      const int buf = it & 1;
      const uint32_t use = (uint32_t)(it >> 1);
      if (first)
        *epi_flag = mbar_wait<true>(saddr(&tfull[buf]), use & 1u, abort_flag, g.status, limit);
      epi_bar();
      const int ok = *epi_flag;
      epi_bar();  // everyone has read it
      if (!ok) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + (uint32_t)(buf * BN) + ((uint32_t)(q * 32) << 16);
      const int lr = q * 32 + lane, r = m * PAIR_M + (int)rank * BM + lr;
      bf16* orow = g.out + (size_t)min(r, g.T - 1) * g.n_out;
      // a split's partial: [4 columns][row][4]
      float4* part = reinterpret_cast<float4*>(g.part) +
                     (wi.whole ? 0
                               : ((size_t)((wi.tile - g.whole) * g.split + wi.s) * 2 + rank) *
                                     (BN / 4) * BM) + lr;
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        const int col = n * BN + c * 32;
        if (col >= g.n_out) break;  // warp-uniform (n_out is a multiple of 64)
        uint32_t v[32];
        tmem_ld32(tb + c * 32, v);
        tmem_ld_wait();
        if (!wi.whole) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            part[(size_t)(c * 8 + j) * BM] =
                make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                            __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
        } else if (r < g.T) {
          uint4* dst = reinterpret_cast<uint4*>(orow + col);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            dst[j] = make_uint4(
                pack_bf16x2(__uint_as_float(v[8 * j]), __uint_as_float(v[8 * j + 1])),
                pack_bf16x2(__uint_as_float(v[8 * j + 2]), __uint_as_float(v[8 * j + 3])),
                pack_bf16x2(__uint_as_float(v[8 * j + 4]), __uint_as_float(v[8 * j + 5])),
                pack_bf16x2(__uint_as_float(v[8 * j + 6]), __uint_as_float(v[8 * j + 7])));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(tempty_leader + (uint32_t)(buf * 8));
    }
  }
  __syncwarp();  // lanes that waited alone are back: a barrier counts a split warp twice
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair is done with both TMEM allocations and all barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<2>(tmem_base, TMEM_COLS);
  }
}

template <bool BWD>
moe_status run(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& ml,
               const CUtensorMap& mm, const AdapterGemmArgs& a, cudaStream_t st) {
  auto kern = adapter_gemm_kernel<BWD>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  const int items = a.whole + (a.mt * a.nt - a.whole) * a.split;
  const int pairs = items < sm_count() / 2 ? items : sm_count() / 2;
  launch_begin(K_ADAPTER_GEMM, st);
  launch_kernel(kern, dim3((unsigned)(2 * pairs)), dim3(THREADS), (size_t)SMEM_BYTES, st, 2, ma,
                mb, ml, mm, a);
  return launch_end(K_ADAPTER_GEMM, st);
}

}  // namespace

// Tiles that do not fill the pairs of SMs once more are cut along the contraction, so that they
// take that part of a tile's time: at most eight splits of at least four k-blocks, whose fp32
// partials another kernel adds in order. (2880 x 2880, 2049 rows: 108 tiles on 74 pairs took two
// rounds.) Returns the number of partials.
int adapter_gemm_split(int T, int k_dim, int n_out, int* whole, int* split) {
  const int pairs = sm_count() > 1 ? sm_count() / 2 : 1;  // a host without a device counts one SM
  const int tiles = ((T + PAIR_M - 1) / PAIR_M) * ((n_out + BN - 1) / BN);
  const int rest = tiles % pairs;
  int s = rest > 0 ? pairs / rest : 1;
  if (s > k_dim / BK / 4) s = k_dim / BK / 4;
  if (s > 8) s = 8;
  // the second kernel takes about 4 us, a k-block 0.29 (300 rows, 768 -> 2048: 27 us whole, 30 cut)
  if (s < 2 || (k_dim / BK) * (s - 1) < 20 * s) {
    *whole = tiles;
    *split = 1;
    return 0;
  }
  *whole = tiles - rest;
  *split = s;
  return rest * s;
}
size_t adapter_gemm_part_bytes(int T, int k_dim, int n_out) {
  int whole, split;
  return (size_t)adapter_gemm_split(T, k_dim, n_out, &whole, &split) * PAIR_M * BN * 4;
}

// in [T, k_dim], w [d_in, d_out]; forward: k_dim = d_in, out [T, d_out], m = B; backward:
// k_dim = d_out, out [T, d_in], m = A. low: [2][T][rank] bf16 terms.
moe_status launch_adapter_gemm(bool bwd, int T, int d_in, int d_out, int n_adapters, int rank,
                               const void* in, const void* w, AdapterTiles tiles,
                               const void* low, const void* m, void* out, float* part,
                               cudaStream_t st) {
  const int k_dim = bwd ? d_out : d_in, n_out = bwd ? d_in : d_out;
  AdapterGemmArgs a = {};
  a.T = T;
  a.n_out = n_out;
  a.kblocks = k_dim / BK;
  a.mt = (T + PAIR_M - 1) / PAIR_M;
  a.nt = (n_out + BN - 1) / BN;
  adapter_gemm_split(T, k_dim, n_out, &a.whole, &a.split);
  a.part = part;
  a.out = (bf16*)out;
  a.rank = rank;
  a.tiles = tiles;
  a.status = device_status_ptr();
  a.limit_ns = kWaitLimitNs;
  CUtensorMap ma, mb, ml, mm;
  const uint64_t r = rank, t = T, n = n_out, L = n_adapters;
  const uint64_t ad[2] = {(uint64_t)k_dim, t}, as[1] = {(uint64_t)k_dim * 2};
  const uint32_t abox[2] = {64, 128};
  const uint64_t bd[2] = {(uint64_t)d_out, (uint64_t)d_in}, bs[1] = {(uint64_t)d_out * 2};
  const uint32_t bbox[2] = {64, bwd ? 128u : 64u};
  const uint64_t ld[3] = {r, t, 2}, ls[2] = {r * 2, t * r * 2};
  const uint32_t lbox[3] = {64, 128, 1};
  const uint64_t md[3] = {bwd ? r : n, bwd ? n : r, L}, ms[2] = {(bwd ? r : n) * 2, r * n * 2};
  const uint32_t mbox[3] = {64, bwd ? 128u : 64u, 1};
  if (!make_map(&ma, in, 2, ad, as, abox) || !make_map(&mb, w, 2, bd, bs, bbox) ||
      !make_map(&ml, low, 3, ld, ls, lbox) || !make_map(&mm, m, 3, md, ms, mbox))
    return MOE_ERR_CUDA;
  return bwd ? run<true>(ma, mb, ml, mm, a, st) : run<false>(ma, mb, ml, mm, a, st);
}

// What launch_adapter_gemm leaves to add.
AdapterTileSums adapter_gemm_sums(int T, int k_dim, int n_out, void* out, const float* part) {
  AdapterTileSums s = {};
  s.T = T;
  s.n_out = n_out;
  s.mt = (T + PAIR_M - 1) / PAIR_M;
  s.nt = (n_out + BN - 1) / BN;
  adapter_gemm_split(T, k_dim, n_out, &s.whole, &s.split);
  s.others = s.mt * s.nt - s.whole;
  s.part = part;
  s.out = (bf16*)out;
  return s;
}

}  // namespace moe
