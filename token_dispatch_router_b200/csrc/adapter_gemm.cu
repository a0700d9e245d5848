// The shared projection with per-row low-rank adapters for many rows:
//
//   forward:      y[t]   = x[t] W     + low[t] B[ids[t]]       W [d_in, d_out], B [L, r, d_out]
//   backward dX:  d_x[t] = d_y[t] W^T + d_low[t] A[ids[t]]^T   A [L, d_in, r]
//
// The large product runs on CTA pairs (tcgen05.mma.cta_group::2, 256 x 256 tiles, TMA-fed,
// accumulators double-buffered in TMEM); W is read as it lies, MN-major forward and K-major
// backward. Bound by the tensor pipe.
//
// The adapter term is added in the epilogue, while the next tile's product runs, so it costs no
// pass over y and no extra k-blocks of the large product: the accumulator is read from TMEM in
// the layout of the warp-level MMA's accumulators (16x256b), the rank-r product of the warp's
// 32 rows and 32 columns is made with that MMA, and added. Rows of one warp may belong to
// several adapters: each one's product is made in registers of its own and selected by row,
// never multiplied by zero, so an infinity or NaN in one adapter stays in its own rows. low is
// fp32: it enters as two bf16 terms (error 2^-17), far inside the rounding of the output.
#include "adapter.cuh"
#include "ffn_args.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int BM = 128, PAIR_M = 256, BK = 64, BN = 256, STAGES = 6;
constexpr int A_BYTES = BM * BK * 2;
constexpr int B_CHUNK = BK * 64 * 2;
constexpr int B_HALF = 2 * B_CHUNK;
constexpr int STAGE_BYTES = A_BYTES + B_HALF;  // 32 KB a CTA
constexpr int THREADS = 192;                   // producer, MMA, 4 epilogue warps
constexpr uint32_t TMEM_COLS = 512;
constexpr int EPI_ROW = 80;  // 32 bf16 of a row, padded: rows hit distinct banks
constexpr int EPI_WARP = 32 * EPI_ROW;
constexpr int SMEM_TAIL = 512;
constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + SMEM_TAIL + 4 * EPI_WARP;
constexpr int GROUP_M = 8;  // row tiles that share the W panels of a wave through L2

struct AdapterGemmArgs {
  int T, n_out, kblocks, mt, nt, n_adapters, rank;
  const int32_t* ids;  // [T]
  const float* low;    // [T, rank]
  const bf16* w2;      // B [L, rank, n_out] forward, A [L, n_out, rank] backward
  bf16* out;           // [T, n_out]
  unsigned* status;
  unsigned long long limit_ns;
};

// Tile w: GROUP_M row tiles at a time, all column tiles of the group.
__device__ __forceinline__ void tile_of(int w, int mt, int nt, int& m, int& n) {
  const int per = GROUP_M * nt, grp = w / per, r = w % per;
  const int gm = min(GROUP_M, mt - grp * GROUP_M);
  m = grp * GROUP_M + r % gm;
  n = r / gm;
}

// Two 16 x 32 halves (TMEM lanes +0 and +16) in the accumulator layout of mma16816: half h,
// 8-column block i: v[h][i][0..1] at row lane / 4, columns 2 (lane % 4) + 0..1; [2..3] 8 rows on.
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, float (&v)[4][4]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i][j] = __uint_as_float(r[4 * i + j]);
}

// Element pair (k, k + 1) of column `col` of the adapter's second matrix as packed bf16.
template <bool BWD>
__device__ __forceinline__ uint32_t w2_pair(const bf16* w2, int n_out, int rank, int k, int col) {
  if (BWD) return *reinterpret_cast<const uint32_t*>(w2 + (size_t)col * rank + k);
  const uint16_t* p = reinterpret_cast<const uint16_t*>(w2) + (size_t)k * n_out + col;
  return (uint32_t)p[0] | ((uint32_t)p[n_out] << 16);
}

template <bool BWD>
__global__ void __launch_bounds__(THREADS, 1)
    adapter_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB, const AdapterGemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = (uint64_t*)(base + STAGES * STAGE_BYTES);  // leader: both CTAs' bytes landed
  uint64_t* empty = full + STAGES;    // both: the MMAs reading the stage completed
  uint64_t* tfull = empty + STAGES;   // both: accumulator b complete
  uint64_t* tempty = tfull + 2;       // leader: both CTAs drained accumulator b
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = (uint32_t*)(done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  uint8_t* epi = base + STAGES * STAGE_BYTES + SMEM_TAIL;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = (int)cluster_id_x(), npairs = (int)num_clusters_x();
  const int total = g.mt * g.nt;
  const uint64_t limit = g.limit_ns;

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
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_par = 0;
      bool ok = true;
      for (int w = pair; w < total && ok; w += npairs) {
        int m, n;
        tile_of(w, g.mt, g.nt, m, n);
        const int m0 = m * PAIR_M + (int)rank * BM, n0 = n * BN + (int)rank * 128;
        for (int kb = 0; kb < g.kblocks; ++kb) {
          if (!mbar_wait<true>(saddr(&empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) {
            ok = false;
            break;
          }
          const uint32_t fb = map_rank(saddr(&full[stage]), 0);  // the leader's barrier
          if (leader) mbar_expect_tx(saddr(&full[stage]), 2 * STAGE_BYTES);
          const uint32_t a = saddr(base + stage * STAGE_BYTES), b = a + A_BYTES;
          tma_load_2d_pair(a, &tmA, kb * BK, m0, fb);
          if (BWD) {
            tma_load_2d_pair(b, &tmB, kb * BK, n0, fb);
          } else {
            tma_load_2d_pair(b, &tmB, n0, kb * BK, fb);
            tma_load_2d_pair(b + B_CHUNK, &tmB, n0 + 64, kb * BK, fb);
          }
          issued_mask |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
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
      bool ok = true;
      for (int w = pair; w < total && ok; w += npairs, ++it) {
        const int buf = it & 1;
        const uint32_t use = (uint32_t)(it >> 1);
        if (!mbar_wait<true>(saddr(&tempty[buf]), (use & 1u) ^ 1u, abort_flag, g.status, limit))
          break;
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(buf * BN);
        for (int kb = 0; kb < g.kblocks; ++kb) {
          if (!mbar_wait<true>(saddr(&full[stage]), phase, abort_flag, g.status, limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = saddr(base + stage * STAGE_BYTES), b = a + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            tc_mma<2>(d, desc_sw128(a + kk * 32, 16, 1024),
                      BWD ? desc_sw128(b + kk * 32, 16, 1024)
                          : desc_sw128(b + kk * 2048, B_CHUNK, 1024),
                      idesc, (kb | kk) != 0 ? 1u : 0u);
          tc_commit<2>(saddr(&empty[stage]));
          tc_commit<2>(map_rank(saddr(&empty[stage]), 1));
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
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
    const int q = warp & 3;  // TMEM lanes 32 q ...
    const uint32_t tempty_leader = map_rank(saddr(&tempty[0]), 0);
    uint8_t* ebuf = epi + q * EPI_WARP;
    const int lr = lane >> 2, lc = lane & 3;
    int it = 0;
    for (int w = pair; w < total; w += npairs, ++it) {
      int m, n;
      tile_of(w, g.mt, g.nt, m, n);
      const int buf = it & 1;
      const uint32_t use = (uint32_t)(it >> 1);
      const int row0 = m * PAIR_M + (int)rank * BM + q * 32;
      // this lane's four rows (lr + 8 i) and their adapters
      int id[4];
      const float* lrow[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = row0 + lr + 8 * i;
        int l = r < g.T ? g.ids[r] : -1;
        if (l < 0 || l >= g.n_adapters) l = -1;  // the grouping kernel has reported bad ids
        id[i] = l;
        lrow[i] = g.low + (size_t)min(r, g.T - 1) * g.rank;
      }
      int w_ok = 0;
      if (lane == 0)
        w_ok = mbar_wait<true>(saddr(&tfull[buf]), use & 1u, abort_flag, g.status, limit);
      w_ok = __shfl_sync(0xffffffffu, w_ok, 0);
      if (!w_ok) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + (uint32_t)(buf * BN) + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        const int col0 = n * BN + c * 32;
        if (col0 >= g.n_out) break;  // warp-uniform (n_out is a multiple of 64)
        float acc[2][4][4];
        tmem_ld_16x256(tb + c * 32, acc[0]);
        tmem_ld_16x256(tb + c * 32 + (16u << 16), acc[1]);
        int last = -1;
        while (true) {  // the warp's adapters, in ascending order
          int nx = 0x7fffffff;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (id[i] > last) nx = min(nx, id[i]);
          nx = __reduce_min_sync(0xffffffffu, nx);
          if (nx == 0x7fffffff) break;
          last = nx;
          const bf16* w2 = g.w2 + (size_t)nx * g.rank * g.n_out;
          float dl[2][4][4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) dl[h][i][j] = 0.f;
          for (int k0 = 0; k0 < g.rank; k0 += 16) {
            const bool second = k0 + 8 < g.rank;  // rank is a multiple of 8
            uint32_t b0[4], b1[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int col = col0 + 8 * i + lr;
              b0[i] = w2_pair<BWD>(w2, g.n_out, g.rank, k0 + 2 * lc, col);
              b1[i] = second ? w2_pair<BWD>(w2, g.n_out, g.rank, k0 + 8 + 2 * lc, col) : 0u;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int p = 0; p < 4; ++p) {  // (rows lr, lr + 8) x (k, k + 8)
                float2 f = make_float2(0.f, 0.f);
                if (p < 2 || second)
                  f = *reinterpret_cast<const float2*>(lrow[2 * h + (p & 1)] + k0 + 8 * (p >> 1) +
                                                       2 * lc);
                hi[p] = take_bf16x2(f.x, f.y);
                lo[p] = pack_bf16x2(f.x, f.y);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                mma16816(dl[h][i], hi, b0[i], b1[i]);
                mma16816(dl[h][i], lo, b0[i], b1[i]);
              }
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (id[2 * h + (j >> 1)] == nx) acc[h][i][j] += dl[h][i][j];
        }
        // through the warp's buffer: 16-byte stores of whole 64-byte row pieces
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              *reinterpret_cast<uint32_t*>(ebuf + (16 * h + 8 * j + lr) * EPI_ROW + i * 16 +
                                           lc * 4) =
                  pack_bf16x2(acc[h][i][2 * j], acc[h][i][2 * j + 1]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = row0 + lr + 8 * i;
          if (r < g.T)
            *reinterpret_cast<uint4*>(g.out + (size_t)r * g.n_out + col0 + lc * 8) =
                *reinterpret_cast<const uint4*>(ebuf + (lr + 8 * i) * EPI_ROW + lc * 16);
        }
        __syncwarp();  // the buffer is free for the next columns
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(tempty_leader + (uint32_t)(buf * 8));
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair is done with both TMEM allocations and all barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<2>(tmem_base, TMEM_COLS);
  }
}

template <bool BWD>
moe_status run(const CUtensorMap& ma, const CUtensorMap& mb, const AdapterGemmArgs& a,
               cudaStream_t st) {
  auto kern = adapter_gemm_kernel<BWD>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  int pairs = sm_count() / 2;
  if (pairs > a.mt * a.nt) pairs = a.mt * a.nt;
  launch_begin(K_ADAPTER_GEMM, st);
  launch_kernel(kern, dim3((unsigned)(2 * pairs)), dim3(THREADS), (size_t)SMEM_BYTES, st, 2, ma,
                mb, a);
  return launch_end(K_ADAPTER_GEMM, st);
}

}  // namespace

// in [T, k_dim], w [d_in, d_out]; forward: k_dim = d_in, out [T, d_out], w2 = B; backward:
// k_dim = d_out, out [T, d_in], w2 = A.
moe_status launch_adapter_gemm(bool bwd, int T, int d_in, int d_out, int n_adapters, int rank,
                               const void* in, const void* w, const int32_t* ids,
                               const float* low, const void* w2, void* out, cudaStream_t st) {
  AdapterGemmArgs a = {};
  const int k_dim = bwd ? d_out : d_in, n_out = bwd ? d_in : d_out;
  a.T = T;
  a.n_out = n_out;
  a.kblocks = k_dim / BK;
  a.mt = (T + PAIR_M - 1) / PAIR_M;
  a.nt = (n_out + BN - 1) / BN;
  a.n_adapters = n_adapters;
  a.rank = rank;
  a.ids = ids;
  a.low = low;
  a.w2 = (const bf16*)w2;
  a.out = (bf16*)out;
  a.status = device_status_ptr();
  a.limit_ns = kWaitLimitNs;
  CUtensorMap ma, mb;
  const uint64_t ad[2] = {(uint64_t)k_dim, (uint64_t)T}, as[1] = {(uint64_t)k_dim * 2};
  const uint32_t abox[2] = {64, 128};
  const uint64_t bd[2] = {(uint64_t)d_out, (uint64_t)d_in}, bs[1] = {(uint64_t)d_out * 2};
  const uint32_t bbox[2] = {64, bwd ? 128u : 64u};
  if (!make_map(&ma, in, 2, ad, as, abox) || !make_map(&mb, w, 2, bd, bs, bbox))
    return MOE_ERR_CUDA;
  return bwd ? run<true>(ma, mb, a, st) : run<false>(ma, mb, a, st);
}

}  // namespace moe
