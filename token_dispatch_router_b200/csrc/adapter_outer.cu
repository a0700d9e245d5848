// Gradients of the adapter matrices: for each adapter l, over its rows t,
//
//   dA_l [d_in, r] = sum_t x[t]^T d_low[t],    dB_l [r, d_out] = sum_t low[t]^T d_y[t]
//
// Bound by reading the wide rows of x and d_y once. Rows come in any order, so they are
// gathered by cp.async into the swizzled layout that the tensor cores read; both operands are
// taken as they lie (a row is one k of the product: MN-major), so nothing is transposed. M is
// the wide side (256 columns a unit, two accumulators), N the rank (16 ... 128), K the rows.
// The low-rank side is fp32: it enters as three bf16 terms, exact to 2^-24; the tensor pipe has
// the time (three MMAs of N = r for each 32 x 256 tile of wide rows). The tensor core cuts what
// it adds to an accumulator off rather than rounding it, an error that grows with the number of
// additions: the small second and third terms have an accumulator of their own, added to the
// first's at the end (512 rows, relative to the gradient: 1.7e-6 in one accumulator, 0.5e-6 in two).
//
// A unit is (adapter, chunk of its rows, 256 columns of x or of d_y). Two CTAs an SM run through
// the units; up to rank 32 TMEM holds the accumulators of two units for each, so that the
// products of the next run beside the stores of the last (many adapters have only a few rows). Chunks of one adapter leave partial sums that a
// second kernel adds in chunk order (results repeat bit for bit); it is launched only where an
// adapter can have two chunks. An adapter without rows has one empty chunk, which writes zeros.
// Every wait is bounded (MOE_ERR_TIMEOUT on expiry).
#include "adapter.cuh"
#include "ffn_args.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int LOADERS = 128, THREADS = 320;  // four gather warps, MMA, TMA, four store warps
constexpr int OC = 256;                      // columns of a unit
constexpr int OT = 32;                       // rows per stage
constexpr int STAGES = 3;
constexpr int CHUNK = OT * 128;              // OT rows x 64 columns
constexpr int BIG_BYTES = OC / 64 * CHUNK;   // 16 KB
constexpr int kMaxAdapters = 256;

struct OuterArgs {
  const bf16* big[2];     // x [T, D0], d_y [T, D1]
  const bf16* planes[2];  // d_low, low: [3][T][r] in slot order
  float* out[2];          // dA [L, D0, r], dB [L, r, D1]
  int D[2], tiles[2];     // widths and their 256-column tiles
  const int32_t* offsets;
  const int32_t* rows;
  float* part;        // [chunk][(D0 + D1) r]: adapters of several chunks
  int T, r, L, chunk;
  int n_mma;          // the rank rounded up to 16
  int nc;             // its 64-column pieces
  int bufs;           // units whose accumulators TMEM holds: 1 or 2
  unsigned* status;
  unsigned long long limit_ns;
};

struct Table {
  int chunk0[kMaxAdapters + 1];  // first chunk of each adapter
  int multi0[kMaxAdapters];      // its first place among the chunks that leave partials
};
struct Unit {
  int l, p, c0, lo, n, slot;  // adapter, side, first column, first slot, rows; partial (-1: whole)
};

__device__ __forceinline__ void make_table(Table& t, const OuterArgs& g) {  // one warp
  const int lane = threadIdx.x & 31;
  int run = 0, mrun = 0;
  for (int l0 = 0; l0 < g.L; l0 += 32) {
    const int l = l0 + lane;
    const int c = l < g.L ? g.offsets[l + 1] - g.offsets[l] : 0;
    const int n = l < g.L ? max(1, (c + g.chunk - 1) / g.chunk) : 0, m = n > 1 ? n : 0;
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
    if (l < g.L) {
      t.chunk0[l] = run + incl - n;
      t.multi0[l] = mrun + mincl - m;
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
    mrun += __shfl_sync(0xffffffffu, mincl, 31);
  }
  if (lane == 0) t.chunk0[g.L] = run;
}
__device__ __forceinline__ Unit unit_of(int u, const Table& t, const OuterArgs& g) {
  const int nct = g.tiles[0] + g.tiles[1], cg = u / nct, ct = u % nct;
  int lo = 0, hi = g.L - 1;  // the last adapter whose chunks begin at cg or before
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.chunk0[mid] <= cg) lo = mid;
    else hi = mid - 1;
  }
  Unit v;
  v.l = lo;
  const int i = cg - t.chunk0[lo], first = g.offsets[lo] + i * g.chunk;
  v.p = ct >= g.tiles[0] ? 1 : 0;
  v.c0 = (ct - (v.p ? g.tiles[0] : 0)) * OC;
  v.lo = first;
  v.n = max(0, min(g.chunk, g.offsets[lo + 1] - first));
  v.slot = t.chunk0[lo + 1] - t.chunk0[lo] > 1 ? t.multi0[lo] + i : -1;
  return v;
}

__global__ void __launch_bounds__(THREADS)
    adapter_outer_kernel(const __grid_constant__ CUtensorMap tmP0,
                         const __grid_constant__ CUtensorMap tmP1, const OuterArgs g) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ Table table;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sb = (saddr(smem_raw) + 1023u) & ~1023u;
  const int p_bytes = g.nc * CHUNK, st_bytes = BIG_BYTES + 3 * p_bytes;
  volatile int* abort_flag = &s_abort;
  const uint32_t tcols = tmem_columns(g.bufs * 4 * g.n_mma);

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(saddr(&full[s]), LOADERS + 1);
      mbar_init(saddr(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(saddr(&tfull[b]), 1);
      mbar_init(saddr(&tempty[b]), 4);  // the store warps
    }
    mbar_init(saddr(&done), 1);
    s_abort = 0;
    mbar_init_fence();
  }
  if (warp == 4) tmem_alloc<1>(saddr(&s_tmem), tcols);
  if (tid == 32) {
    prefetch_map(&tmP0);
    prefetch_map(&tmP1);
  }
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();
  if (warp == 0) make_table(table, g);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const uint64_t limit = g.limit_ns;
  const int units = table.chunk0[g.L] * (g.tiles[0] + g.tiles[1]), step = (int)gridDim.x;

  if (warp < 4) {
    // ------------------------------------------------------------ gather
    // wide rows: warp w copies rows w, w + 4, ..., 512 bytes (one 16-byte piece a lane) each
    const int chunk_at = (lane >> 3) * CHUNK, pieces = g.n_mma / 8;
    const size_t plane = (size_t)g.T * g.r;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += step) {
      const Unit v = unit_of(u, table, g);
      const int steps = (v.n + OT - 1) / OT, D = g.D[v.p];
      const bf16* big = g.big[v.p] + v.c0 + lane * 8;
      const bool col_on = v.c0 + lane * 8 < D;
      // lane i < 8 holds the row of this warp's i-th row in the next stage
      auto row_of = [&](int s) {
        const int r = s * OT + warp + 4 * (lane & 7);
        return r < v.n ? g.rows[v.lo + r] : -1;
      };
      int ahead = steps > 0 ? row_of(0) : -1;
      for (int s = 0; s < steps; ++s) {
        const int mine = ahead;
        if (s + 1 < steps) ahead = row_of(s + 1);
        if (!mbar_wait_warp(saddr(&empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) {
          ok = false;
          break;
        }
        const uint32_t bs = sb + stage * st_bytes, ps = bs + BIG_BYTES;
#pragma unroll
        for (int i = 0; i < OT / 4; ++i) {
          const int t = __shfl_sync(0xffffffffu, mine, i), r = warp + 4 * i;
          const bool on = t >= 0 && col_on;
          cp_async16_if(bs + chunk_at + r * 128 + (((lane & 7) ^ (r & 7)) << 4),
                        on ? big + (size_t)t * D : g.big[v.p], on);
        }
        if ((s + 1) * OT > v.n)  // the last rows: the slots behind them are another adapter's
          for (int i = tid; i < 3 * OT * pieces; i += LOADERS) {
            const int q = i / (OT * pieces), r = i / pieces % OT, c = i % pieces;
            const bool on = s * OT + r < v.n && c * 8 < g.r;
            cp_async16_if(
                ps + q * p_bytes + (c >> 3) * CHUNK + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                g.planes[v.p] + (on ? q * plane + (size_t)(v.lo + s * OT + r) * g.r + c * 8 : 0),
                on);
          }
        cp_async_arrive_noinc(saddr(&full[stage]));
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    cp_async_wait_all();
  } else if (warp == 5) {
    // ------------------------------------------------------------ low-rank terms (TMA)
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_par = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += step) {
      const Unit v = unit_of(u, table, g);
      const int steps = (v.n + OT - 1) / OT;
      for (int s = 0; s < steps; ++s) {
        if (!mbar_wait_warp(saddr(&empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t fb = saddr(&full[stage]), ps = sb + stage * st_bytes + BIG_BYTES;
          if ((s + 1) * OT <= v.n) {
            mbar_expect_tx(fb, (uint32_t)(3 * p_bytes));
            for (int q = 0; q < 3; ++q)
              for (int c = 0; c < g.nc; ++c)
                tma_load_3d(ps + q * p_bytes + c * CHUNK, v.p ? &tmP1 : &tmP0, 64 * c,
                            v.lo + s * OT, q, fb);
          } else {
            mbar_arrive(fb);  // the gather warps copy these
          }
        }
        __syncwarp();
        issued_mask |= 1u << stage;
        issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (lane == 0)
      for (int s = 0; s < STAGES; ++s) {  // nothing of ours is in flight after this (bounded)
        if (!(issued_mask & (1u << s))) continue;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try(saddr(&full[s]), (issued_par >> s) & 1u) &&
               globaltimer_ns() - t0 < limit) {
        }
      }
  } else if (warp == 4) {
    // ------------------------------------------------------------ MMA issuer
    // D fp32, A and B bf16, both MN-major (bits 15 and 16), M = 128, N = n_mma
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                           ((uint32_t)(g.n_mma >> 3) << 17) | (8u << 24);
    const uint64_t bd0 = desc_sw128(sb, CHUNK, 1024), pd0 = desc_sw128(sb + BIG_BYTES, CHUNK, 1024);
    int stage = 0, it = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += step, ++it) {
      const Unit v = unit_of(u, table, g);
      const int steps = (v.n + OT - 1) / OT, buf = it & (g.bufs - 1);
      if (!mbar_wait_warp(saddr(&tempty[buf]), ((uint32_t)(it >> (g.bufs - 1)) & 1u) ^ 1u,
                          abort_flag, g.status, limit))
        break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(buf * 4 * g.n_mma);
      for (int s = 0; s < steps; ++s) {
        if (!mbar_wait_warp(saddr(&full[stage]), phase, abort_flag, g.status, limit)) {
          ok = false;
          break;
        }
        fence_proxy_async_smem();  // the gathered rows (cp.async) -> MMA reads
        tc_fence_after();
        if (elect_one()) {
          const uint64_t so = (uint64_t)((stage * st_bytes) >> 4);
#pragma unroll
          for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int kk = 0; kk < OT / 16; ++kk)
#pragma unroll
              for (int m = 0; m < 2; ++m)
                tc_mma<1>(acc + (uint32_t)(((q > 0 ? 2 : 0) + m) * g.n_mma),
                          bd0 + so + (uint64_t)((m * 2 * CHUNK + kk * 2048) >> 4),
                          pd0 + so + (uint64_t)((q * p_bytes + kk * 2048) >> 4), idesc,
                          (s > 0 || q > 1 || kk > 0) ? 1u : 0u);
          tc_commit<1>(saddr(&empty[stage]));
        }
        __syncwarp();
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok && elect_one()) tc_commit<1>(saddr(&tfull[buf]));
      __syncwarp();
    }
    if (elect_one()) tc_commit<1>(saddr(&done));
    __syncwarp();
    if (lane == 0) {  // every MMA has completed before TMEM is freed (bounded)
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try(saddr(&done), 0) && globaltimer_ns() - t0 < limit) {
      }
    }
  } else {
    // ------------------------------------------------------------ store
    const int q = warp & 3;  // TMEM lanes 32 q ...: columns of x or d_y
    const size_t wide = (size_t)(g.D[0] + g.D[1]) * g.r;
    int it = 0;
    for (int u = blockIdx.x; u < units; u += step, ++it) {
      const Unit v = unit_of(u, table, g);
      const int buf = it & (g.bufs - 1), D = g.D[v.p];
      float* dst = v.slot < 0 ? g.out[v.p] + (size_t)v.l * D * g.r
                              : g.part + (size_t)v.slot * wide + (v.p ? (size_t)g.D[0] * g.r : 0);
      if (!mbar_wait_warp(saddr(&tfull[buf]), (uint32_t)(it >> (g.bufs - 1)) & 1u, abort_flag,
                          g.status, limit))
        break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(buf * 4 * g.n_mma) + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
      for (int m = 0; m < 2; ++m) {
        const int c = v.c0 + m * 128 + q * 32 + lane;
#pragma unroll 2
        for (int j0 = 0; j0 < g.r; j0 += 8) {
          uint32_t f[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}, f2[8];
          if (v.n > 0) {  // else no rows: zeros
            tmem_ld8(acc + (uint32_t)(m * g.n_mma + j0), f);
            tmem_ld8(acc + (uint32_t)((2 + m) * g.n_mma + j0), f2);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              f[j] = __float_as_uint(__uint_as_float(f[j]) + __uint_as_float(f2[j]));
          }
          if (c >= D) continue;
          if (v.p == 0) {
            uint4* o = reinterpret_cast<uint4*>(dst + (size_t)c * g.r + j0);
            o[0] = make_uint4(f[0], f[1], f[2], f[3]);
            o[1] = make_uint4(f[4], f[5], f[6], f[7]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) dst[(size_t)(j0 + j) * D + c] = __uint_as_float(f[j]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(saddr(&tempty[buf]));
    }
  }
  __syncwarp();  // lanes that waited alone are back
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, tcols);
  }
}

// dA and dB of the adapters with several chunks: their partial sums in chunk order. CTA (piece,
// adapter): 4096 of the adapter's (D0 + D1) r values.
constexpr int SUM_THREADS = 256, SUM_PIECE = 4 * 4 * SUM_THREADS;
__global__ void __launch_bounds__(SUM_THREADS) adapter_outer_sum_kernel(const OuterArgs g) {
  __shared__ int s_before[SUM_THREADS / 32];
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();
  const int tid = threadIdx.x, l = blockIdx.y;
  auto chunks = [&](int a) {
    const int n = (g.offsets[a + 1] - g.offsets[a] + g.chunk - 1) / g.chunk;
    return n > 1 ? n : 0;
  };
  const int n = chunks(l);
  if (n == 0) return;
  int before = tid < l ? chunks(tid) : 0;  // L <= 256
  before = __reduce_add_sync(0xffffffffu, before);
  if ((tid & 31) == 0) s_before[tid >> 5] = before;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int i = 0; i < SUM_THREADS / 32; ++i) base += s_before[i];
  const size_t na = (size_t)g.D[0] * g.r, wide = na + (size_t)g.D[1] * g.r;
  const float* p0 = g.part + (size_t)base * wide;
  float4 v[4];
  size_t at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    at[i] = (size_t)blockIdx.x * SUM_PIECE + (size_t)(i * SUM_THREADS + tid) * 4;
    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll 2
  for (int q = 0; q < n; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at[i] < wide) {
        const float4 u = *reinterpret_cast<const float4*>(p0 + (size_t)q * wide + at[i]);
        v[i].x += u.x; v[i].y += u.y; v[i].z += u.z; v[i].w += u.w;
      }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (at[i] < wide)  // D0 r is a multiple of four: a vector lies in one of the two
      *reinterpret_cast<float4*>(at[i] < na
                                     ? g.out[0] + (size_t)l * na + at[i]
                                     : g.out[1] + (size_t)l * (wide - na) + (at[i] - na)) = v[i];
}

int tiles_of(int d) { return (d + OC - 1) / OC; }

// Rows of a unit: enough units for four a SM, at least 512 rows each.
int chunk_of(int T, int d_in, int d_out) {
  long long c = (long long)T * (tiles_of(d_in) + tiles_of(d_out)) / (4 * 148);
  c = (c + 63) / 64 * 64;
  return (int)(c < 512 ? 512 : c);
}

}  // namespace

// Partial sums of adapters with more than one chunk: at most 2 T / chunk chunks.
size_t adapter_outer_part_bytes(int T, int d_in, int d_out, int r) {
  const size_t chunks = 2 * (size_t)(T / chunk_of(T, d_in, d_out));
  return chunks * (size_t)(d_in + d_out) * r * 4;
}

moe_status launch_adapter_outer(int T, int d_in, int d_out, int r, int L, const void* x,
                                const void* d_y, const void* planes_d_low,
                                const void* planes_low, const int32_t* offsets,
                                const int32_t* rows, float* d_a, float* d_b, float* part,
                                cudaStream_t st) {
  OuterArgs a = {};
  a.big[0] = (const bf16*)x;
  a.big[1] = (const bf16*)d_y;
  a.planes[0] = (const bf16*)planes_d_low;
  a.planes[1] = (const bf16*)planes_low;
  a.out[0] = d_a;
  a.out[1] = d_b;
  a.D[0] = d_in;
  a.D[1] = d_out;
  a.tiles[0] = tiles_of(d_in);
  a.tiles[1] = tiles_of(d_out);
  a.offsets = offsets;
  a.rows = rows;
  a.part = part;
  a.T = T;
  a.r = r;
  a.L = L;
  a.chunk = chunk_of(T, d_in, d_out);
  a.n_mma = (r + 15) / 16 * 16;
  a.nc = (r + 63) / 64;
  a.bufs = a.n_mma <= 32 ? 2 : 1;
  a.status = device_status_ptr();
  a.limit_ns = kWaitLimitNs;
  const int smem = 1024 + STAGES * (BIG_BYTES + 3 * a.nc * CHUNK);
  if (cudaFuncSetAttribute(adapter_outer_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           160 * 1024) != cudaSuccess)
    return MOE_ERR_CUDA;
  CUtensorMap m0, m1;
  const uint64_t pd[3] = {(uint64_t)r, (uint64_t)T, 3}, ps[2] = {pd[0] * 2, pd[0] * pd[1] * 2};
  const uint32_t pbox[3] = {64, OT, 1};
  if (!make_map(&m0, planes_d_low, 3, pd, ps, pbox) || !make_map(&m1, planes_low, 3, pd, ps, pbox))
    return MOE_ERR_CUDA;
  launch_begin(K_ADAPTER_OUTER, st);
  // two CTAs an SM, of 256 TMEM columns each (one for a rank above 64, which takes all 512)
  const long long most = (long long)(T / a.chunk + L) * (a.tiles[0] + a.tiles[1]);
  const int ctas = (a.nc == 1 ? 2 : 1) * sm_count();
  launch_kernel(adapter_outer_kernel, dim3((unsigned)(most < ctas ? most : ctas)), dim3(THREADS),
                (size_t)smem, st, 1, m0, m1, a);
  const moe_status s = launch_end(K_ADAPTER_OUTER, st);
  if (s != MOE_OK || T <= a.chunk) return s;
  const size_t wide = (size_t)(d_in + d_out) * r;
  launch_begin(K_ADAPTER_OUTER_SUM, st);
  launch_kernel(adapter_outer_sum_kernel,
                dim3((unsigned)((wide + SUM_PIECE - 1) / SUM_PIECE), (unsigned)L),
                dim3(SUM_THREADS), 0, st, 1, a);
  return launch_end(K_ADAPTER_OUTER_SUM, st);
}

}  // namespace moe
