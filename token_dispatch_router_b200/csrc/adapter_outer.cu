// Gradients of the adapter matrices: for each adapter l, over its rows t,
//
//   dA_l [d_in, r] = sum_t x[t]^T d_low[t],    dB_l [r, d_out] = sum_t low[t]^T d_y[t]
//
// Bound by reading the wide rows of x and d_y once. Rows come in any order, so they are
// gathered by cp.async into the swizzled layout that the tensor cores read; both operands are
// taken as they lie (a row is one k of the product: MN-major), so nothing is transposed. M is
// the wide side (256 columns a unit, two accumulators), N the rank (16 ... 128), K the rows.
// The low-rank side is fp32: it enters as three bf16 terms, which hold it exactly (bf16_terms); the
// tensor pipe has the time (three MMAs of N = r for each 32 x 256 tile of wide rows). The tensor core cuts what
// it adds to an accumulator off rather than rounding it, an error that grows with the number of
// additions: the small second and third terms have an accumulator of their own, added to the
// first's at the end (512 rows, relative to the gradient: 1.7e-6 in one accumulator, 0.5e-6 in two).
//
// A unit is (adapter, 256 columns of x or of d_y). The units' row steps lie on a line, each unit
// with a few positions more for its stores, and the line is cut into equal pieces, one a CTA, two
// CTAs an SM: adapters have any number of rows (units of at most 512 rows, taken in turn, left
// some CTAs three of them and others two: 8192 rows of 8 adapters, 4096 + 4096 columns, the last
// CTA ended 36 us after the median one, of 77). Units that a cut goes through leave partial sums,
// at most two a CTA, that the sum kernel adds in order (results repeat bit for bit). Up to 512
// rows units stay whole and leave nothing to add. An adapter without rows writes zeros. Up to rank
// 32 TMEM holds the accumulators of two units, so that the products of the next run beside the
// stores of the last.
//
// After the large product the kernel starts as that one's CTAs leave: it reads nothing of it
// (300 rows, 2048 -> 768: 28.0 us a call after it, 23.7 beside its end).
// What bounds it is latency: 8192 rows as above take a CTA 37 us for 23 steps, neither fewer
// copies nor a third of the MMAs change the call by more than 2 %, and six stages for one CTA an
// SM take as long as three for two. The stores of a unit are 14 us of the call's 284.
// Every wait (but tmem_alloc's) is bounded (MOE_ERR_TIMEOUT on expiry).
#include "adapter.cuh"
#include "few.cuh"
#include "ffn_args.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int LOADERS = 128, THREADS = 320;  // four gather warps, MMA, TMA, four store warps
constexpr int OC = kAdapterUnitCols;         // columns of a unit
constexpr int OT = 32;                       // rows per stage
constexpr int STAGES = 3;
constexpr int CHUNK = OT * 128;              // OT rows x 64 columns
constexpr int BIG_BYTES = OC / 64 * CHUNK;   // 16 KB
constexpr int kMaxAdapters = 256;
constexpr int CHAIN = 32;    // steps in one accumulator; a longer unit's sums are added in fp32
// Up to here units are not cut: the longest takes 16 steps, the sum's launch about as long
// (backward, 500 rows, 1024 -> 1024, rank 32: six adapters 22.8 us whole, 26.2 cut; one, 28.3 and
// 25.8; 300 rows, 2048 -> 768, rank 8: 20.6 and 22.7).
constexpr int WHOLE_ROWS = 512;

struct OuterArgs {
  const bf16* big[2];     // x [T, D0], d_y [T, D1]
  const bf16* planes[2];  // d_low, low: [3][T][r] in slot order
  float* out[2];          // dA [L, D0, r], dB [L, r, D1]
  int D[2], tiles[2];     // widths and their 256-column tiles
  const int32_t* offsets;
  const int32_t* rows;
  float* part;        // [2 CTAs][256 r]: the units that a piece begins and ends inside
  AdapterCut* cuts;    // [CTAs]
  int T, r, L;
  int ctas, cut;      // pieces at most; whether a piece may end inside a unit
  int store;          // positions of a unit's stores
  int early;          // the previous kernel is none that this one reads from
  int n_mma;          // the rank rounded up to 16
  int nc;             // its 64-column pieces
  int bufs;           // units whose accumulators TMEM holds: 1 or 2
  unsigned* status;
  unsigned long long limit_ns;
};

// The line: first position of each adapter (`base`), whose units, one a column tile, have
// steps + store positions each.
struct Line {
  int base[kMaxAdapters + 1];
};
__device__ __forceinline__ int steps_of(int l, const OuterArgs& g) {
  return (g.offsets[l + 1] - g.offsets[l] + OT - 1) / OT;
}
__device__ __forceinline__ void make_line(Line& t, const OuterArgs& g) {  // one warp
  const int lane = threadIdx.x & 31, nct = g.tiles[0] + g.tiles[1];
  int run = 0;
  for (int l0 = 0; l0 < g.L; l0 += 32) {
    const int l = l0 + lane, n = l < g.L ? (steps_of(l, g) + g.store) * nct : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (l < g.L) t.base[l] = run + incl - n;
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) t.base[g.L] = run;
}
__device__ __forceinline__ int adapter_at(int pos, const Line& t, int L) {
  int lo = 0, hi = L - 1;  // the last adapter that begins at pos or before
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.base[mid] <= pos) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ FewPieces pieces_of(const Line& t, const OuterArgs& g) {
  return FewPieces(t.base[g.L], 4, g.ctas);
}

// The parts of units in this CTA's piece, one after another.
struct Walk {
  int pos, end;                  // of the piece, still to come
  int l, p, c0, lo, n, s0, s1;   // adapter, side, first column; the adapter's first slot and rows; steps
  int slot;                      // place of the partial, -1 where the unit is whole
  __device__ __forceinline__ Walk(const Line& t, const OuterArgs& g) {
    const FewPieces pc = pieces_of(t, g);
    const int c = blockIdx.x;
    pos = c < pc.n ? pc.begin(c) : 0;
    end = c < pc.n ? pc.begin(c + 1) : 0;
    l = pos < end ? adapter_at(pos, t, g.L) : 0;
  }
  __device__ __forceinline__ bool next(const Line& t, const OuterArgs& g) {
    while (pos < end) {
      while (t.base[l + 1] <= pos) ++l;
      lo = g.offsets[l];
      n = g.offsets[l + 1] - lo;
      const int steps = (n + OT - 1) / OT, w = steps + g.store;
      const int ct = (pos - t.base[l]) / w, u0 = t.base[l] + ct * w;
      const int a = pos - u0, b = g.cut ? min(end - u0, w) : w;
      pos = u0 + b;
      s0 = a;
      s1 = min(b, steps);
      // a unit that is not cut belongs to the piece that holds its first position
      if (steps == 0 || !g.cut ? a > 0 : s0 >= s1) continue;
      p = ct >= g.tiles[0] ? 1 : 0;
      c0 = (ct - (p ? g.tiles[0] : 0)) * OC;
      slot = s0 > 0 ? 2 * (int)blockIdx.x : s1 < steps ? 2 * (int)blockIdx.x + 1 : -1;
      return true;
    }
    return false;
  }
};

// Whether this CTA's piece is the first that begins inside a unit.
__device__ __forceinline__ AdapterCut cut_of(const Line& t, const OuterArgs& g) {
  const FewPieces pc = pieces_of(t, g);
  const int c = blockIdx.x;
  if (c == 0 || c >= pc.n) return AdapterCut{-1, 0, 0, 0};
  const int b = pc.begin(c), l = adapter_at(b, t, g.L);
  const int steps = steps_of(l, g), w = steps + g.store, ct = (b - t.base[l]) / w;
  const int u0 = t.base[l] + ct * w;
  if (b == u0 || b - u0 >= steps || pc.begin(c - 1) > u0) return AdapterCut{-1, 0, 0, 0};
  const int p = ct >= g.tiles[0] ? 1 : 0;
  return AdapterCut{l, p, (ct - (p ? g.tiles[0] : 0)) * OC, pc.of(u0 + steps - 1)};
}

__global__ void __launch_bounds__(THREADS)
    adapter_outer_kernel(const __grid_constant__ CUtensorMap tmP0,
                         const __grid_constant__ CUtensorMap tmP1, const OuterArgs g) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ Line line;
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
  if (tid == 32) {
    prefetch_map(&tmP0);
    prefetch_map(&tmP1);
  }
  // early: the large product before this kernel waited for what both read, and wrote none of it
  if (!g.early) pdl_wait();  // the previous kernel in the stream has completed
  // TMEM is taken after that wait (the previous kernel's CTAs may still be waiting for theirs), and
  // the next kernel in the stream may start only then: one that takes TMEM before it waits for this
  // kernel, beside this CTA, could hold what this CTA still needs.
  if (warp == 4) {
    tmem_alloc<1>(saddr(&s_tmem), tcols);
    pdl_trigger();
  }
  if (warp == 0) make_line(line, g);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const uint64_t limit = g.limit_ns;
  Walk v(line, g);
  if (g.cut && tid == 0) g.cuts[blockIdx.x] = cut_of(line, g);

  if (warp < 4) {
    // ------------------------------------------------------------ gather
    // wide rows: warp w copies rows w, w + 4, ..., 512 bytes (one 16-byte piece a lane) each
    const int chunk_at = (lane >> 3) * CHUNK, pieces = g.n_mma / 8;
    const size_t plane = (size_t)g.T * g.r;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && v.next(line, g)) {
      const int D = g.D[v.p];
      const bf16* big = g.big[v.p] + v.c0 + lane * 8;
      const bool col_on = v.c0 + lane * 8 < D;
      // lane i < 8 holds the row of this warp's i-th row in the next stage
      auto row_of = [&](int s) {
        const int r = s * OT + warp + 4 * (lane & 7);
        return r < v.n ? g.rows[v.lo + r] : -1;
      };
      int ahead = v.s0 < v.s1 ? row_of(v.s0) : -1;
      for (int s = v.s0; s < v.s1; ++s) {
        const int mine = ahead;
        if (s + 1 < v.s1) ahead = row_of(s + 1);
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
    while (ok && v.next(line, g)) {
      for (int s = v.s0; s < v.s1; ++s) {
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
    while (ok && v.next(line, g)) {
      int s = v.s0;
      do {  // chains of at most CHAIN steps
        const int c0 = s, c1 = min(v.s1, s + CHAIN), buf = it & (g.bufs - 1);
        if (!mbar_wait_warp(saddr(&tempty[buf]), ((uint32_t)(it >> (g.bufs - 1)) & 1u) ^ 1u,
                            abort_flag, g.status, limit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t acc = tmem + (uint32_t)(buf * 4 * g.n_mma);
        for (; s < c1; ++s) {
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
                            (s > c0 || q > 1 || kk > 0) ? 1u : 0u);
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
        ++it;
      } while (ok && s < v.s1);
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
    int it = 0;
    bool ok = true;
    while (ok && v.next(line, g)) {
      const int D = g.D[v.p], width = v.slot < 0 ? D : OC;  // of the destination
      float* dst = v.slot < 0 ? g.out[v.p] + (size_t)v.l * D * g.r +
                                    (v.p ? (size_t)v.c0 : (size_t)v.c0 * g.r)
                              : g.part + (size_t)v.slot * OC * g.r;
      int s = v.s0;
      do {
        const int buf = it & (g.bufs - 1);
        const bool more = s > v.s0;  // another chain of the same unit: added to what is there
        if (!mbar_wait_warp(saddr(&tfull[buf]), (uint32_t)(it >> (g.bufs - 1)) & 1u, abort_flag,
                            g.status, limit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t acc = tmem + (uint32_t)(buf * 4 * g.n_mma) + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
        for (int m = 0; m < 2; ++m) {
          const int c = m * 128 + q * 32 + lane;
#pragma unroll 2
          for (int j0 = 0; j0 < g.r; j0 += 8) {
            float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (v.n > 0) {  // else no rows: zeros
              uint32_t f1[8], f2[8];
              tmem_ld8(acc + (uint32_t)(m * g.n_mma + j0), f1);
              tmem_ld8(acc + (uint32_t)((2 + m) * g.n_mma + j0), f2);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(f1[j]) + __uint_as_float(f2[j]);
            }
            if (v.c0 + c >= D) continue;
            if (v.p == 0) {
              float4* o = reinterpret_cast<float4*>(dst + (size_t)c * g.r + j0);
              float4 u0 = make_float4(f[0], f[1], f[2], f[3]);
              float4 u1 = make_float4(f[4], f[5], f[6], f[7]);
              if (more) {
                const float4 w0 = o[0], w1 = o[1];
                u0.x += w0.x; u0.y += w0.y; u0.z += w0.z; u0.w += w0.w;
                u1.x += w1.x; u1.y += w1.y; u1.z += w1.z; u1.w += w1.w;
              }
              o[0] = u0;
              o[1] = u1;
            } else {
              float* o = dst + (size_t)j0 * width + c;
              if (more)
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] += o[(size_t)j * width];
#pragma unroll
              for (int j = 0; j < 8; ++j) o[(size_t)j * width] = f[j];
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(saddr(&tempty[buf]));
        s = min(v.s1, s + CHAIN);
        ++it;
      } while (s < v.s1);
    }
  }
  __syncwarp();  // lanes that waited alone are back
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, tcols);
  }
  if (g.early) pdl_wait();  // what follows this kernel finds the one before it complete, too
}

int tiles_of(int d) { return (d + OC - 1) / OC; }

// Pieces: two CTAs an SM, of 256 TMEM columns each (one for a rank above 64, which takes all 512).
int ctas_of(int r) { return (r <= 64 ? 2 : 1) * sm_count(); }

}  // namespace

// Partial sums, two a piece, and the table of cuts.
size_t adapter_outer_part_bytes(int T, int r) {
  return T <= WHOLE_ROWS ? 0 : (size_t)ctas_of(r) * (2 * OC * r * 4 + sizeof(AdapterCut));
}

// early: the kernel launched last is the large product, which waited for all that is read here.
moe_status launch_adapter_outer(int T, int d_in, int d_out, int r, int L, const void* x,
                                const void* d_y, const void* planes_d_low,
                                const void* planes_low, const int32_t* offsets,
                                const int32_t* rows, float* d_a, float* d_b, float* part,
                                bool early, cudaStream_t st) {
  OuterArgs a = {};
  a.out[0] = d_a;
  a.out[1] = d_b;
  a.D[0] = d_in;
  a.D[1] = d_out;
  a.tiles[0] = tiles_of(d_in);
  a.tiles[1] = tiles_of(d_out);
  a.offsets = offsets;
  a.part = part;
  a.cuts = (AdapterCut*)(part + (size_t)2 * ctas_of(r) * OC * r);
  a.T = T;
  a.r = r;
  a.L = L;
  a.ctas = ctas_of(r);
  a.cut = T > WHOLE_ROWS;
  a.store = 1 + r / 32;
  a.big[0] = (const bf16*)x;
  a.big[1] = (const bf16*)d_y;
  a.planes[0] = (const bf16*)planes_d_low;
  a.planes[1] = (const bf16*)planes_low;
  a.rows = rows;
  a.early = early;
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
  launch_kernel(adapter_outer_kernel, dim3((unsigned)a.ctas), dim3(THREADS), (size_t)smem, st, 1,
                m0, m1, a);
  return launch_end(K_ADAPTER_OUTER, st);
}

// What launch_adapter_outer leaves to add.
AdapterUnitSums adapter_outer_sums(int T, int d_in, int d_out, int r, float* d_a, float* d_b,
                                   const float* part) {
  AdapterUnitSums s = {};
  s.D[0] = d_in;
  s.D[1] = d_out;
  s.r = r;
  s.pieces = T > WHOLE_ROWS ? ctas_of(r) : 0;
  s.part = part;
  s.cuts = (const AdapterCut*)(part + (size_t)2 * ctas_of(r) * OC * r);
  s.out[0] = d_a;
  s.out[1] = d_b;
  return s;
}

}  // namespace moe
