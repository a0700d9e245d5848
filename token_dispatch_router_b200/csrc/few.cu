// The products of a few tokens (at most 128) with weights that are read once: the expert half
// of the layer for single-token serving, and a shared projection with per-request adapters.
//
//   layer:       act = silu(x W_gate[e]) * (x W_up[e]),  y = act W_down[e],
//                out[t] = sum_k w[t, k] y[slot(t, k)]          (three phases, one kernel)
//   projection:  out = x W + low B[ids]                        (the last two phases)
//
// Bound by reading the weights of the experts that any token takes. So the weights are the
// MMA's A operand, 128 of their output columns on M, and the tokens its N (16 ... 128): a
// weight box goes from HBM to shared memory by TMA and into the tensor cores from there
// (MN-major, as it lies in memory), with no padding of tokens to 128 rows. Every token is on N
// for every expert: a token that is not routed to it costs a column that nobody reads, which
// is cheaper than gathering rows (the MMA of N = 128 takes a fraction of the time in which its
// 32 KB of weights arrive). Columns do not mix, so a NaN of one token stays in its row.
//
// Work is cut into units (expert, output tile, contraction split) that the CTAs take from one
// counter in order: all units of the first product, then all of the second, then the combine.
// A second-product unit waits for its expert's act tiles, a combine unit for all second-product
// units: both only wait for units with smaller numbers, which running CTAs hold and which wait
// for nothing larger, so the kernel ends however few of its CTAs are resident at a time.
// The contraction is split when there are fewer tiles than would fill the SMs a few times over
// (one token, few experts). First-product partials are added in split order by the CTA that
// arrives last; second-product partials by the combine: fixed orders, so results repeat bit
// for bit.
//
// Roles (256 threads): warp 0 takes units and loads weights, warp 2 loads x or act rows (it
// does the waiting, so weights run ahead), warp 1 issues the MMAs (two 128-column
// accumulators, double-buffered: all of TMEM), warp 3 owns the TMEM allocation, warps 4-7
// read the accumulators (lane = output column, column = token) and combine.
// Every wait is bounded; on expiry the status word records MOE_ERR_TIMEOUT and the CTA ends
// after its copies and MMAs in flight.
#include <math.h>

#include "few.cuh"
#include "ffn_args.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int THREADS = 256;
constexpr int BK = 64;
constexpr int W_CHUNK = 8192;         // 64 k-rows x 64 columns
constexpr int W_BYTES = 4 * W_CHUNK;  // gate 128 + up 128 columns, or 256 columns
constexpr int X_BOX = 2048;           // 16 rows x 64 k
constexpr int QD = 4;                 // units in flight inside a CTA
constexpr int MAX_STAGES = 6;
constexpr int COMBINE_COLS = 512;
constexpr uint32_t TMEM_COLS = 512;
constexpr int SMEM_LIMIT = 227 * 1024;

struct Tail {
  uint64_t full_w[MAX_STAGES], full_x[MAX_STAGES], empty[MAX_STAGES];
  uint64_t qfull[QD], qempty[QD], tfull[2], tempty[2], done;
  uint32_t tmem;
  int abort;
  int unit[QD];
  int epi_ok, epi_last;
  int n_act, off_total, s1, s2, u1, u2, u3;
  int off[kFewMaxExperts + 1];       // first slot of each expert
  unsigned mask[kFewMaxExperts][4];  // kept tokens of each expert
  short act[kFewMaxExperts];         // experts with at least one kept token
  float low[128];                    // projection: one token's low-rank values
};

// A unit: phase 1, 2 or 3 (0: no more). Phases 1 and 2: active expert a, output tile,
// contraction split s; phase 3: token a, 512-column piece `tile`.
struct Unit {
  int phase, a, tile, s;
};

__device__ __forceinline__ Unit decode_unit(int u, const FewArgs& g, const Tail& t) {
  if (u < t.u1) {
    const int per = g.nt1 * t.s1, r = u % per;
    return Unit{1, u / per, r % g.nt1, r / g.nt1};
  }
  u -= t.u1;
  if (u < t.u2) {
    const int per = g.nt2 * t.s2, r = u % per;
    return Unit{2, u / per, r % g.nt2, r / g.nt2};
  }
  u -= t.u2;
  const int nc = (g.d + COMBINE_COLS - 1) / COMBINE_COLS;
  if (u < t.u3) return Unit{3, u / nc, u % nc, 0};
  return Unit{0, 0, 0, 0};
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7])
      : "r"(taddr));
}
__device__ __forceinline__ unsigned ld_acquire(const uint32_t* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void add_release(uint32_t* p, unsigned v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Bounded wait for *p >= want (written by other CTAs).
__device__ __forceinline__ bool wait_count(const uint32_t* p, unsigned want, volatile int* abort,
                                           unsigned* status, uint64_t limit) {
  if (ld_acquire(p) >= want) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (ld_acquire(p) >= want) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > limit) {
      report(status, MOE_ERR_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ void epi_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}
__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fdividef(g, 1.f + __expf(-g)) * u;
}
// Kept tokens of expert e below token t.
__device__ __forceinline__ int rank_below(const unsigned (&m)[4], int t) {
  int r = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int lo = 32 * w;
    if (t >= lo + 32) r += __popc(m[w]);
    else if (t > lo) r += __popc(m[w] & ((1u << (t - lo)) - 1u));
  }
  return r;
}
__device__ __forceinline__ int split_of(int tiles, int target, int kb, int smax) {
  if (tiles <= 0 || tiles >= target) return 1;
  int s = (target + tiles - 1) / tiles;
  s = min(s, kb / 4);
  s = min(s, smax);
  return max(s, 1);
}

template <bool PROJ>
__global__ void __launch_bounds__(THREADS, 1)
    few_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmG,
               const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmA,
               const __grid_constant__ CUtensorMap tmD, const FewArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Tail& t = *reinterpret_cast<Tail*>(base + g.stages * g.stage_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &t.abort;

  if (tid == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(saddr(&t.full_w[s]), 1);
      mbar_init(saddr(&t.full_x[s]), 1);
      mbar_init(saddr(&t.empty[s]), 1);
    }
    for (int q = 0; q < QD; ++q) {
      mbar_init(saddr(&t.qfull[q]), 1);
      mbar_init(saddr(&t.qempty[q]), 3);  // MMA thread, x thread, the epilogue's first thread
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(saddr(&t.tfull[b]), 1);
      mbar_init(saddr(&t.tempty[b]), 4);  // the epilogue warps
    }
    mbar_init(saddr(&t.done), 1);
    t.abort = 0;
    mbar_init_fence();
  }
  if (warp == 3) tmem_alloc<1>(saddr(&t.tmem), TMEM_COLS);
  if (!PROJ)
    for (int i = tid; i < 4 * g.E; i += THREADS) (&t.mask[0][0])[i] = 0u;
  __syncthreads();
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();

  // ---- slots: each expert's kept tokens as a bit mask, its first slot, the active experts
  if (!PROJ) {
    for (int a = tid; a < g.T * g.K; a += THREADS) {
      const int e = g.ids[a], tok = a / g.K;
      if (e >= 0 && e < g.E) atomicOr(&t.mask[e][tok >> 5], 1u << (tok & 31));
    }
    __syncthreads();
    if (warp == 0) {
      int run = 0, nact = 0;
      for (int e0 = 0; e0 < g.E; e0 += 32) {
        const int e = e0 + lane;
        int c = 0;
        if (e < g.E) {
          // over the capacity: the first `cap` tokens stay
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            unsigned m = t.mask[e][w];
            while (c + __popc(m) > g.cap) m &= ~(0x80000000u >> __clz(m));
            t.mask[e][w] = m;
            c += __popc(m);
          }
        }
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        if (e < g.E) t.off[e] = run + incl - c;
        const unsigned has = __ballot_sync(0xffffffffu, c > 0);
        if (c > 0) t.act[nact + __popc(has & lanemask_lt())] = (short)e;
        nact += __popc(has);
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (lane == 0) {
        t.off[g.E] = run;
        t.n_act = nact;
      }
    }
  } else if (tid == 0) {
    t.off[0] = 0;
    t.off[1] = g.T;
    t.act[0] = 0;
    t.n_act = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0) {
    const int target = min(4 * (int)gridDim.x, kFewTarget);
    t.s1 = PROJ ? 1 : split_of(t.n_act * g.nt1, target, g.kb1, g.smax1);
    t.s2 = split_of(t.n_act * g.nt2, target, g.kb2, g.smax2);
    t.u1 = PROJ ? 0 : t.n_act * g.nt1 * t.s1;
    t.u2 = t.n_act * g.nt2 * t.s2;
    t.u3 = g.T * ((g.d + COMBINE_COLS - 1) / COMBINE_COLS);
  }
  __syncthreads();
  const uint32_t tmem = t.tmem;
  const uint64_t limit = g.limit_ns;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- units and weights
      int stage = 0, q = 0;
      uint32_t phase = 0, qphase = 0, issued_mask = 0, issued_par = 0;
      int next = (int)atomicAdd(g.ctl + kFewTicket, 1u);
      while (true) {
        const Unit u = decode_unit(next, g, t);
        if (!mbar_wait(saddr(&t.qempty[q]), qphase ^ 1u, abort_flag, g.status, limit)) break;
        t.unit[q] = next;
        mbar_arrive(saddr(&t.qfull[q]));
        if (++q == QD) {
          q = 0;
          qphase ^= 1u;
        }
        if (u.phase == 0) break;
        next = (int)atomicAdd(g.ctl + kFewTicket, 1u);  // one ahead: its latency is hidden
        if (u.phase == 3) continue;
        const int kb = u.phase == 1 ? g.kb1 : g.kb2, S = u.phase == 1 ? t.s1 : t.s2;
        const int k0 = u.s * kb / S, k1 = (u.s + 1) * kb / S;
        const int e = t.act[u.a];
        bool ok = true;
        for (int k = k0; k < k1; ++k) {
          if (!mbar_wait(saddr(&t.empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) {
            ok = false;
            break;
          }
          const uint32_t fb = saddr(&t.full_w[stage]);
          const uint32_t dst = saddr(base + stage * g.stage_bytes);
          mbar_expect_tx(fb, W_BYTES);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (u.phase == 1)
              tma_load_3d(dst + c * W_CHUNK, c < 2 ? &tmG : &tmU, u.tile * 128 + (c & 1) * 64,
                          k * BK, e, fb);
            else
              tma_load_3d(dst + c * W_CHUNK, &tmD, u.tile * 256 + c * 64, k * BK, e, fb);
          }
          issued_mask |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          if (++stage == g.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
      }
      for (int s = 0; s < g.stages; ++s) {  // nothing of ours is in flight after this (bounded)
        if (!(issued_mask & (1u << s))) continue;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try(saddr(&t.full_w[s]), (issued_par >> s) & 1u) &&
               globaltimer_ns() - t0 < limit) {
        }
      }
    }
  } else if (warp == 2) {
    if (lane == 0) {
      // ---------------------------------------------------------- x or act rows
      int stage = 0, q = 0;
      uint32_t phase = 0, qphase = 0, issued_mask = 0, issued_par = 0;
      while (true) {
        if (!mbar_wait(saddr(&t.qfull[q]), qphase, abort_flag, g.status, limit)) break;
        const Unit u = decode_unit(t.unit[q], g, t);
        mbar_arrive(saddr(&t.qempty[q]));
        if (++q == QD) {
          q = 0;
          qphase ^= 1u;
        }
        if (u.phase == 0) break;
        if (u.phase == 3) continue;
        const int kb = u.phase == 1 ? g.kb1 : g.kb2, S = u.phase == 1 ? t.s1 : t.s2;
        const int k0 = u.s * kb / S, k1 = (u.s + 1) * kb / S;
        const int e = t.act[u.a];
        int row0 = 0, boxes = g.npad / 16;
        const CUtensorMap* map = &tmX;
        if (u.phase == 2 && !PROJ) {
          if (!wait_count(g.ctl + kFewExpert + u.a, (unsigned)g.nt1, abort_flag, g.status, limit))
            break;
          fence_proxy_async_all();  // act was written by ordinary stores
          row0 = t.off[e];
          boxes = (t.off[e + 1] - row0 + 15) / 16;
          map = &tmA;
        }
        bool ok = true;
        for (int k = k0; k < k1; ++k) {
          if (!mbar_wait(saddr(&t.empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) {
            ok = false;
            break;
          }
          const uint32_t fb = saddr(&t.full_x[stage]);
          const uint32_t dst = saddr(base + stage * g.stage_bytes) + W_BYTES;
          mbar_expect_tx(fb, (uint32_t)(boxes * X_BOX));
          for (int i = 0; i < boxes; ++i)
            tma_load_2d(dst + i * X_BOX, map, k * BK, row0 + 16 * i, fb);
          issued_mask |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          if (++stage == g.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
      }
      for (int s = 0; s < g.stages; ++s) {
        if (!(issued_mask & (1u << s))) continue;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try(saddr(&t.full_x[s]), (issued_par >> s) & 1u) &&
               globaltimer_ns() - t0 < limit) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      // D fp32, A and B bf16, A MN-major (bit 15), B K-major, M = 128
      const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (8u << 24);
      int stage = 0, q = 0, it = 0;
      uint32_t phase = 0, qphase = 0;
      while (true) {
        if (!mbar_wait(saddr(&t.qfull[q]), qphase, abort_flag, g.status, limit)) break;
        const Unit u = decode_unit(t.unit[q], g, t);
        mbar_arrive(saddr(&t.qempty[q]));
        if (++q == QD) {
          q = 0;
          qphase ^= 1u;
        }
        if (u.phase == 0) break;
        if (u.phase == 3) continue;
        const int kb = u.phase == 1 ? g.kb1 : g.kb2, S = u.phase == 1 ? t.s1 : t.s2;
        const int k0 = u.s * kb / S, k1 = (u.s + 1) * kb / S;
        int N = g.npad;
        if (u.phase == 2 && !PROJ) {
          const int e = t.act[u.a];
          N = (t.off[e + 1] - t.off[e] + 15) / 16 * 16;
        }
        const uint32_t idesc = idesc0 | ((uint32_t)(N >> 3) << 17);
        const int buf = it & 1;
        const uint32_t use = (uint32_t)(it >> 1);
        ++it;
        if (!mbar_wait(saddr(&t.tempty[buf]), (use & 1u) ^ 1u, abort_flag, g.status, limit)) break;
        tc_fence_after();
        const uint32_t acc = tmem + (uint32_t)(buf * 256);
        bool ok = true;
        for (int k = k0; k < k1; ++k) {
          if (!mbar_wait(saddr(&t.full_w[stage]), phase, abort_flag, g.status, limit) ||
              !mbar_wait(saddr(&t.full_x[stage]), phase, abort_flag, g.status, limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t w = saddr(base + stage * g.stage_bytes), x = w + W_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t xd = desc_sw128(x + kk * 32, 16, 1024);
#pragma unroll
            for (int m = 0; m < 2; ++m)
              tc_mma<1>(acc + (uint32_t)(m * 128),
                        desc_sw128(w + m * 2 * W_CHUNK + kk * 2048, W_CHUNK, 1024), xd, idesc,
                        (k > k0 || kk > 0) ? 1u : 0u);
          }
          tc_commit<1>(saddr(&t.empty[stage]));
          if (++stage == g.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit<1>(saddr(&t.tfull[buf]));
      }
      tc_commit<1>(saddr(&t.done));  // every MMA has completed before TMEM is freed (bounded)
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try(saddr(&t.done), 0) && globaltimer_ns() - t0 < limit) {
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue and combine
    // One thread waits for all four warps, so that they leave a wait that ran out together.
    const int et = tid - 128, ew = warp - 4;
    const bool first = et == 0;
    int q = 0, it = 0;
    uint32_t qphase = 0;
    bool all_done = false;
    while (true) {
      if (first) {
        t.epi_ok = mbar_wait(saddr(&t.qfull[q]), qphase, abort_flag, g.status, limit) ? 1 : 0;
        if (t.epi_ok) {
          const Unit v = decode_unit(t.unit[q], g, t);
          if (v.phase == 1 || v.phase == 2)
            t.epi_ok = mbar_wait(saddr(&t.tfull[it & 1]), (uint32_t)(it >> 1) & 1u, abort_flag,
                                 g.status, limit) ? 1 : 0;
          else if (v.phase == 3 && !all_done)
            t.epi_ok = wait_count(g.ctl + kFewDone, (unsigned)t.u2, abort_flag, g.status, limit)
                           ? 1 : 0;
        }
      }
      epi_bar();
      if (!t.epi_ok) break;
      const Unit u = decode_unit(t.unit[q], g, t);
      epi_bar();  // every thread has read the unit and epi_ok
      if (first) mbar_arrive(saddr(&t.qempty[q]));
      if (++q == QD) {
        q = 0;
        qphase ^= 1u;
      }
      if (u.phase == 0) break;
      if (u.phase != 3) {
        const int buf = it & 1;
        ++it;
        tc_fence_after();
        const uint32_t acc = tmem + (uint32_t)(buf * 256) + ((uint32_t)(ew * 32) << 16);
        const int e = t.act[u.a], off = t.off[e], m_e = t.off[e + 1] - off;
        if (u.phase == 1) {
          const int cl = ew * 32 + lane, col = u.tile * 128 + cl;
          const bool col_ok = col < g.n;
          int slot = off;
          for (int c0 = 0; c0 < g.T; c0 += 8) {
            const unsigned bits = (t.mask[e][c0 >> 5] >> (c0 & 31)) & 0xffu;
            if (bits == 0) continue;
            uint32_t gv[8], uv[8];
            tmem_ld8(acc + (uint32_t)c0, gv);
            tmem_ld8(acc + (uint32_t)(128 + c0), uv);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (!(bits >> j & 1u)) continue;
              if (col_ok) {
                const float gf = __uint_as_float(gv[j]), uf = __uint_as_float(uv[j]);
                if (t.s1 == 1) {
                  g.act[(size_t)slot * g.n + col] = __float2bfloat16(silu_mul(gf, uf));
                } else {
                  float* p = g.part1 + (((size_t)slot * g.nt1 + u.tile) * t.s1 + u.s) * 256 + cl;
                  p[0] = gf;
                  p[128] = uf;
                }
              }
              ++slot;
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(saddr(&t.tempty[buf]));
          bool publish = true;
          if (t.s1 > 1) {  // the last of the tile's splits adds them up
            __threadfence();
            epi_bar();
            if (first)
              t.epi_last = atomicAdd(g.ctl + kFewTile + u.a * g.nt1 + u.tile, 1u) ==
                           (unsigned)(t.s1 - 1);
            epi_bar();
            publish = t.epi_last != 0;
            if (publish) {
              __threadfence();
              if (col_ok)
                for (int j = 0; j < m_e; ++j) {
                  const float* p =
                      g.part1 + ((size_t)(off + j) * g.nt1 + u.tile) * t.s1 * 256 + cl;
                  float gf = 0.f, uf = 0.f;
#pragma unroll 4
                  for (int s = 0; s < t.s1; ++s) {
                    gf += __ldcg(p + s * 256);
                    uf += __ldcg(p + s * 256 + 128);
                  }
                  g.act[(size_t)(off + j) * g.n + col] = __float2bfloat16(silu_mul(gf, uf));
                }
            }
          }
          if (publish) {
            fence_proxy_async_all();  // act is read by TMA
            __threadfence();
            epi_bar();
            if (first) add_release(g.ctl + kFewExpert + u.a, 1u);
          }
        } else {
          const int col = u.tile * 256 + ew * 32 + lane;
          const size_t rows = (size_t)g.T * g.K;
          float* y = g.y32 + ((size_t)u.s * rows + off) * g.d + col;
          for (int c0 = 0; c0 < m_e; c0 += 8) {
            uint32_t v0[8], v1[8];
            tmem_ld8(acc + (uint32_t)c0, v0);
            tmem_ld8(acc + (uint32_t)(128 + c0), v1);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (c0 + j >= m_e) continue;
              float* p = y + (size_t)(c0 + j) * g.d;
              if (col < g.d) p[0] = __uint_as_float(v0[j]);
              if (col + 128 < g.d) p[128] = __uint_as_float(v1[j]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(saddr(&t.tempty[buf]));
          __threadfence();
          epi_bar();
          if (first) add_release(g.ctl + kFewDone, 1u);
        }
        continue;
      }
      // ---- combine: 512 columns of one token, 4 a thread
      all_done = true;
      const int tok = u.a, col = u.tile * COMBINE_COLS + et * 4;
      const size_t rows = (size_t)g.T * g.K;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!PROJ) {
        if (col < g.d) {
          for (int k = 0; k < g.K; ++k) {
            const int e = g.ids[tok * g.K + k];
            const float w = g.topk_w[tok * g.K + k];
            if (e < 0 || e >= g.E) {  // NaN logits: no expert, and the row is NaN
              acc.x += NAN; acc.y += NAN; acc.z += NAN; acc.w += NAN;
              continue;
            }
            if (!(t.mask[e][tok >> 5] >> (tok & 31) & 1u)) continue;  // over the capacity
            const size_t slot = (size_t)(t.off[e] + rank_below(t.mask[e], tok));
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int s = 0; s < t.s2; ++s) {
              const float4 p = __ldcg(
                  reinterpret_cast<const float4*>(g.y32 + (s * rows + slot) * g.d + col));
              y.x += p.x; y.y += p.y; y.z += p.z; y.w += p.w;
            }
            acc.x = fmaf(w, y.x, acc.x); acc.y = fmaf(w, y.y, acc.y);
            acc.z = fmaf(w, y.z, acc.z); acc.w = fmaf(w, y.w, acc.w);
          }
        }
      } else {
        const int l = g.ids[tok];
        const bool has = l >= 0 && l < g.n_adapters;
        for (int j = et; j < g.rank; j += 128) {
          float v = 0.f;
          if (has)
            for (int s = 0; s < g.low_splits; ++s)
              v += g.low_part[((size_t)s * g.T + tok) * g.rank + j];
          if (has) v *= g.scale[l];
          t.low[j] = v;
          if (u.tile == 0) g.low[(size_t)tok * g.rank + j] = v;
        }
        epi_bar();
        if (col < g.d) {
#pragma unroll 4
          for (int s = 0; s < t.s2; ++s) {
            const float4 p = __ldcg(
                reinterpret_cast<const float4*>(g.y32 + (s * rows + tok) * g.d + col));
            acc.x += p.x; acc.y += p.y; acc.z += p.z; acc.w += p.w;
          }
          if (has) {
            const bf16* bp = g.b + (size_t)l * g.rank * g.d + col;
#pragma unroll 8
            for (int j = 0; j < g.rank; ++j) {
              const uint2 raw = *reinterpret_cast<const uint2*>(bp + (size_t)j * g.d);
              const float v = t.low[j];
              acc.x = fmaf(v, __uint_as_float(raw.x << 16), acc.x);
              acc.y = fmaf(v, __uint_as_float(raw.x & 0xffff0000u), acc.y);
              acc.z = fmaf(v, __uint_as_float(raw.y << 16), acc.z);
              acc.w = fmaf(v, __uint_as_float(raw.y & 0xffff0000u), acc.w);
            }
          }
        }
        epi_bar();  // t.low is free for the next unit
      }
      if (col < g.d)
        *reinterpret_cast<uint2*>(g.out + (size_t)tok * g.d + col) =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, TMEM_COLS);
  }
}

template <bool PROJ>
moe_status run_few(const CUtensorMap& x, const CUtensorMap& wg, const CUtensorMap& wu,
                   const CUtensorMap& act, const CUtensorMap& wd, FewArgs& a, cudaStream_t st) {
  a.npad = (a.T + 15) / 16 * 16;
  a.stage_bytes = W_BYTES + a.npad * 128;
  a.stages = (SMEM_LIMIT - 1024 - (int)sizeof(Tail)) / a.stage_bytes;
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  const int smem = 1024 + a.stages * a.stage_bytes + (int)sizeof(Tail);
  auto kern = few_kernel<PROJ>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  const int kid = PROJ ? K_ADAPTER_FEW : K_DECODE;
  launch_begin(kid, st);
  launch_kernel(kern, dim3((unsigned)sm_count()), dim3(THREADS), (size_t)smem, st, 1, x, wg, wu,
                act, wd, a);
  return launch_end(kid, st);
}

}  // namespace

// How many contraction splits of `bytes` a partial buffer is given room for: 32 MB in all.
static int split_room(size_t bytes) {
  const size_t n = ((size_t)32 << 20) / (bytes > 0 ? bytes : 1);
  return n < 1 ? 1 : n > (size_t)kFewMaxSplit ? kFewMaxSplit : (int)n;
}

static size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Workspace of the layer for few tokens (bytes from its start).
struct DecodeLayout {
  size_t ctl, ids, w, act, part1, y32, total;
  int smax1, smax2;
};

static DecodeLayout decode_layout(const moe_shape& s) {
  DecodeLayout L;
  const size_t A = (size_t)s.T * s.K, nt1 = (size_t)(s.n + 127) / 128;
  const size_t p1 = A * nt1 * 256 * 4, p2 = A * (size_t)s.d * 4;
  L.smax1 = split_room(p1);
  L.smax2 = split_room(p2);
  size_t o = 0;
  L.ctl = o;
  o = up256(o + kFewCtlWords * 4);
  L.ids = o;
  o = up256(o + A * 4);
  L.w = o;
  o = up256(o + A * 4);
  L.act = o;
  o = up256(o + A * (size_t)s.n * 2);
  L.part1 = o;
  if (L.smax1 > 1) o = up256(o + p1 * (size_t)L.smax1);
  L.y32 = o;
  o = up256(o + p2 * (size_t)L.smax2);
  L.total = o;
  return L;
}

size_t decode_workspace_bytes(const moe_shape& s) { return decode_layout(s).total; }

moe_status launch_few_route(const moe_shape& s, const void* x, const void* w_r, const float* bias,
                            const float* logits_in, int32_t* ids, float* w, uint32_t* clear,
                            int n_clear, cudaStream_t st);

moe_status launch_decode(const moe_shape& s, const void* x, const void* w_r, const float* bias,
                         const float* logits_in, const void* w_gate, const void* w_up,
                         const void* w_down, void* out, int cap, uint8_t* ws,
                         cudaStream_t st) {
  const DecodeLayout L = decode_layout(s);
  int32_t* ids = (int32_t*)(ws + L.ids);
  float* w = (float*)(ws + L.w);
  uint32_t* ctl = (uint32_t*)(ws + L.ctl);
  FewArgs a = {};
  a.T = s.T;
  a.K = s.K;
  a.E = s.E;
  a.kb1 = s.d / BK;
  a.kb2 = s.n / BK;
  a.n = s.n;
  a.nt1 = (s.n + 127) / 128;
  a.d = s.d;
  a.nt2 = (s.d + 255) / 256;
  a.smax1 = L.smax1;
  a.smax2 = L.smax2;
  a.cap = cap;
  a.ids = ids;
  a.topk_w = w;
  a.ctl = ctl;
  a.act = (bf16*)(ws + L.act);
  a.part1 = (float*)(ws + L.part1);
  a.y32 = (float*)(ws + L.y32);
  a.out = (bf16*)out;
  a.status = device_status_ptr();
  a.limit_ns = kWaitLimitNs;
  CUtensorMap mx, mg, mu, ma, md;
  const uint64_t d = s.d, n = s.n, E = s.E, A = (uint64_t)s.T * s.K;
  const uint32_t wbox[3] = {64, 64, 1}, xbox[2] = {64, 16};
  const uint64_t wd1[3] = {n, d, E}, ws1[2] = {n * 2, d * n * 2};
  const uint64_t wd2[3] = {d, n, E}, ws2[2] = {d * 2, n * d * 2};
  const uint64_t xd[2] = {d, (uint64_t)s.T}, xs[1] = {d * 2};
  const uint64_t ad[2] = {n, A}, as[1] = {n * 2};
  if (!make_map(&mx, x, 2, xd, xs, xbox) || !make_map(&mg, w_gate, 3, wd1, ws1, wbox) ||
      !make_map(&mu, w_up, 3, wd1, ws1, wbox) || !make_map(&ma, a.act, 2, ad, as, xbox) ||
      !make_map(&md, w_down, 3, wd2, ws2, wbox))
    return MOE_ERR_CUDA;
  const moe_status r =
      launch_few_route(s, x, w_r, bias, logits_in, ids, w, ctl, kFewCtlWords, st);
  if (r != MOE_OK) return r;
  return run_few<false>(mx, mg, mu, ma, md, a, st);
}

// y = x W + low B[ids] for at most kFewMaxTokens rows; low_part [low_splits][T][rank] are the
// partial sums of x A[ids], y32 has room for `smax` partials of [T, d_out].
int adapter_few_splits(int T, int d_out) { return split_room((size_t)T * d_out * 4); }

moe_status launch_adapter_few(int T, int d_in, int d_out, int n_adapters, int rank, const void* x,
                              const void* w, const void* b, const int32_t* ids,
                              const float* scale, const float* low_part, int low_splits,
                              float* low, void* y, float* y32, int smax, uint32_t* ctl,
                              cudaStream_t st) {
  FewArgs a = {};
  a.T = T;
  a.K = 1;
  a.E = 1;
  a.kb1 = 0;
  a.kb2 = d_in / BK;
  a.d = d_out;
  a.nt2 = (d_out + 255) / 256;
  a.smax1 = 1;
  a.smax2 = smax;
  a.cap = T;
  a.ids = ids;
  a.ctl = ctl;
  a.y32 = y32;
  a.out = (bf16*)y;
  a.low_part = low_part;
  a.low = low;
  a.b = (const bf16*)b;
  a.scale = scale;
  a.rank = rank;
  a.low_splits = low_splits;
  a.n_adapters = n_adapters;
  a.status = device_status_ptr();
  a.limit_ns = kWaitLimitNs;
  CUtensorMap mx, mw;
  const uint32_t wbox[3] = {64, 64, 1}, xbox[2] = {64, 16};
  const uint64_t k = d_in, n = d_out;
  const uint64_t wd[3] = {n, k, 1}, ws[2] = {n * 2, k * n * 2};
  const uint64_t xd[2] = {k, (uint64_t)T}, xs[1] = {k * 2};
  if (!make_map(&mx, x, 2, xd, xs, xbox) || !make_map(&mw, w, 3, wd, ws, wbox))
    return MOE_ERR_CUDA;
  return run_few<true>(mx, mw, mw, mx, mw, a, st);
}

}  // namespace moe
