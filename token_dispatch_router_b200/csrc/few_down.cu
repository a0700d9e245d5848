// Second expert product of the few-token layer:
//   out[t] = sum over the experts e that keep t of  act[a(e), t] W_down[e]
// (act carries the routing weight: few_up.cu), tokens on M, one lane each, at most 128.
//
// Bound by reading W_down of those experts. For one output tile they are one long contraction,
// the k-blocks of all active experts in a line, accumulated in one place: no per-expert outputs
// and no combine. The MMA's lane mask (disable-output-lane) adds each expert's k-blocks to its
// own tokens only: the other rows of act are never written, nor read into a result, and an
// infinity or NaN in an expert that a token does not use cannot reach it.
//
// As in few_up.cu, the lines of all 128-column tiles are one line cut into equal pieces, one per
// SM; a tile cut by a piece's end leaves fp32 partials that the last of its SMs to finish adds in
// the line's order (nobody waits; results repeat bit for bit).
// The weights do not depend on the kernel before this one: a CTA fills its ring with them before
// it waits for that kernel (its launch follows that kernel's own wait, so everything older, the
// ids among it, is complete).
// Roles (256 threads): warp 0 copies weights, warp 1 rows of act, warp 2 issues the MMAs (two
// accumulators, so that one is read while the next is made), warps 4-7 read them. A finished wait
// costs a warp about 200 cycles and a copy or an MMA 60 to issue, so a stage is 128 k of 128
// columns, 32 KB brought by one copy and taken by eight MMAs.
// Every wait is bounded (MOE_ERR_TIMEOUT on expiry).
#include <math.h>

#include "few.cuh"
#include "few_args.cuh"
#include "ffn_args.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int THREADS = 256;
constexpr int BN = 128, BK = 128, PIECES = BK / 64;
constexpr int W_BYTES = BN * BK * 2;
constexpr int ROW_BOX = 8;     // rows of an act box
constexpr int MAX_STAGES = 6;
constexpr int MIN_BLOCKS = 2;  // stages of a piece, at least
constexpr int SMEM_LIMIT = 227 * 1024;
// A stage is the rows (for each 64 k: T rounded up to 8 rows of 128 bytes), then the weights. The
// MMA reads 128 rows: past T it runs on into what lies behind in the same stage, and those lanes
// are masked.

struct Tail {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES], tfull[2], tempty[2], done;
  uint32_t tmem;
  int abort, epi_ok, last;
  FewMasks m;
};

// D += A B in the lanes whose bit in `off` is clear.
__device__ __forceinline__ void mma_lanes(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, const uint32_t (&off)[4]) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.b32 p, %3, %3;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7}, p;\n\t}\n" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3])
      : "memory");
}
// 128 columns of 32 lanes set to zero.
__device__ __forceinline__ void tmem_zero(uint32_t at) {
#pragma unroll 1
  for (int c = 0; c < BN; c += 8)
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %1, %1, %1, %1, %1, %1, %1};" ::"r"(
            at + (uint32_t)c),
        "r"(0u)
        : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(THREADS, 1)
    few_down_kernel(const __grid_constant__ CUtensorMap tmA,
                    const __grid_constant__ CUtensorMap tmAll,
                    const __grid_constant__ CUtensorMap tmW, const FewDownArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Tail& t = *reinterpret_cast<Tail*>(base + g.stages * g.stage_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &t.abort;

  if (tid == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(saddr(&t.full[s]), 2);  // weights and rows
      mbar_init(saddr(&t.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(saddr(&t.tfull[b]), 1);
      mbar_init(saddr(&t.tempty[b]), 4);  // the epilogue warps
    }
    mbar_init(saddr(&t.done), 1);
    t.abort = 0;
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc<1>(saddr(&t.tmem), 2 * BN);
  // ids: written by the kernel before the previous one, which is complete
  few_build_masks(t.m, g.ids, g.T, g.K, g.E, g.cap, THREADS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = t.tmem;
  const uint64_t limit = g.limit_ns;
  const uint32_t x_piece = (uint32_t)(g.T + 7) / 8u * 1024u, x_bytes = PIECES * x_piece;
  const long long line = (long long)t.m.n_act * g.kb, total = line * g.nt;
  const int pieces = few_pieces(total, MIN_BLOCKS, (int)gridDim.x);
  const bool work = (int)blockIdx.x < pieces && total > 0;
  const long long b0 = work ? few_piece_begin(blockIdx.x, total, pieces) : 0;
  const long long b1 = work ? few_piece_begin(blockIdx.x + 1, total, pieces) : 0;

  if (warp == 0 || warp == 1) {
    // ------------------------------------------------------------ loads
    const bool x_warp = warp == 1;
    const int at0 = line > 0 ? (int)(b0 % line) : 0;
    int tile = line > 0 ? (int)(b0 / line) : 0, a = at0 / g.kb, k = at0 % g.kb, e = 0, groups = 0;
    unsigned mine = 0;  // warp 1: lane i copies the rows of tokens 8 i ... (groups with one)
    auto enter = [&]() {
      e = t.m.act[a];
      if (!x_warp) return;
      mine = lane < 16 ? t.m.mask[e][lane >> 2] >> (8 * (lane & 3)) & 0xffu : 0u;
      groups = __popc(__ballot_sync(0xffffffffu, mine != 0));
      if (2 * groups * 8 >= g.T || groups > 6) groups = 0;  // many: all rows in one copy
    };
    if (work) enter();
    if (x_warp) {
      pdl_wait();  // act is complete
      asm volatile("fence.proxy.async;" ::: "memory");  // and read by TMA
    }
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_par = 0;
    for (long long b = b0; b < b1; ++b) {
      if (!mbar_wait_warp(saddr(&t.empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) break;
      const uint32_t x = saddr(base + stage * g.stage_bytes), fb = saddr(&t.full[stage]);
      if (!x_warp) {
        if (elect_one()) {
          mbar_expect_tx(fb, W_BYTES);
          tma_load_4d(x + x_bytes, &tmW, 0, k * BK, tile * (BN / 64), e, fb);
        }
      } else if (groups == 0) {
        if (elect_one()) {
          mbar_expect_tx(fb, x_bytes);
          tma_load_4d(x, &tmAll, 0, a * g.T, k * PIECES, 0, fb);
        }
      } else {
        if (lane == 0) mbar_expect_tx(fb, (uint32_t)(groups * PIECES * ROW_BOX * 128));
        __syncwarp();
        if (mine != 0)
#pragma unroll
          for (int p = 0; p < PIECES; ++p)
            tma_load_4d(x + p * x_piece + lane * (ROW_BOX * 128), &tmA, 0, a * g.T + ROW_BOX * lane,
                        k * PIECES + p, 0, fb);
      }
      __syncwarp();
      issued_mask |= 1u << stage;
      issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
      if (++stage == g.stages) {
        stage = 0;
        phase ^= 1u;
      }
      if (++k == g.kb) {
        k = 0;
        if (++a == t.m.n_act) {
          a = 0;
          ++tile;
        }
        enter();
      }
    }
    if (lane == 0 && *abort_flag)
      for (int s = 0; s < g.stages; ++s) {
        // a wait ran out: let the copies in flight land (bounded; else the MMAs have read them)
        if (!(issued_mask & (1u << s))) continue;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try(saddr(&t.full[s]), (issued_par >> s) & 1u) &&
               globaltimer_ns() - t0 < limit) {
        }
      }
  } else if (warp == 2) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = idesc_bf16(128, BN);  // A (tokens) K-major, B (weights) MN-major
    const uint64_t xd0 = desc_sw128(saddr(base), 16, 1024);
    const uint64_t wd0 = desc_sw128(saddr(base) + x_bytes, BK * 128, 1024);
    const int at0 = line > 0 ? (int)(b0 % line) : 0;
    int stage = 0, it = 0, a = at0 / g.kb, k = at0 % g.kb;
    uint32_t phase = 0;
    bool ok = true;
    for (long long b = b0; b < b1 && ok; ++it) {
      const long long stop = min(b1, (b / line + 1) * line);
      const int buf = it & 1;
      // the accumulator has been read and set to zero
      if (!mbar_wait_warp(saddr(&t.tempty[buf]), (uint32_t)(it >> 1) & 1u, abort_flag, g.status,
                          limit))
        break;
      tc_fence_after();
      for (; b < stop; ++b) {
        // The mask is loaded anew for every stage. (Kept in registers across stages and replaced
        // only where the expert changes, some MMAs of later stages were issued with the mask of
        // an earlier expert.)
        const int e = t.m.act[a];
        uint32_t off[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) off[i] = ~*(volatile unsigned*)&t.m.mask[e][i];
        if (!mbar_wait_warp(saddr(&t.full[stage]), phase, abort_flag, g.status, limit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          uint64_t xd = xd0 + (uint64_t)((stage * g.stage_bytes) >> 4);
          uint64_t wd = wd0 + (uint64_t)((stage * g.stage_bytes) >> 4);
#pragma unroll 1
          for (int p = 0; p < PIECES; ++p, xd += x_piece >> 4, wd += 4 * 128)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_lanes(tmem + (uint32_t)(buf * BN), xd + (uint64_t)(kk * 2),
                        wd + (uint64_t)(kk * 128), idesc, off);
          tc_commit<1>(saddr(&t.empty[stage]));
        }
        __syncwarp();
        if (++stage == g.stages) {
          stage = 0;
          phase ^= 1u;
        }
        if (++k == g.kb) {
          k = 0;
          if (++a == t.m.n_act) a = 0;
        }
      }
      if (ok && elect_one()) tc_commit<1>(saddr(&t.tfull[buf]));
      __syncwarp();
    }
    if (elect_one()) tc_commit<1>(saddr(&t.done));
    __syncwarp();
    if (lane == 0) {  // every MMA has completed before TMEM is freed (bounded)
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try(saddr(&t.done), 0) && globaltimer_ns() - t0 < limit) {
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    // One thread waits for all four warps, so that they leave a wait that ran out together.
    const int q = warp & 3, row = q * 32 + lane;  // TMEM lane = token
    const bool first = tid == 128, rows_here = q * 32 < g.T, row_ok = row < g.T;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    for (int b = 0; b < 2; ++b) {  // accumulators start at zero: MMAs under a mask only add
      tmem_zero(tmem + (uint32_t)(b * BN) + lanes);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(saddr(&t.tempty[b]));
    }
    pdl_wait();  // the previous kernel in the stream has completed (order of writes to out)
    pdl_trigger();
    const bool bad = row_ok && (t.m.bad[row >> 5] >> (row & 31) & 1u);
    auto store = [&](int col, float (&f)[8]) {  // eight columns of this lane's row
      if (bad)  // NaN logits: no expert, and the row is NaN
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = NAN;
      if (row_ok && col < g.d)
        *reinterpret_cast<uint4*>(g.out + (size_t)row * g.d + col) = pack16(f, bf16());
    };
    if (total == 0 && row_ok) {  // no expert at all
      for (int c = 8 * (int)blockIdx.x; c < g.d; c += 8 * (int)gridDim.x) {
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        store(c, f);
      }
    }
    int it = 0;
    for (long long b = b0; b < b1; ++it) {
      const int tile = (int)(b / line);
      const long long tile0 = (long long)tile * line, tile1 = tile0 + line;
      const long long stop = min(b1, tile1);
      const bool whole = b == tile0 && stop == tile1;
      const int buf = it & 1, n0 = tile * BN;
      if (first)
        t.epi_ok = mbar_wait(saddr(&t.tfull[buf]), (uint32_t)(it >> 1) & 1u, abort_flag, g.status,
                             limit) ? 1 : 0;
      epi_bar();
      const bool ok = t.epi_ok != 0;
      epi_bar();  // everyone has read epi_ok
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(buf * BN) + lanes;
      // partials of a cut tile: [slot][4 columns][token][4]; a piece has at most two, the tile
      // that it begins in and the tile that begins in it
      const int slot = 2 * (int)blockIdx.x + (tile0 >= b0 ? 1 : 0);
      float4* part = reinterpret_cast<float4*>(g.part) + (size_t)slot * (BN / 4) * g.T + row;
      if (rows_here) {
#pragma unroll 2
        for (int c = 0; c < BN; c += 8) {
          uint32_t v[8];
          tmem_ld8(acc + (uint32_t)c, v);
          tmem_ld_wait();
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(v[j]);
          if (whole) {
            store(n0 + c, f);
          } else if (row_ok) {
            part[(size_t)(c / 4) * g.T] = make_float4(f[0], f[1], f[2], f[3]);
            part[(size_t)(c / 4 + 1) * g.T] = make_float4(f[4], f[5], f[6], f[7]);
          }
        }
        tmem_zero(acc);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(saddr(&t.tempty[buf]));
      if (!whole) {
        const int p0 = few_piece_of(tile0, total, pieces), p1 = few_piece_of(tile1 - 1, total, pieces);
        __threadfence();
        epi_bar();
        if (first) t.last = atomicAdd(g.arrived + p0, 1u) == (unsigned)(p1 - p0);
        epi_bar();
        if (t.last) {
          __threadfence();
          // all 128 threads over the tile's [8 columns][token] pieces
          for (int i = tid - 128; i < BN / 8 * g.T; i += 128) {
            const int c8 = i / g.T, tok = i % g.T, col = n0 + c8 * 8;
            if (col >= g.d) break;
            float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int p = p0; p <= p1; ++p) {
              const int s = 2 * p + (tile0 >= few_piece_begin(p, total, pieces) ? 1 : 0);
              const float4* pp = reinterpret_cast<const float4*>(g.part) +
                                 ((size_t)s * (BN / 4) + 2 * c8) * g.T + tok;
              const float4 u = __ldcg(pp), v = __ldcg(pp + g.T);
              f[0] += u.x; f[1] += u.y; f[2] += u.z; f[3] += u.w;
              f[4] += v.x; f[5] += v.y; f[6] += v.z; f[7] += v.w;
            }
            if (t.m.bad[tok >> 5] >> (tok & 31) & 1u)
#pragma unroll
              for (int j = 0; j < 8; ++j) f[j] = NAN;
            *reinterpret_cast<uint4*>(g.out + (size_t)tok * g.d + col) = pack16(f, bf16());
          }
        }
      }
      b = stop;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, 2 * BN);
  }
}

}  // namespace

size_t few_down_part_bytes(int T) { return (size_t)2 * sm_count() * T * BN * 4; }

// act: [active experts][T][n]; `active`: how many there can be.
moe_status launch_few_down(FewDownArgs a, int active, const void* act, const void* w_down,
                           cudaStream_t st) {
  a.kb = (a.n + BK - 1) / BK;
  a.nt = (a.d + BN - 1) / BN;
  const int rows = (a.T + 7) / 8 * 8;
  a.stage_bytes = W_BYTES + PIECES * rows * 128;
  const int fixed = 1024 + (int)sizeof(Tail);
  a.stages = (SMEM_LIMIT - fixed) / a.stage_bytes;
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  a.status = device_status_ptr();
  a.limit_ns = kWaitLimitNs;
  CUtensorMap boxes, all, mw;
  if (!make_piece_map(&boxes, act, (uint64_t)active * a.T, a.n, 1, ROW_BOX, 1) ||
      !make_piece_map(&all, act, (uint64_t)active * a.T, a.n, 1, (uint32_t)rows, PIECES) ||
      !make_piece_map(&mw, w_down, a.n, a.d, a.E, BK, BN / 64))
    return MOE_ERR_CUDA;
  if (cudaFuncSetAttribute(few_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           SMEM_LIMIT) != cudaSuccess)
    return MOE_ERR_CUDA;
  launch_begin(K_FEW_DOWN, st);
  launch_kernel(few_down_kernel, dim3((unsigned)sm_count()), dim3(THREADS),
                (size_t)(fixed + a.stages * a.stage_bytes), st, 1, boxes, all, mw, a);
  return launch_end(K_FEW_DOWN, st);
}

}  // namespace moe
