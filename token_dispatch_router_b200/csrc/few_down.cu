// Second expert product of the few-token layer:
//   out[t] = sum over the experts e that keep t of  act[a(e), t] W_down[e]
// (act carries the routing weight: few_up.cu), at most 128 tokens.
//
// Bound by reading W_down of those experts; as in few_up.cu the weights are the MMA's A operand,
// 128 output columns on M, and an expert's tokens its N. An output tile's line is the k-blocks of
// all active experts; each expert's product is made in an accumulator of its own and then added
// to its tokens' columns of the tile, which stays in TMEM for the whole line: no per-expert
// outputs in memory and no combine, and what an expert computes touches its own tokens only.
//
// The lines of all tiles are one line cut into equal pieces, one per SM. A tile cut by a piece's
// end leaves fp32 partials that a small kernel behind this one adds in the line's order (results
// repeat bit for bit). Its CTAs wait beside the running ones and all SMs take part; the last SM to
// finish a tile adding them up alone took 40 us of 230 (128 tokens, width 4096, 8 experts of
// 14336), and clusters that split a tile and add through distributed shared memory find no room
// for all of them while the kernel before drains.
// The weights do not depend on the kernel before this one: a CTA fills its ring with them before
// it waits for that kernel (its launch follows that kernel's own wait, so everything older, the
// ids among it, is complete).
// Roles (256 threads): warp 0 copies weights, warp 1 the expert's rows of act, eight a copy (two
// warps with cp.async: 30 us of 515 at 128 tokens, width 4096, 8 experts of 14336), warp 2 issues
// the MMAs (two accumulators, so that one is added while the next is made), warps 4-7 add and store. A finished wait costs a warp about 200 cycles and a copy or an
// MMA 60 to issue, so a stage is 128 k of 128 columns, 32 KB brought by one copy and taken by
// eight MMAs.
// Every wait (but tmem_alloc's) is bounded (MOE_ERR_TIMEOUT on expiry).
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
constexpr int X_ROWS = 8;      // rows of act a copy
constexpr int MAX_STAGES = 6;
constexpr int MIN_BLOCKS = 2;  // stages of a piece, at least
constexpr int SMEM_LIMIT = 227 * 1024;
// TMEM: columns 0 ... 127 the tile (column = token), then two accumulators of up to 128 tokens
constexpr uint32_t TMEM_COLS = 512, ACC = kFewMaxTokens;

struct Tail {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES], tfull[2], tempty[2], done;
  uint32_t tmem;
  int abort;
  FewMasks m;
  // every expert's tokens, ascending: expert e's from first[e]
  short first[kFewMaxExperts];
  unsigned char tok[kFewMaxTokens * 32];
};

__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr));
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(THREADS, 1)
    few_down_kernel(const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ CUtensorMap tmX, const FewDownArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Tail& t = *reinterpret_cast<Tail*>(base + g.ring_bytes);  // behind rows and weights
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &t.abort;
  if (tid == 0) {
    for (int s = 0; s < MAX_STAGES; ++s) {
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
  if (warp == 2) tmem_alloc<1>(saddr(&t.tmem), TMEM_COLS);
  if (tid == 96) {
    prefetch_map(&tmW);
    prefetch_map(&tmX);
  }
  few_clear_masks(t.m, g.E, THREADS);
  // ids: written by the kernel before the previous one, which is complete
  few_build_masks(t.m, g.ids, g.T, g.K, g.E, g.cap, THREADS);
  for (int i = tid; i < t.m.n_act; i += THREADS) {
    int at = 0;
    for (int j = 0; j < i; ++j) at += few_count(t.m.mask[t.m.act[j]]);
    const int e = t.m.act[i];
    t.first[e] = (short)at;
    for (int w = 0; w < 4; ++w)
      for (unsigned m = t.m.mask[e][w]; m != 0; m &= m - 1)
        t.tok[at++] = (unsigned char)(32 * w + __ffs(m) - 1);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = t.tmem;
  const uint64_t limit = g.limit_ns;
  // a stage: the weights, then for each 64 k a row of 128 bytes for each of an expert's tokens;
  // the largest expert's tokens, rounded up to 16, set its size
  const uint32_t x_most = (uint32_t)(t.m.most + 15) / 16u * (16u * 128u);
  const uint32_t stage_bytes = W_BYTES + PIECES * x_most, ring = saddr(base);
  const int stages = min(MAX_STAGES, (int)((uint32_t)g.ring_bytes / stage_bytes));
  const int line = t.m.n_act * g.kb, total = line * g.nt;
  const FewPieces cut(total, MIN_BLOCKS, (int)gridDim.x);
  const bool work = (int)blockIdx.x < cut.n && total > 0;
  const int b0 = work ? cut.begin(blockIdx.x) : 0, b1 = work ? cut.begin(blockIdx.x + 1) : 0;
  const int at0 = line > 0 ? b0 % line : 0;  // of the first block, in its tile's line

  // Nothing that a load warp issued is in flight after this (bounded). A stage is full once both
  // warps' copies into it have landed; one that the other never issued runs out, too.
  auto drain = [&](uint32_t issued, uint32_t par) {
    if (lane == 0)
      for (int s = 0; s < stages; ++s) {
        if (!(issued & (1u << s))) continue;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try(saddr(&t.full[s]), (par >> s) & 1u) && globaltimer_ns() - t0 < limit) {
        }
      }
  };

  if (warp == 0) {
    // ------------------------------------------------------------ weights
    int tile = line > 0 ? b0 / line : 0, a = at0 / g.kb, k = at0 % g.kb, stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_par = 0;
    const uint64_t once = l2_policy_evict_first();  // read once: act stays in L2
    for (int b = b0; b < b1; ++b) {
      if (!mbar_wait_warp(saddr(&t.empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) break;
      if (elect_one()) {
        const uint32_t fb = saddr(&t.full[stage]);
        mbar_expect_tx(fb, W_BYTES);
        tma_load_4d_hint(ring + (uint32_t)stage * stage_bytes, &tmW, 0, k * BK, tile * (BN / 64),
                         t.m.act[a], fb, once);
      }
      __syncwarp();
      issued_mask |= 1u << stage;
      issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
      if (++k == g.kb) {
        k = 0;
        if (++a == t.m.n_act) {
          a = 0;
          ++tile;
        }
      }
    }
    drain(issued_mask, issued_par);
  } else if (warp == 1) {
    // ------------------------------------------------------------ rows of act
    // a lane copies 64 k of eight of the expert's tokens (what lies behind the last one fills
    // columns that nobody reads; k behind n are zeros)
    int a = at0 / g.kb, k = at0 % g.kb, groups = 0;
    auto enter = [&]() {
      groups = (few_count(t.m.mask[t.m.act[a]]) + X_ROWS - 1) / X_ROWS;
    };
    if (work) enter();
    pdl_wait();  // act is complete
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_par = 0;
    for (int b = b0; b < b1; ++b) {
      if (!mbar_wait_warp(saddr(&t.empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) break;
      const uint32_t fb = saddr(&t.full[stage]);
      if (lane == 0) mbar_expect_tx(fb, (uint32_t)(PIECES * groups * X_ROWS * 128));
      __syncwarp();
      const int piece = lane >= groups ? 1 : 0, grp = lane - piece * groups;
      if (lane < PIECES * groups)
        tma_load_2d(ring + (uint32_t)stage * stage_bytes + W_BYTES + (uint32_t)piece * x_most +
                        (uint32_t)(grp * X_ROWS * 128),
                    &tmX, k * BK + piece * 64, a * g.T + grp * X_ROWS, fb);
      __syncwarp();
      issued_mask |= 1u << stage;
      issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
      if (++k == g.kb) {
        k = 0;
        if (++a == t.m.n_act) a = 0;
        enter();
      }
    }
    drain(issued_mask, issued_par);
  } else if (warp == 2) {
    // ------------------------------------------------------------ MMA issuer
    // D fp32, A and B bf16, A MN-major (bit 15), B K-major, M = 128, N = the expert's tokens
    const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (8u << 24);
    const uint64_t wd0 = desc_sw128(ring, BK * 128, 1024);
    const uint64_t xd0 = desc_sw128(ring + W_BYTES, 16, 1024);
    int stage = 0, it = 0, a = at0 / g.kb, k = at0 % g.kb;
    uint32_t phase = 0;
    bool ok = true;
    for (int b = b0; b < b1 && ok; ++it) {  // an expert's blocks at a time
      const int stop = min(b1, b + g.kb - k);
      const int buf = it & 1, n_tok = few_count(t.m.mask[t.m.act[a]]);
      const uint32_t idesc = idesc0 | ((uint32_t)((n_tok + 15) / 16 * 2) << 17);
      if (!mbar_wait_warp(saddr(&t.tempty[buf]), ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag,
                          g.status, limit))
        break;
      tc_fence_after();
      const uint32_t acc = tmem + ACC + (uint32_t)buf * ACC;
      for (bool first = true; b < stop; ++b, first = false) {
        if (!mbar_wait_warp(saddr(&t.full[stage]), phase, abort_flag, g.status, limit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t so = (uint64_t)(((uint32_t)stage * stage_bytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            tc_mma<1>(acc, wd0 + so + (uint64_t)(kk * 128),
                      xd0 + so + (uint64_t)(((kk >> 2) * x_most + (kk & 3) * 32) >> 4), idesc,
                      (!first || kk > 0) ? 1u : 0u);
          tc_commit<1>(saddr(&t.empty[stage]));
        }
        __syncwarp();
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok && elect_one()) tc_commit<1>(saddr(&t.tfull[buf]));
      __syncwarp();
      k = 0;
      if (++a == t.m.n_act) a = 0;
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
    const int q = warp & 3, cl = q * 32 + lane;  // TMEM lane = output column of the tile
    const uint32_t tile_at = tmem + ((uint32_t)(q * 32) << 16);
    pdl_wait();  // the previous kernel in the stream has completed (order of writes to out)
    pdl_trigger();
    int it = 0, a = at0 / g.kb, k = at0 % g.kb;
    bool fresh = true;  // the tile has no sum yet
    int tile_b = b0;
    for (int b = b0; b < b1; ++it) {
      const int stop = min(b1, b + g.kb - k);
      const int buf = it & 1, e = t.m.act[a], n_tok = few_count(t.m.mask[e]);
      const unsigned char* tok = t.tok + t.first[e];
      if (fresh) {
        for (int c = 0; c < g.T; ++c) tmem_st1(tile_at + (uint32_t)c, 0u);
        tmem_st_wait();
        fresh = false;
      }
      if (!mbar_wait_warp(saddr(&t.tfull[buf]), (uint32_t)(it >> 1) & 1u, abort_flag, g.status,
                          limit))
        break;
      tc_fence_after();
      const uint32_t acc = tile_at + ACC + (uint32_t)buf * ACC;
      for (int j0 = 0; j0 < n_tok; j0 += 8) {
        uint32_t v[8], u[8];
        tmem_ld8(acc + (uint32_t)j0, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) tmem_ld1(tile_at + tok[min(j0 + i, n_tok - 1)], u[i]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (j0 + i < n_tok)
            tmem_st1(tile_at + tok[j0 + i],
                     __float_as_uint(__uint_as_float(u[i]) + __uint_as_float(v[i])));
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(saddr(&t.tempty[buf]));
      b = stop;
      k = 0;
      if (++a == t.m.n_act) a = 0;
      if (a != 0 && b < b1) continue;
      // ---- the tile's end, or the piece's
      const int tile = (b - 1) / line, col = tile * BN + cl, tile0 = tile * line;
      const bool whole = tile_b == tile0 && b == tile0 + line;
      // partials of a cut tile: [slot][token][128]; a piece has at most two, the tile that it
      // begins in and the tile that begins in it
      float* part =
          g.part + (size_t)(2 * (int)blockIdx.x + (tile0 >= b0 ? 1 : 0)) * g.T * BN + cl;
      for (int c0 = 0; c0 < g.T; c0 += 8) {
        uint32_t v[8];
        tmem_ld8(tile_at + (uint32_t)c0, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tk = c0 + i;
          if (tk >= g.T) continue;
          if (!whole) part[(size_t)tk * BN] = __uint_as_float(v[i]);
          else if (col < g.d)
            g.out[(size_t)tk * g.d + col] = __float2bfloat16(
                t.m.bad[tk >> 5] >> (tk & 31) & 1u ? NAN : __uint_as_float(v[i]));
        }
      }
      fresh = true;
      tile_b = b;
    }
  }
  __syncwarp();  // lanes that waited alone are back: a barrier counts a split warp twice
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, TMEM_COLS);
  }
}

// The tiles that the pieces of few_down_kernel cut: their partials in the line's order, four
// columns of one token a thread. g as few_down_kernel had it, `ctas` its grid.
__global__ void __launch_bounds__(THREADS) few_sum_kernel(const FewDownArgs g, int ctas) {
  __shared__ FewMasks m;
  few_clear_masks(m, g.E, THREADS);
  few_build_masks(m, g.ids, g.T, g.K, g.E, g.cap, THREADS);  // complete before that kernel began
  const int line = m.n_act * g.kb, total = line * g.nt;
  const FewPieces cut(total, MIN_BLOCKS, ctas);
  const int i = (int)blockIdx.x * THREADS + (int)threadIdx.x;
  const int c4 = i % (BN / 4) * 4, tok = i / (BN / 4) % g.T, tile = i / (BN / 4) / g.T;
  const int col = tile * BN + c4;
  const int tile0 = tile * line, p0 = total > 0 && tile < g.nt ? cut.of(tile0) : 0;
  const int p1 = total > 0 && tile < g.nt ? cut.of(tile0 + line - 1) : 0;
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();
  if (tile >= g.nt || col >= g.d) return;
  float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
  if (total > 0) {
    if (p0 == p1) return;  // one piece held all of it and wrote it
#pragma unroll 8
    for (int p = p0; p <= p1; ++p) {
      const int s = 2 * p + (tile0 >= cut.begin(p) ? 1 : 0);
      const float4 v =
          __ldcg(reinterpret_cast<const float4*>(g.part + ((size_t)s * g.T + tok) * BN + c4));
      f.x += v.x; f.y += v.y; f.z += v.z; f.w += v.w;
    }
  }
  if (m.bad[tok >> 5] >> (tok & 31) & 1u)  // NaN logits: no expert, and the row is NaN
    f = make_float4(NAN, NAN, NAN, NAN);
  *reinterpret_cast<uint2*>(g.out + (size_t)tok * g.d + col) =
      make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
}

}  // namespace

size_t few_down_part_bytes(int T) { return (size_t)2 * sm_count() * T * BN * 4; }

// act: [active experts][T][n]
moe_status launch_few_down(FewDownArgs a, const void* w_down, cudaStream_t st) {
  a.kb = (a.n + BK - 1) / BK;
  a.nt = (a.d + BN - 1) / BN;
  const int fixed = 1024 + (int)sizeof(Tail);
  a.ring_bytes = (SMEM_LIMIT - fixed) / 1024 * 1024;
  a.status = device_status_ptr();
  a.limit_ns = kWaitLimitNs;
  CUtensorMap mw, mx;
  const uint64_t xd[2] = {(uint64_t)a.n, (uint64_t)a.rows}, xs[1] = {(uint64_t)a.n * 2};
  const uint32_t xbox[2] = {64, X_ROWS};
  if (!make_piece_map(&mw, w_down, a.n, a.d, a.E, BK, BN / 64) ||
      !make_map(&mx, a.act, 2, xd, xs, xbox, false))
    return MOE_ERR_CUDA;
  if (cudaFuncSetAttribute(few_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           SMEM_LIMIT) != cudaSuccess)
    return MOE_ERR_CUDA;
  const int ctas = sm_count();
  launch_begin(K_FEW_DOWN, st);
  launch_kernel(few_down_kernel, dim3((unsigned)ctas), dim3(THREADS),
                (size_t)(fixed + a.ring_bytes), st, 1, mw, mx, a);
  const moe_status r = launch_end(K_FEW_DOWN, st);
  if (r != MOE_OK) return r;
  launch_begin(K_FEW_SUM, st);
  launch_kernel(few_sum_kernel, dim3((unsigned)((a.nt * (BN / 4) * a.T + THREADS - 1) / THREADS)),
                dim3(THREADS), 0, st, 1, a, ctas);
  return launch_end(K_FEW_SUM, st);
}

}  // namespace moe
