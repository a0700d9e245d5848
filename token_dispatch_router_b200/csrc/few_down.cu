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
// SM. A tile cut by a piece's end leaves fp32 partials that a small kernel behind this one adds in
// the line's order (results repeat bit for bit). Its CTAs wait beside the running ones and all
// SMs take part; the last SM to finish a tile adding them up alone took 40 us of 230 (128 tokens,
// width 4096, 8 experts of 14336), and clusters that split a tile and add through distributed
// shared memory find no room for all of them while the kernel before drains.
// The weights do not depend on the kernel before this one: a CTA fills its ring with them before
// it waits for that kernel (its launch follows that kernel's own wait, so everything older, the
// ids among it, is complete).
// Roles (256 threads): warp 0 copies weights by TMA, warps 1 and 3 the expert's rows of act by
// cp.async, each to its token's lane, warp 2 issues the MMAs (two accumulators, so that one is
// read while the next is made), warps 4-7 read them. A finished wait costs a warp about 200
// cycles and a copy or an MMA 60 to issue, so a stage is 128 k of 128 columns, 32 KB brought by
// one copy and taken by eight MMAs. Rows come from L2 and have a short ring of their own, which
// leaves most of the shared memory to weights in flight.
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
constexpr int GATHER = 64;     // threads that copy rows
constexpr int W_STAGES = 6, X_STAGES = 4;  // at most
constexpr int MIN_BLOCKS = 2;  // stages of a piece, at least
constexpr int SMEM_LIMIT = 227 * 1024;
// A stage of rows is, for each 64 k, T rounded up to 8 rows of 128 bytes. The MMA reads 128 rows:
// past T it runs on into what lies behind, at most the weights' ring, and those lanes are masked.

struct Tail {
  uint64_t full[W_STAGES], empty[W_STAGES], full_x[X_STAGES], empty_x[X_STAGES], tfull[2],
      tempty[2], done;
  uint32_t tmem;
  int abort, epi_ok;
  FewMasks m;
  // every expert's tokens, ascending: expert e's from first[e]
  short first[kFewMaxExperts];
  unsigned char tok[kFewMaxTokens * 32];
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
// BN columns of 32 lanes set to zero.
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
__device__ __forceinline__ void store8(const FewDownArgs& g, const FewMasks& m, int tok, int col,
                                       float (&f)[8]) {
  if (m.bad[tok >> 5] >> (tok & 31) & 1u)  // NaN logits: no expert, and the row is NaN
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = NAN;
  *reinterpret_cast<uint4*>(g.out + (size_t)tok * g.d + col) = pack16(f, bf16());
}

__global__ void __launch_bounds__(THREADS, 1)
    few_down_kernel(const __grid_constant__ CUtensorMap tmW, const FewDownArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Tail& t = *reinterpret_cast<Tail*>(base + g.ring_bytes);  // behind rows and weights
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &t.abort;
  if (tid == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(saddr(&t.full[s]), 1);
      mbar_init(saddr(&t.empty[s]), 1);
    }
    for (int s = 0; s < g.x_stages; ++s) {
      mbar_init(saddr(&t.full_x[s]), GATHER);
      mbar_init(saddr(&t.empty_x[s]), 1);
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
  const uint32_t x_piece = (uint32_t)(g.T + 7) / 8u * 1024u, x_bytes = PIECES * x_piece;
  const uint32_t x_ring = saddr(base), w_ring = x_ring + (uint32_t)g.x_stages * x_bytes;
  const int line = t.m.n_act * g.kb;
  const long long total = (long long)line * g.nt;
  const int pieces = few_pieces(total, MIN_BLOCKS, (int)gridDim.x);
  const bool work = (int)blockIdx.x < pieces && total > 0;
  const long long b0 = work ? few_piece_begin(blockIdx.x, total, pieces) : 0;
  const long long b1 = work ? few_piece_begin(blockIdx.x + 1, total, pieces) : 0;
  const int at0 = line > 0 ? (int)(b0 % line) : 0;  // of the first block, in its tile's line

  if (warp == 0) {
    // ------------------------------------------------------------ weights
    int tile = line > 0 ? (int)(b0 / line) : 0, a = at0 / g.kb, k = at0 % g.kb, stage = 0;
    uint32_t phase = 0;
    const uint64_t once = l2_policy_evict_first();  // read once: act stays in L2
    for (long long b = b0; b < b1; ++b) {
      if (!mbar_wait_warp(saddr(&t.empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) break;
      if (elect_one()) {
        const uint32_t fb = saddr(&t.full[stage]);
        mbar_expect_tx(fb, W_BYTES);
        tma_load_4d_hint(w_ring + (uint32_t)(stage * W_BYTES), &tmW, 0, k * BK, tile * (BN / 64),
                         t.m.act[a], fb, once);
      }
      __syncwarp();
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
      }
    }
    if (lane == 0 && *abort_flag) {
      // a wait ran out: give the copies in flight time to land (else the MMAs have read them)
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000) {
      }
    }
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ rows of act
    // a thread copies one 16-byte piece of a row of the stage, for every fourth of the tokens
    constexpr int ROW_PIECES = BK / 8;
    const int gt = lane + (warp == 3 ? 32 : 0), piece = gt % ROW_PIECES;
    int a = at0 / g.kb, k = at0 % g.kb, e = 0, n_tok = 0;
    auto enter = [&]() {
      e = t.m.act[a];
      n_tok = few_count(t.m.mask[e]);
    };
    if (work) enter();
    pdl_wait();  // act is complete
    int stage = 0;
    uint32_t phase = 0;
    for (long long b = b0; b < b1; ++b) {
      if (!mbar_wait_warp(saddr(&t.empty_x[stage]), phase ^ 1u, abort_flag, g.status, limit)) break;
      const uint32_t x = x_ring + (uint32_t)stage * x_bytes + (uint32_t)(piece >> 3) * x_piece;
      const int col = k * BK + piece * 8;
      const bf16* src = g.act + (size_t)a * g.T * g.n + (col < g.n ? col : 0);
      const unsigned char* tok = t.tok + t.first[e];
      for (int j = gt / ROW_PIECES; j < n_tok; j += GATHER / ROW_PIECES) {
        const int r = tok[j];
        cp_async16_if(x + (uint32_t)(r * 128 + (((piece & 7) ^ (r & 7)) << 4)),
                      src + (size_t)r * g.n, col < g.n);
      }
      cp_async_arrive_noinc(saddr(&t.full_x[stage]));
      if (++stage == g.x_stages) {
        stage = 0;
        phase ^= 1u;
      }
      if (++k == g.kb) {
        k = 0;
        if (++a == t.m.n_act) a = 0;
        enter();
      }
    }
    cp_async_wait_all();
  } else if (warp == 2) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = idesc_bf16(128, BN);  // A (tokens) K-major, B (weights) MN-major
    const uint64_t xd0 = desc_sw128(x_ring, 16, 1024), wd0 = desc_sw128(w_ring, BK * 128, 1024);
    int stage = 0, xs = 0, it = 0, a = at0 / g.kb, k = at0 % g.kb;
    uint32_t phase = 0, xphase = 0;
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
        if (!mbar_wait_warp(saddr(&t.full_x[xs]), xphase, abort_flag, g.status, limit) ||
            !mbar_wait_warp(saddr(&t.full[stage]), phase, abort_flag, g.status, limit)) {
          ok = false;
          break;
        }
        fence_proxy_async_smem();  // the rows (cp.async) -> MMA reads
        tc_fence_after();
        if (elect_one()) {
          uint64_t xd = xd0 + (uint64_t)((xs * x_bytes) >> 4);
          uint64_t wd = wd0 + (uint64_t)((stage * W_BYTES) >> 4);
#pragma unroll 1
          for (int p = 0; p < PIECES; ++p, xd += x_piece >> 4, wd += 4 * 128)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_lanes(tmem + (uint32_t)(buf * BN), xd + (uint64_t)(kk * 2),
                        wd + (uint64_t)(kk * 128), idesc, off);
          tc_commit<1>(saddr(&t.empty[stage]));
          tc_commit<1>(saddr(&t.empty_x[xs]));
        }
        __syncwarp();
        if (++stage == g.stages) {
          stage = 0;
          phase ^= 1u;
        }
        if (++xs == g.x_stages) {
          xs = 0;
          xphase ^= 1u;
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
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, row = q * 32 + lane;  // TMEM lane = token
    const bool rows_here = q * 32 < g.T, row_ok = row < g.T;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    for (int b = 0; b < 2; ++b) {  // accumulators start at zero: MMAs under a mask only add
      tmem_zero(tmem + (uint32_t)(b * BN) + lanes);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(saddr(&t.tempty[b]));
    }
    pdl_wait();  // the previous kernel in the stream has completed (order of writes to out)
    pdl_trigger();
    int it = 0;
    for (long long b = b0; b < b1; ++it) {
      const int tile = (int)(b / line), buf = it & 1, n0 = tile * BN;
      const long long tile0 = (long long)tile * line, stop = min(b1, tile0 + line);
      const bool whole = b == tile0 && stop == tile0 + line;
      if (!mbar_wait_warp(saddr(&t.tfull[buf]), (uint32_t)(it >> 1) & 1u, abort_flag, g.status,
                          limit))
        break;
      tc_fence_after();
      if (rows_here) {
        const uint32_t acc = tmem + (uint32_t)(buf * BN) + lanes;
        // partials of a cut tile: [slot][4 columns][token][4]; a piece has at most two, the tile
        // that it begins in and the tile that begins in it
        const int slot = 2 * (int)blockIdx.x + (tile0 >= b0 ? 1 : 0);
        float4* part = reinterpret_cast<float4*>(g.part) + (size_t)slot * (BN / 4) * g.T + row;
#pragma unroll 2
        for (int c = 0; c < BN; c += 8) {
          uint32_t v[8];
          tmem_ld8(acc + (uint32_t)c, v);
          tmem_ld_wait();
          if (!row_ok) continue;
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(v[j]);
          if (!whole) {
            part[(size_t)(c / 4) * g.T] = make_float4(f[0], f[1], f[2], f[3]);
            part[(size_t)(c / 4 + 1) * g.T] = make_float4(f[4], f[5], f[6], f[7]);
          } else if (n0 + c < g.d) {
            store8(g, t.m, row, n0 + c, f);
          }
        }
        tmem_zero(acc);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(saddr(&t.tempty[buf]));
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

// The tiles that the pieces of few_down_kernel cut: their partials in the line's order, eight
// columns of one token a thread. g as few_down_kernel had it, `ctas` its grid.
__global__ void __launch_bounds__(THREADS) few_sum_kernel(const FewDownArgs g, int ctas) {
  __shared__ FewMasks m;
  few_build_masks(m, g.ids, g.T, g.K, g.E, g.cap, THREADS);  // complete before that kernel began
  const int line = m.n_act * g.kb;
  const long long total = (long long)line * g.nt;
  const int pieces = few_pieces(total, MIN_BLOCKS, ctas);
  const int i = (int)blockIdx.x * THREADS + (int)threadIdx.x;
  const int tok = i % g.T, c8 = i / g.T % (BN / 8), tile = i / g.T / (BN / 8);
  const int col = tile * BN + c8 * 8;
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();
  if (tile >= g.nt || col >= g.d) return;
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (total > 0) {
    const long long tile0 = (long long)tile * line;
    const int p0 = few_piece_of(tile0, total, pieces);
    const int p1 = few_piece_of(tile0 + line - 1, total, pieces);
    if (p0 == p1 && few_piece_begin(p0, total, pieces) <= tile0 &&
        few_piece_begin(p0 + 1, total, pieces) >= tile0 + line)
      return;  // written whole
#pragma unroll 4
    for (int p = p0; p <= p1; ++p) {
      const int s = 2 * p + (tile0 >= few_piece_begin(p, total, pieces) ? 1 : 0);
      const float4* pp =
          reinterpret_cast<const float4*>(g.part) + ((size_t)s * (BN / 4) + 2 * c8) * g.T + tok;
      const float4 u = __ldcg(pp), v = __ldcg(pp + g.T);
      f[0] += u.x; f[1] += u.y; f[2] += u.z; f[3] += u.w;
      f[4] += v.x; f[5] += v.y; f[6] += v.z; f[7] += v.w;
    }
  }
  store8(g, m, tok, col, f);
}

}  // namespace

size_t few_down_part_bytes(int T) { return (size_t)2 * sm_count() * T * BN * 4; }

// act: [active experts][T][n]
moe_status launch_few_down(FewDownArgs a, const void* w_down, cudaStream_t st) {
  a.kb = (a.n + BK - 1) / BK;
  a.nt = (a.d + BN - 1) / BN;
  const int fixed = 1024 + (int)sizeof(Tail), x_bytes = PIECES * ((a.T + 7) / 8 * 1024);
  a.x_stages = a.T > 64 ? 2 : a.T > 32 ? 3 : X_STAGES;
  a.stages = (SMEM_LIMIT - fixed - a.x_stages * x_bytes) / W_BYTES;
  if (a.stages > W_STAGES) a.stages = W_STAGES;
  a.ring_bytes = a.stages * W_BYTES + a.x_stages * x_bytes;
  a.status = device_status_ptr();
  a.limit_ns = kWaitLimitNs;
  CUtensorMap mw;
  if (!make_piece_map(&mw, w_down, a.n, a.d, a.E, BK, BN / 64)) return MOE_ERR_CUDA;
  if (cudaFuncSetAttribute(few_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           SMEM_LIMIT) != cudaSuccess)
    return MOE_ERR_CUDA;
  const int ctas = sm_count();
  launch_begin(K_FEW_DOWN, st);
  launch_kernel(few_down_kernel, dim3((unsigned)ctas), dim3(THREADS),
                (size_t)(fixed + a.ring_bytes), st, 1, mw, a);
  const moe_status r = launch_end(K_FEW_DOWN, st);
  if (r != MOE_OK) return r;
  launch_begin(K_FEW_SUM, st);
  launch_kernel(few_sum_kernel, dim3((unsigned)((a.nt * (BN / 8) * a.T + THREADS - 1) / THREADS)),
                dim3(THREADS), 0, st, 1, a, ctas);
  return launch_end(K_FEW_SUM, st);
}

}  // namespace moe
