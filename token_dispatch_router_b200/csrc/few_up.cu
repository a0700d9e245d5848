// First expert product of the few-token layer: for each expert e that keeps a token,
//   act[a, j] = w[t, e] silu(x_t W_gate[e]) * (x_t W_up[e])      (a: e's place among them)
// for its tokens t (t its j-th one), at most 128 of them. w is the routing weight: the second
// product then only adds up. Everything is fp32 up to act, which is rounded to bf16, the type that
// the second product's MMA takes (at most 2^-8 of each value; the layer's output is 2.3e-3 from the
// exact one in the mean, 1.7e-3 of which its own rounding alone makes). Two bf16 terms of act would
// take that away, for twice the second product's rows and MMAs; moe_forward rounds here, too.
//
// Bound by reading W_gate and W_up of those experts. They are the MMA's A operand, 128 columns
// of each on M (MN-major: a box goes by TMA from where it lies into shared memory and into the
// tensor cores), the expert's tokens its N, rounded up to 16: no padding of tokens to 128 rows.
// Their rows of x are gathered by TMA, four a copy. (With all 128 tokens on N for every expert a
// stage is half as large again and L2 becomes the bound: 128 tokens, 8 experts of 14336, width
// 4096: 344 us.) Columns do not mix, so a NaN of one token stays with it.
//
// The k-blocks of all (expert, 128-column tile) pairs form one line, cut into equal pieces, one
// per SM: every SM reads the same number of bytes whatever the number of experts and tiles. A
// tile cut by a piece's end leaves fp32 partials, which the last of its SMs to finish adds in
// the line's order (nobody waits; results repeat bit for bit).
// Roles (256 threads): warp 0 copies the weights, warp 2 the rows of x (a copy takes its warp
// about 60 cycles to issue, a finished wait 200: one warp for both was the bound), warp 1 issues
// the MMAs (two accumulators, double-buffered), warps 4-7 read them (lane = weight column, column
// = token). Every wait (but tmem_alloc's) is bounded; on expiry the status word records
// MOE_ERR_TIMEOUT and the CTA ends after its copies and MMAs in flight.
#include <type_traits>

#include "few.cuh"
#include "few_args.cuh"
#include "ffn_args.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int THREADS = 256;
constexpr int BK = 64;
constexpr int W_CHUNK = 8192;         // 64 k-rows x 64 columns
constexpr int W_BYTES = 4 * W_CHUNK;  // 128 columns of W_gate and of W_up
constexpr int X_BOX = 512;            // four tokens x 64 k
constexpr int MAX_STAGES = 6;
constexpr int MIN_BLOCKS = 4;         // k-blocks of a piece, at least
constexpr int SMEM_LIMIT = 227 * 1024;

struct Tail {
  uint64_t full[MAX_STAGES], full_x[MAX_STAGES], empty[MAX_STAGES], tfull[2], tempty[2], done;
  uint32_t tmem;
  int abort, epi_ok, last;
  FewMasks m;
  float w[kFewMaxTokens];  // the tile's expert: the routing weights of its tokens, ascending
};

// The j-th token of a mask (j below its count).
__device__ __forceinline__ int token_at(const unsigned (&m)[4], int j) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int c = __popc(m[w]);
    if (j < c) {
      unsigned b = m[w];
      for (int i = 0; i < j; ++i) b &= b - 1;
      return 32 * w + __ffs(b) - 1;
    }
    j -= c;
  }
  return 0;
}
__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fdividef(g, 1.f + __expf(-g)) * u;
}

__global__ void __launch_bounds__(THREADS, 1)
    few_up_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmG,
                  const __grid_constant__ CUtensorMap tmU, const FewUpArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Tail& t = *reinterpret_cast<Tail*>(base + g.stages * g.stage_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &t.abort;
  const uint32_t tcols = tmem_columns(4 * g.npad);

  if (tid == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(saddr(&t.full[s]), 1);
      mbar_init(saddr(&t.full_x[s]), 1);
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
  if (warp == 1) tmem_alloc<1>(saddr(&t.tmem), tcols);
  if (tid == 64) {
    prefetch_map(&tmX);
    prefetch_map(&tmG);
    prefetch_map(&tmU);
  }
  tc_fence_before();
  few_clear_masks(t.m, g.E, THREADS);  // a barrier for the whole block
  tc_fence_after();
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();
  few_build_masks(t.m, g.ids, g.T, g.K, g.E, g.cap, THREADS);
  const uint32_t tmem = t.tmem;
  const uint64_t limit = g.limit_ns;
  const int total = t.m.n_act * g.nt * g.kblocks;
  const FewPieces cut(total, MIN_BLOCKS, (int)gridDim.x);
  const bool work = (int)blockIdx.x < cut.n && total > 0;
  const int b0 = work ? cut.begin(blockIdx.x) : 0, b1 = work ? cut.begin(blockIdx.x + 1) : 0;

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ loads
    // warp 0: a copy each of W_gate and W_up; warp 2: lane i four of the expert's tokens
    const bool x_warp = warp == 2;
    const uint64_t once = l2_policy_evict_first();  // weights are read once: x and act stay in L2
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_par = 0;
    int k = b0 % g.kblocks, ct = b0 / g.kblocks % g.nt;
    int a = b0 / g.kblocks / g.nt, e = 0, quads = 0;
    int row[4] = {0, 0, 0, 0};
    auto enter = [&]() {  // the rows behind the last token repeat the first one
      e = t.m.act[a];
      const int n = few_count(t.m.mask[e]);
      quads = (n + 15) / 16 * 4;
      if (x_warp)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          row[i] = token_at(t.m.mask[e], 4 * lane + i < n ? 4 * lane + i : 0);
    };
    if (work) enter();
    for (int b = b0; b < b1; ++b) {
      if (!mbar_wait_warp(saddr(&t.empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) break;
      const uint32_t fb = saddr(x_warp ? &t.full_x[stage] : &t.full[stage]);
      const uint32_t w = saddr(base + stage * g.stage_bytes);
      if (x_warp) {
        if (lane == 0) mbar_expect_tx(fb, (uint32_t)(quads * X_BOX));
        __syncwarp();
        if (lane < quads) tma_gather4(w + W_BYTES + lane * X_BOX, &tmX, k * BK, row, fb);
      } else if (elect_one()) {
        mbar_expect_tx(fb, W_BYTES);
        tma_load_4d_hint(w, &tmG, 0, k * BK, ct * 2, e, fb, once);
        tma_load_4d_hint(w + 2 * W_CHUNK, &tmU, 0, k * BK, ct * 2, e, fb, once);
      }
      __syncwarp();
      issued_mask |= 1u << stage;
      issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
      if (++stage == g.stages) {
        stage = 0;
        phase ^= 1u;
      }
      if (++k == g.kblocks) {
        k = 0;
        if (++ct == g.nt) {
          ct = 0;
          if (++a < t.m.n_act) enter();
        }
      }
    }
    if (lane == 0)
      for (int s = 0; s < g.stages; ++s) {  // nothing of ours is in flight after this (bounded)
        if (!(issued_mask & (1u << s))) continue;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try(saddr(x_warp ? &t.full_x[s] : &t.full[s]), (issued_par >> s) & 1u) &&
               globaltimer_ns() - t0 < limit) {
        }
      }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // D fp32, A and B bf16, A MN-major (bit 15), B K-major, M = 128, N = the expert's tokens
    const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (8u << 24);
    // descriptors of stage 0; a stage or a k step moves the address field (byte address / 16)
    const uint64_t wd0 = desc_sw128(saddr(base), W_CHUNK, 1024);
    const uint64_t xd0 = desc_sw128(saddr(base) + W_BYTES, 16, 1024);
    int stage = 0, it = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int b = b0; b < b1 && ok; ++it) {
      const int stop = min(b1, (b / g.kblocks + 1) * g.kblocks);
      const int n_tok = few_count(t.m.mask[t.m.act[b / g.kblocks / g.nt]]);
      const uint32_t idesc = idesc0 | ((uint32_t)((n_tok + 15) / 16 * 2) << 17);
      const int buf = it & 1;
      if (!mbar_wait_warp(saddr(&t.tempty[buf]), ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag,
                          g.status, limit))
        break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(buf * 2 * g.npad);
      for (bool first = true; b < stop; ++b, first = false) {
        if (!mbar_wait_warp(saddr(&t.full[stage]), phase, abort_flag, g.status, limit) ||
            !mbar_wait_warp(saddr(&t.full_x[stage]), phase, abort_flag, g.status, limit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t so = (uint64_t)((stage * g.stage_bytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
#pragma unroll
            for (int m = 0; m < 2; ++m)
              tc_mma<1>(acc + (uint32_t)(m * g.npad),
                        wd0 + so + (uint64_t)((m * 2 * W_CHUNK + kk * 2048) >> 4),
                        xd0 + so + (uint64_t)(kk * 2), idesc, (!first || kk > 0) ? 1u : 0u);
          tc_commit<1>(saddr(&t.empty[stage]));
        }
        __syncwarp();
        if (++stage == g.stages) {
          stage = 0;
          phase ^= 1u;
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
    const int et = tid - 128, q = warp & 3;  // TMEM lanes 32 q ...
    const bool first = et == 0;
    const int cl = q * 32 + lane;
    int it = 0, last_e = -1;
    for (int b = b0; b < b1; ++it) {
      const int tile = b / g.kblocks;
      const int tile0 = tile * g.kblocks, tile1 = tile0 + g.kblocks, stop = min(b1, tile1);
      const bool whole = b == tile0 && stop == tile1;
      const int a = tile / g.nt, e = t.m.act[a], ct = tile % g.nt;
      const int buf = it & 1;
      if (e != last_e) {  // the weights of this expert's tokens
        last_e = e;
        epi_bar();  // everyone is done with those of the expert before
        const unsigned(&m)[4] = t.m.mask[e];
        if (et < g.T && (m[et >> 5] >> (et & 31) & 1u)) {
          int j = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            j += __popc(i < (et >> 5) ? m[i] : i == (et >> 5) ? m[i] & ((1u << (et & 31)) - 1u) : 0u);
          for (int k = 0; k < g.K; ++k)
            if (g.ids[et * g.K + k] == e) t.w[j] = g.topk_w[et * g.K + k];
        }
      }
      if (first)
        t.epi_ok = mbar_wait(saddr(&t.tfull[buf]), (uint32_t)(it >> 1) & 1u, abort_flag, g.status,
                             limit) ? 1 : 0;
      epi_bar();
      const bool ok = t.epi_ok != 0;
      epi_bar();  // everyone has read epi_ok
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(buf * 2 * g.npad) + ((uint32_t)(q * 32) << 16);
      const int col = ct * 128 + cl;
      const bool col_ok = col < g.n;
      bf16* act = g.act + (size_t)a * g.T * g.n + col;
      // partials of a cut tile: [slot][token of the expert][gate 128 | up 128]; a piece has at
      // most two, the tile that it begins in and the tile that begins in it
      const int slot = 2 * (int)blockIdx.x + (tile0 >= b0 ? 1 : 0);
      float* part = g.part + (size_t)slot * g.T * 256 + cl;
      const int n_tok = few_count(t.m.mask[e]);
      for (int j0 = 0; j0 < n_tok; j0 += 8) {
        uint32_t gv[8], uv[8];
        tmem_ld8(acc + (uint32_t)j0, gv);
        tmem_ld8(acc + (uint32_t)(g.npad + j0), uv);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int j = j0 + i;
          if (j >= n_tok) continue;
          const float gf = __uint_as_float(gv[i]), uf = __uint_as_float(uv[i]);
          if (whole) {
            if (col_ok) act[(size_t)j * g.n] = __float2bfloat16(t.w[j] * silu_mul(gf, uf));
          } else {
            part[(size_t)j * 256] = gf;
            part[(size_t)j * 256 + 128] = uf;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(saddr(&t.tempty[buf]));
      if (!whole) {
        const int p0 = cut.of(tile0), p1 = cut.of(tile1 - 1);
        __threadfence();
        epi_bar();
        if (first) t.last = atomicAdd(g.arrived + p0, 1u) == (unsigned)(p1 - p0);
        epi_bar();
        if (t.last) {
          __threadfence();
          // 16 partials of a column at a time, so that their loads are in flight together: of
          // eight tokens, or of the tile's pieces where there are few tokens
          auto join = [&](auto tokens, auto pieces) {
            constexpr int NT = decltype(tokens)::value, NP = decltype(pieces)::value;
            for (int j0 = 0; j0 < n_tok; j0 += NT) {
              float gf[NT], uf[NT];
#pragma unroll
              for (int i = 0; i < NT; ++i) gf[i] = uf[i] = 0.f;
              for (int p = p0; p <= p1; p += NP) {
                float gv[NP][NT], uv[NP][NT];
#pragma unroll
                for (int z = 0; z < NP; ++z) {
                  const int s = 2 * (p + z) + (tile0 >= cut.begin(p + z) ? 1 : 0);
                  const float* pp = g.part + ((size_t)s * g.T + j0) * 256 + cl;
#pragma unroll
                  for (int i = 0; i < NT; ++i) {
                    const bool on = p + z <= p1 && j0 + i < n_tok;
                    gv[z][i] = on ? __ldcg(pp + i * 256) : 0.f;
                    uv[z][i] = on ? __ldcg(pp + i * 256 + 128) : 0.f;
                  }
                }
#pragma unroll
                for (int z = 0; z < NP; ++z)
#pragma unroll
                  for (int i = 0; i < NT; ++i) {
                    gf[i] += gv[z][i];
                    uf[i] += uv[z][i];
                  }
              }
#pragma unroll
              for (int i = 0; i < NT; ++i)
                if (j0 + i < n_tok && col_ok)
                  act[(size_t)(j0 + i) * g.n] =
                      __float2bfloat16(t.w[j0 + i] * silu_mul(gf[i], uf[i]));
            }
          };
          using std::integral_constant;
          if (n_tok <= 2) join(integral_constant<int, 2>{}, integral_constant<int, 8>{});
          else join(integral_constant<int, 8>{}, integral_constant<int, 2>{});
        }
      }
      b = stop;
    }
  }
  __syncwarp();  // lanes that waited alone are back: a barrier counts a split warp twice
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, tcols);
  }
}

}  // namespace

int few_up_pieces() { return sm_count(); }
size_t few_up_part_bytes(int T) { return (size_t)2 * few_up_pieces() * T * 256 * 4; }

moe_status launch_few_up(FewUpArgs a, int d, int n_experts, const void* x, const void* w_gate,
                         const void* w_up, cudaStream_t st) {
  a.kblocks = d / BK;
  a.nt = (a.n + 127) / 128;
  a.npad = (a.T + 15) / 16 * 16;
  a.stage_bytes = W_BYTES + a.npad * 128;
  a.stages = (SMEM_LIMIT - 1024 - (int)sizeof(Tail)) / a.stage_bytes;
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  a.status = device_status_ptr();
  a.limit_ns = kWaitLimitNs;
  CUtensorMap mx, mg, mu;
  const uint64_t xd[2] = {(uint64_t)d, (uint64_t)a.T}, xs[1] = {(uint64_t)d * 2};
  const uint32_t xbox[2] = {64, 1};
  if (!make_map(&mx, x, 2, xd, xs, xbox) || !make_piece_map(&mg, w_gate, d, a.n, n_experts, BK, 2) ||
      !make_piece_map(&mu, w_up, d, a.n, n_experts, BK, 2))
    return MOE_ERR_CUDA;
  if (cudaFuncSetAttribute(few_up_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           SMEM_LIMIT) != cudaSuccess)
    return MOE_ERR_CUDA;
  const int smem = 1024 + a.stages * a.stage_bytes + (int)sizeof(Tail);
  launch_begin(K_FEW_UP, st);
  launch_kernel(few_up_kernel, dim3((unsigned)few_up_pieces()), dim3(THREADS), (size_t)smem, st, 1,
                mx, mg, mu, a);
  return launch_end(K_FEW_UP, st);
}

}  // namespace moe
