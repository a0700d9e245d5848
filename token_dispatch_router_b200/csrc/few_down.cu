// Second product for a few tokens, at most 128 (M, one lane each):
//   layer:       out[t] = sum over the experts e that keep t of  act[a(e), t] W_down[e]
//                (act carries the routing weight: few_up.cu)
//   projection:  out[t] = x_t W + scale_l (x_t A_l) B_l,  l = ids[t]
//
// Bound by reading the weights. The layer's experts are one long contraction, k-blocks of all
// active experts in a line, accumulated in one place: no per-expert outputs and no combine.
// The MMA's lane mask (disable-output-lane) adds each expert's k-blocks to its own tokens only:
// the other rows of act are never written, nor read into a result, and an infinity or NaN in
// an expert that a token does not use cannot reach it.
//
// An output tile of 64 or 128 columns belongs to a cluster of up to four CTAs that split the line
// into equal parts; the partial tiles are added in rank order through distributed shared memory
// (results repeat bit for bit), each rank a share of the tokens. So there are enough CTAs to
// fill the GPU, all resident at once, with no scratch in global memory and no waiting on
// anything but the cluster.
// The weights do not depend on the kernel before this one: every CTA fills its ring with them
// before it waits for that kernel (its launch follows that kernel's own wait, so everything
// older is complete), which hides the kernel boundary: for one token most of the matrix is in
// shared memory by then.
// Roles (256 threads): a k-block is small (8 or 16 KB of weights), and a warp takes 500 to 650
// cycles to wait for it and issue its copies, or its MMAs, whatever its size. So two warps load
// and two issue MMAs, alternate k-blocks each, into an accumulator a warp (64 tokens, 128
// experts of 768, width 2048: 141 us with one of each, 97 with two); four warps read them.
// Every wait is bounded (MOE_ERR_TIMEOUT on expiry).
#include <math.h>

#include "few.cuh"
#include "few_args.cuh"
#include "ffn_args.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int THREADS = 256;
constexpr int BK = 64;
constexpr int W_CHUNK = 8192;
constexpr int ROW_BOX = 8;                       // rows of an act / x box
// A stage is the rows (T rounded up to 8, 128 bytes each), then the weights. The MMA reads 128
// rows: past T it runs into the stage's own weights, and those lanes are masked.
constexpr int MAX_STAGES = 10;
constexpr int SMEM_ONE = 200 * 1024, SMEM_TWO = 108 * 1024;  // one or two CTAs on an SM

struct Tail {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES], done;
  uint32_t tmem;
  int abort;
  int issued[MAX_STAGES];  // 1 + parity of the last copies issued into a stage
  FewMasks m;
  float low[8][128];  // projection: the low-rank values of the rows in hand
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
__device__ __forceinline__ float4 ld_dsmem_v4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

// BN: columns of an output tile, 64 or 128.
template <bool PROJ, int BN>
__global__ void __launch_bounds__(THREADS, 2)
    few_down_kernel(const __grid_constant__ CUtensorMap tmA,
                    const __grid_constant__ CUtensorMap tmAll,
                    const __grid_constant__ CUtensorMap tmW, const FewDownArgs g) {
  constexpr int W_BYTES = BN / 64 * W_CHUNK;
  constexpr int PITCH = BN + 4;     // floats per row of the partial tile
  constexpr int LANES = BN / 4;     // lanes on a row of it, four columns each
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Tail& t = *reinterpret_cast<Tail*>(base + g.ring_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &t.abort;
  const int S = g.split, rank = S > 1 ? (int)cluster_rank() : 0;
  const int tile = (int)blockIdx.x / S, n0 = tile * BN;

  if (tid == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(saddr(&t.full[s]), 1);
      mbar_init(saddr(&t.empty[s]), 1);
    }
    mbar_init(saddr(&t.done), 2);  // the MMA warps
    t.abort = 0;
    for (int s = 0; s < g.stages; ++s) t.issued[s] = 0;
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc<1>(saddr(&t.tmem), 2 * BN);
  if (PROJ) {
    if (tid < 4) {
      const int n = g.T - 32 * tid;
      t.m.mask[0][tid] = n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1u : 0u;
    }
    if (tid == 0) {
      t.m.n_act = 1;
      t.m.act[0] = 0;
    }
  } else {
    // ids: written by the kernel before the previous one, which is complete
    few_build_masks(t.m, g.ids, g.T, g.K, g.E, g.cap, THREADS);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = t.tmem;
  if (warp >= 4) {  // the accumulators start at zero: masked lanes are added to, never set
    const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll 1
    for (int c = 0; c < 2 * BN; c += 8)
      asm volatile(
          "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %1, %1, %1, %1, %1, %1, %1};" ::"r"(
              at + (uint32_t)c),
          "r"(0u)
          : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint64_t limit = g.limit_ns;
  const uint32_t x_bytes = (uint32_t)(g.T + 7) / 8u * 1024u;
  const int total = t.m.n_act * g.kb;
  const int b0 = (int)((long long)rank * total / S), b1 = (int)((long long)(rank + 1) * total / S);

  if (warp < 2) {
    // ------------------------------------------------------------ loads
    // Warp w copies blocks b0 + w, b0 + w + 2, ... (stages of its parity: the ring is even): lane
    // i < 16 the rows of tokens 8 i ... (or lane 0 all rows in one box), lanes 16 ... the weights,
    // side by side.
    const int row_groups = (g.T + 7) / 8;
    int a = 0, k = 0, e = 0;
    bool mine = false, all = false;  // this lane's group holds a token of the expert; one box
    uint32_t tx = 0;
    auto enter = [&](int active) {
      e = t.m.act[active];
      mine = lane < 16 && (t.m.mask[e][lane >> 2] >> (8 * (lane & 3)) & 0xffu) != 0;
      const int n = __popc(__ballot_sync(0xffffffffu, mine));
      all = 2 * n >= row_groups;
      if (all) mine = lane == 0;
      tx = W_BYTES + (all ? x_bytes : (uint32_t)n * (ROW_BOX * 128));
    };
    auto seek = [&](int b) {  // to block b of the line
      a = b / g.kb;
      k = b % g.kb;
      if (b < b1) enter(a);
    };
    auto step = [&](int b) {  // to b, two blocks on
      k += 2;
      if (k < g.kb) return;
      k -= g.kb;
      ++a;
      if (k >= g.kb) {  // kb == 1
        k -= g.kb;
        ++a;
      }
      if (b < b1) enter(a);
    };
    auto weights = [&](int stage, uint32_t phase) {
      const uint32_t fb = saddr(&t.full[stage]);
      if (lane == 16) {
        t.issued[stage] = 1 + (int)phase;
        mbar_expect_tx(fb, tx);
      }
      __syncwarp();
      if (lane >= 16 && lane < 16 + BN / 64)
        tma_load_3d(saddr(base + stage * g.stage_bytes) + x_bytes + (lane - 16) * W_CHUNK, &tmW,
                    n0 + 64 * (lane - 16), k * BK, e, fb);
    };
    auto rows = [&](int stage) {
      if (mine)
        tma_load_2d(saddr(base + stage * g.stage_bytes) + lane * (ROW_BOX * 128),
                    all ? &tmAll : &tmA, k * BK, a * g.T + ROW_BOX * lane, saddr(&t.full[stage]));
    };
    const int n = b1 - b0, ahead = min(n, g.stages);
    seek(b0 + warp);
    for (int i = warp; i < ahead; i += 2) {
      weights(i, 0);
      step(b0 + i + 2);
    }
    if (!PROJ) {
      pdl_wait();  // act is complete
      asm volatile("fence.proxy.async;" ::: "memory");  // and read by TMA
    }
    seek(b0 + warp);
    int i = warp;
    for (; i < ahead; i += 2) {
      rows(i);
      step(b0 + i + 2);
    }
    int stage = i;  // i is ahead or ahead + 1, and ahead the ring unless nothing is left
    uint32_t phase = 0;
    for (; i < n; i += 2) {
      while (stage >= g.stages) {
        stage -= g.stages;
        phase ^= 1u;
      }
      if (!mbar_wait_warp(saddr(&t.empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) break;
      weights(stage, phase);
      rows(stage);
      step(b0 + i + 2);
      stage += 2;
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ MMA issuers
    const int w = warp - 2;
    const uint32_t idesc = idesc_bf16(128, BN);  // A (tokens) K-major, B (weights) MN-major
    const uint64_t xd0 = desc_sw128(saddr(base), 16, 1024);
    const uint64_t wd0 = desc_sw128(saddr(base) + x_bytes, W_CHUNK, 1024);
    int stage = w, last = -1;
    uint32_t phase = 0, off[4];
    for (int b = b0 + w; b < b1; b += 2) {
      while (stage >= g.stages) {
        stage -= g.stages;
        phase ^= 1u;
      }
      const int a = b / g.kb;
      if (a != last) {
        last = a;
        const int e = t.m.act[a];
#pragma unroll
        for (int i = 0; i < 4; ++i) off[i] = ~t.m.mask[e][i];
      }
      if (!mbar_wait_warp(saddr(&t.full[stage]), phase, abort_flag, g.status, limit)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t so = (uint64_t)((stage * g.stage_bytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          mma_lanes(tmem + (uint32_t)(w * BN), xd0 + so + (uint64_t)(kk * 2),
                    wd0 + so + (uint64_t)(kk * 128), idesc, off);
        tc_commit<1>(saddr(&t.empty[stage]));
      }
      __syncwarp();
      stage += 2;
    }
    if (elect_one()) tc_commit<1>(saddr(&t.done));
  } else {
    pdl_wait();  // the previous kernel in the stream has completed (low; order of writes to out)
    pdl_trigger();
  }
  __syncwarp();
  int w_ok = 0;
  if (lane == 0) w_ok = mbar_wait(saddr(&t.done), 0, nullptr, g.status, limit);
  w_ok = __shfl_sync(0xffffffffu, w_ok, 0);
  if (warp == 0 && lane == 0 && *abort_flag) {
    // a wait ran out: let the copies in flight land (bounded; otherwise the MMAs have read all)
    const uint64_t t0 = globaltimer_ns();
    for (int s = 0; s < g.stages; ++s)
      while (t.issued[s] != 0 && !mbar_try(saddr(&t.full[s]), (uint32_t)(t.issued[s] - 1)) &&
             globaltimer_ns() - t0 < limit) {
      }
  }
  tc_fence_before();
  __syncthreads();  // every copy and MMA is done: the ring is free
  tc_fence_after();
  const bool ok = w_ok && !*abort_flag;
  float* part = reinterpret_cast<float*>(base);  // [T][PITCH]
  if (warp >= 4) {
    const int q = warp & 3, row = q * 32 + lane;
    if (q * 32 < g.T) {
#pragma unroll 1
      for (int c = 0; c < BN; c += 8) {
        uint32_t v[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          tmem_ld8(tmem + (uint32_t)(i * BN + c) + ((uint32_t)(q * 32) << 16), v[i]);
        tmem_ld_wait();
        if (row < g.T) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            f[j] = __uint_as_float(v[0][j]);
#pragma unroll
            for (int i = 1; i < 2; ++i) f[j] += __uint_as_float(v[i][j]);
          }
          float4* o = reinterpret_cast<float4*>(part + (size_t)row * PITCH + c);
          o[0] = make_float4(f[0], f[1], f[2], f[3]);
          o[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  if (S > 1) cluster_sync();
  else __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, 2 * BN);
  }
  // ---- this rank's tokens: the partial rows of all ranks in rank order, four columns a lane
  if (warp >= 4 && ok) {
    // a warp takes 32 / LANES rows at a time
    const int ew = warp - 4, sub = lane / LANES, c4 = lane % LANES * 4, col = n0 + c4;
    constexpr int PER = 32 / LANES;
    for (int i0 = 0; rank + S * PER * (i0 + ew) < g.T; i0 += 4) {
      const int tok = rank + S * (PER * (i0 + ew) + sub);
      const bool row_on = tok < g.T;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      const uint32_t at = saddr(part) + (uint32_t)(((row_on ? tok : 0) * PITCH + c4) * 4);
      if (S > 1) {
        for (int r = 0; r < S; ++r) {
          const float4 v = ld_dsmem_v4(map_rank(at, (uint32_t)r));
          acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
        }
      } else {
        acc = *reinterpret_cast<const float4*>(part + (size_t)(row_on ? tok : 0) * PITCH + c4);
      }
      if (PROJ) {
        const int l = row_on ? g.ids[tok] : -1;
        const bool has = l >= 0 && l < g.n_adapters;
        float* low = t.low[ew * PER + sub];
        __syncwarp();  // the rows before are done with low
        for (int j = lane % LANES; j < g.rank; j += LANES) {
          float v = 0.f;
          if (has) {
            for (int s = 0; s < g.low_splits; ++s)
              v += g.low_part[((size_t)s * g.T + tok) * g.rank + j];
            v *= g.scale[l];
          }
          low[j] = v;
          if (tile == 0 && row_on) g.low[(size_t)tok * g.rank + j] = v;
        }
        __syncwarp();
        if (has && col < g.d) {
          const bf16* bp = g.b + (size_t)l * g.rank * g.d + col;
#pragma unroll 8
          for (int j = 0; j < g.rank; ++j) {
            const uint2 raw = *reinterpret_cast<const uint2*>(bp + (size_t)j * g.d);
            const float v = low[j];
            acc.x = fmaf(v, __uint_as_float(raw.x << 16), acc.x);
            acc.y = fmaf(v, __uint_as_float(raw.x & 0xffff0000u), acc.y);
            acc.z = fmaf(v, __uint_as_float(raw.y << 16), acc.z);
            acc.w = fmaf(v, __uint_as_float(raw.y & 0xffff0000u), acc.w);
          }
        }
      } else if (row_on && (t.m.bad[tok >> 5] >> (tok & 31) & 1u)) {
        acc = make_float4(NAN, NAN, NAN, NAN);  // NaN logits: no expert, and the row is NaN
      }
      if (row_on && col < g.d)
        *reinterpret_cast<uint2*>(g.out + (size_t)tok * g.d + col) =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    }
  }
  __syncwarp();
  if (S > 1) cluster_sync();  // no rank leaves while its partial may be read
}

struct DownMaps {
  CUtensorMap boxes, all, w;
};
bool maps(DownMaps& m, const void* rows, int T, uint64_t n_rows, const void* w, uint64_t k,
          uint64_t d, uint64_t experts) {
  const uint32_t wbox[3] = {64, 64, 1}, abox[2] = {64, ROW_BOX},
                 xbox[2] = {64, (uint32_t)(T + 7) / 8 * 8};
  const uint64_t wd[3] = {d, k, experts}, ws[2] = {d * 2, k * d * 2};
  const uint64_t ad[2] = {k, n_rows}, as[1] = {k * 2};
  return make_map(&m.boxes, rows, 2, ad, as, abox) && make_map(&m.all, rows, 2, ad, as, xbox) &&
         make_map(&m.w, w, 3, wd, ws, wbox);
}

template <bool PROJ, int BN>
moe_status run_bn(FewDownArgs a, long long blocks, const DownMaps& m, cudaStream_t st) {
  // The largest cluster of 4, 2 or 1 that leaves every CTA two k-blocks and the grid at most
  // two CTAs an SM, all resident at once. (Clusters of eight fit worse between the SMs that the
  // kernel before still holds: 128 tokens, width 4096, 8 experts of 14336: 309 us alone and 600
  // behind it, against 157 and 160 with four.)
  const int tiles = (a.d + BN - 1) / BN, sms = sm_count();
  a.split = 1;
  while (a.split < 4 && 2 * a.split * tiles <= 2 * sms - 16 && blocks >= 4LL * a.split)
    a.split *= 2;
  a.stage_bytes = BN / 64 * W_CHUNK + (a.T + 7) / 8 * 1024;
  const int budget = a.split * tiles <= sms - 16 ? SMEM_ONE : SMEM_TWO;
  a.stages = (budget - 1024 - (int)sizeof(Tail)) / a.stage_bytes;
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  // An even ring: each pair of a loading and an MMA warp then has stages of its own. (A stage that
  // both pairs used in turn could be found free by a pair two rounds ahead of the other.)
  a.stages &= ~1;
  a.ring_bytes = a.stages * a.stage_bytes;
  const int part = (a.T * (BN + 4) * 4 + 1023) / 1024 * 1024;  // the partial tile takes its place
  if (a.ring_bytes < part) a.ring_bytes = part;
  const int smem = 1024 + a.ring_bytes + (int)sizeof(Tail);
  a.status = device_status_ptr();
  a.limit_ns = kWaitLimitNs;
  auto kern = few_down_kernel<PROJ, BN>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_ONE) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  const int kid = PROJ ? K_ADAPTER_FEW : K_FEW_DOWN;
  launch_begin(kid, st);
  launch_kernel(kern, dim3((unsigned)(a.split * tiles)), dim3(THREADS), (size_t)smem, st,
                (unsigned)a.split, m.boxes, m.all, m.w, a);
  return launch_end(kid, st);
}

template <bool PROJ>
moe_status run_down(const FewDownArgs& a, int experts, const DownMaps& m, cudaStream_t st) {
  // 128 columns a tile where clusters of four then give most SMs a CTA, else 64
  const long long blocks = (long long)experts * a.kb;
  return (a.d + 127) / 128 * 4 >= 100 ? run_bn<PROJ, 128>(a, blocks, m, st)
                                      : run_bn<PROJ, 64>(a, blocks, m, st);
}

}  // namespace

// act: [active experts][T][n]; `active`: how many there can be.
moe_status launch_few_down(FewDownArgs a, int n, int active, const void* act, const void* w_down,
                           cudaStream_t st) {
  DownMaps m;
  a.kb = n / BK;
  if (!maps(m, act, a.T, (uint64_t)active * a.T, w_down, n, a.d, a.E)) return MOE_ERR_CUDA;
  return run_down<false>(a, active, m, st);
}

moe_status launch_adapter_few(FewDownArgs a, int d_in, const void* x, const void* w,
                              cudaStream_t st) {
  DownMaps m;
  a.kb = d_in / BK;
  if (!maps(m, x, a.T, a.T, w, d_in, a.d, 1)) return MOE_ERR_CUDA;
  return run_down<true>(a, 1, m, st);
}

}  // namespace moe
