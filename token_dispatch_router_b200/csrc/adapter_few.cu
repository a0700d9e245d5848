// The shared projection with per-request adapters for at most 128 rows (M, one lane each):
//   y[t] = x_t W + low_t B_l,  l = ids[t]   (low_t = scale_l x_t A_l from partial sums)
//
// Bound by reading W, or, for the few rows of a decode step, by latency. An output tile of 64 or
// 128 columns belongs to a cluster of up to four CTAs that split the contraction; the partial
// tiles are added in rank order through distributed shared memory (results repeat bit for bit),
// each rank a share of the rows, to which it adds the adapter's product: r values of low against
// r rows of B_l, in fp32, four columns a lane. So the whole GPU reads W and takes part in the
// adapter term, and rows do not mix.
// x and W do not depend on the kernel before this one (it makes low), so their product starts
// before that kernel has ended: its own launch follows that kernel's wait, so everything older
// is complete. Only the last step waits for low.
// Roles (256 threads): warp 0 copies weights, warp 1 rows, warp 2 issues the MMAs, warps 4-7
// read the accumulator and add up the partials. A finished wait costs a warp about 200 cycles
// and a copy or an MMA 60 to issue, so a stage holds 32 KB of weights (128 or 256 k) brought by
// one copy, and rows have a warp of their own.
// Every wait (but tmem_alloc's) is bounded (MOE_ERR_TIMEOUT on expiry).
#include "few.cuh"
#include "few_args.cuh"
#include "ffn_args.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int THREADS = 256;
constexpr int W_BYTES = 32768;                   // weights of a stage
// A stage is the rows (for each 64 k: T rounded up to 8 rows of 128 bytes), then the weights. The
// MMA reads 128 rows: past T it runs on into what lies behind in the same stage; nobody reads
// those lanes.
constexpr int MAX_STAGES = 6;
constexpr int SMEM_ONE = 200 * 1024, SMEM_TWO = 108 * 1024;  // one or two CTAs on an SM
constexpr int SMEM_MAX = 227 * 1024;

struct Tail {
  uint64_t full[MAX_STAGES], full_x[MAX_STAGES], empty[MAX_STAGES], done;
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ float4 ld_dsmem_v4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

// BN: columns of an output tile, 64 or 128.
template <int BN>
__global__ void __launch_bounds__(THREADS, 2)
    adapter_few_kernel(const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmW, const AdapterFewArgs g) {
  constexpr int BK = W_BYTES / (2 * BN);  // k of a stage
  constexpr int PIECES = BK / 64;
  constexpr int PITCH = BN + 4;     // floats per row of the partial tile
  constexpr int LANES = BN / 4;     // lanes on a row of it, four columns each
  extern __shared__ uint8_t smem_raw[];
  // the ring (later the partial tile, at most 528 bytes a row: less than a ring), low, barriers
  uint8_t* base = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Tail& t = *reinterpret_cast<Tail*>(base + g.ring_bytes + g.low_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &t.abort;
  const int S = g.split, rank = S > 1 ? (int)cluster_rank() : 0;
  const int tile = (int)blockIdx.x / S, n0 = tile * BN;

  if (tid == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(saddr(&t.full[s]), 1);
      mbar_init(saddr(&t.full_x[s]), 1);
      mbar_init(saddr(&t.empty[s]), 1);
    }
    mbar_init(saddr(&t.done), 1);
    t.abort = 0;
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc<1>(saddr(&t.tmem), BN);
  if (tid == 96) {
    prefetch_map(&tmX);
    prefetch_map(&tmW);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = t.tmem;
  const uint64_t limit = g.limit_ns;
  const int mine = (g.T - rank + S - 1) / S;  // rows rank, rank + S, ... are this rank's
  float* low = reinterpret_cast<float*>(base + g.ring_bytes);  // [mine][rank]
  const uint32_t x_piece = (uint32_t)(g.T + 7) / 8u * 1024u, x_bytes = PIECES * x_piece;
  const int b0 = rank * g.kb / S, b1 = (rank + 1) * g.kb / S;

  if (warp == 0 || warp == 1) {
    // ------------------------------------------------------------ loads
    const bool x_warp = warp == 1;
    const uint64_t once = l2_policy_evict_first();  // W is read once
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_par = 0;
    for (int b = b0; b < b1; ++b) {
      if (!mbar_wait_warp(saddr(&t.empty[stage]), phase ^ 1u, abort_flag, g.status, limit)) break;
      const uint32_t x = saddr(base + stage * g.stage_bytes);
      const uint32_t fb = saddr(x_warp ? &t.full_x[stage] : &t.full[stage]);
      if (elect_one()) {
        mbar_expect_tx(fb, x_warp ? x_bytes : (uint32_t)W_BYTES);
        if (x_warp) tma_load_4d(x, &tmX, 0, 0, b * PIECES, 0, fb);
        else tma_load_4d_hint(x + x_bytes, &tmW, 0, b * BK, tile * (BN / 64), 0, fb, once);
      }
      __syncwarp();
      issued_mask |= 1u << stage;
      issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
      if (++stage == g.stages) {
        stage = 0;
        phase ^= 1u;
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
  } else if (warp == 2) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = idesc_bf16(128, BN);  // A (tokens) K-major, B (weights) MN-major
    const uint64_t xd0 = desc_sw128(saddr(base), 16, 1024);
    const uint64_t wd0 = desc_sw128(saddr(base) + x_bytes, BK * 128, 1024);
    int stage = 0;
    uint32_t phase = 0;
    for (int b = b0; b < b1; ++b) {
      if (!mbar_wait_warp(saddr(&t.full[stage]), phase, abort_flag, g.status, limit) ||
          !mbar_wait_warp(saddr(&t.full_x[stage]), phase, abort_flag, g.status, limit))
        break;
      tc_fence_after();
      if (elect_one()) {
        uint64_t xd = xd0 + (uint64_t)((stage * g.stage_bytes) >> 4);
        uint64_t wd = wd0 + (uint64_t)((stage * g.stage_bytes) >> 4);
#pragma unroll 1
        for (int p = 0; p < PIECES; ++p, xd += x_piece >> 4, wd += 4 * 128)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma<1>(tmem, xd + (uint64_t)(kk * 2), wd + (uint64_t)(kk * 128), idesc,
                      (b > b0 || p > 0 || kk > 0) ? 1u : 0u);
        tc_commit<1>(saddr(&t.empty[stage]));
      }
      __syncwarp();
      if (++stage == g.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (elect_one()) tc_commit<1>(saddr(&t.done));
  } else if (warp >= 4) {
    pdl_wait();  // the previous kernel in the stream has completed (low; order of writes to out)
    pdl_trigger();
    // meanwhile: low of this rank's rows, and their adapters' pieces of B on their way to L2
    for (int i = tid - 128; i < mine * g.rank; i += 128) {
      const int tok = rank + S * (i / g.rank), j = i % g.rank, l = g.ids[tok];
      float v = 0.f;
      if (l >= 0 && l < g.n_adapters) {
        for (int s = 0; s < g.low_splits; ++s)
          v += g.low_part[((size_t)s * g.T + tok) * g.rank + j];
        v *= g.scale[l];
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            g.b + ((size_t)l * g.rank + j) * g.d + n0));  // the first line of the piece
      }
      low[i] = v;
      if (tile == 0) g.low[(size_t)tok * g.rank + j] = v;
    }
  }
  __syncwarp();
  int w_ok = 0;
  if (lane == 0) w_ok = mbar_wait(saddr(&t.done), 0, nullptr, g.status, limit);
  w_ok = __shfl_sync(0xffffffffu, w_ok, 0);
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
        uint32_t v[8];
        tmem_ld8(tmem + (uint32_t)c + ((uint32_t)(q * 32) << 16), v);
        tmem_ld_wait();
        if (row < g.T) {
          uint4* o = reinterpret_cast<uint4*>(part + (size_t)row * PITCH + c);
          o[0] = make_uint4(v[0], v[1], v[2], v[3]);
          o[1] = make_uint4(v[4], v[5], v[6], v[7]);
        }
      }
    }
  }
  // TMEM is given back before the peers are waited for: one of them may be waiting for TMEM itself,
  // beside another call's CTA that waits for a peer of its own
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<1>(tmem, BN);
  }
  __syncwarp();
  if (S > 1) cluster_sync();
  // ---- this rank's tokens: the partial rows of all ranks in rank order, four columns a lane
  if (ok) {
    // a warp takes 32 / LANES rows at a time
    const int sub = lane / LANES, c4 = lane % LANES * 4, col = n0 + c4;
    constexpr int PER = 32 / LANES;
    for (int i0 = PER * warp; i0 < mine; i0 += PER * (THREADS / 32)) {
      const int i = i0 + sub, tok = rank + S * i;
      const bool row_on = i < mine;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      const uint32_t at = saddr(part) + (uint32_t)(((row_on ? tok : 0) * PITCH + c4) * 4);
      const int l = row_on ? g.ids[tok] : -1;
      if (S > 1) {
        for (int r = 0; r < S; ++r) {
          const float4 v = ld_dsmem_v4(map_rank(at, (uint32_t)r));
          acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
        }
      } else {
        acc = *reinterpret_cast<const float4*>(part + (size_t)(row_on ? tok : 0) * PITCH + c4);
      }
      if (l >= 0 && l < g.n_adapters && col < g.d) {
        const bf16* bp = g.b + (size_t)l * g.rank * g.d + col;
        const float* lw = low + (size_t)i * g.rank;
#pragma unroll 8
        for (int j = 0; j < g.rank; ++j) {
          const uint2 raw = *reinterpret_cast<const uint2*>(bp + (size_t)j * g.d);
          const float v = lw[j];
          acc.x = fmaf(v, __uint_as_float(raw.x << 16), acc.x);
          acc.y = fmaf(v, __uint_as_float(raw.x & 0xffff0000u), acc.y);
          acc.z = fmaf(v, __uint_as_float(raw.y << 16), acc.z);
          acc.w = fmaf(v, __uint_as_float(raw.y & 0xffff0000u), acc.w);
        }
      }
      if (row_on && col < g.d)
        *reinterpret_cast<uint2*>(g.out + (size_t)tok * g.d + col) =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    }
  }
  __syncwarp();
  if (S > 1) cluster_sync();  // no rank leaves while its partial may be read
}

template <int BN>
moe_status run_bn(AdapterFewArgs a, int d_in, const void* x, const void* w, cudaStream_t st) {
  constexpr int BK = W_BYTES / (2 * BN), PIECES = BK / 64;
  a.kb = (d_in + BK - 1) / BK;
  // The largest cluster of 4, 2 or 1 with which the whole grid runs at once: two CTAs an SM where
  // two stages of each fit beside the cluster's share of low, else one (16 SMs are left out: clusters
  // stay inside a group of SMs). More tiles than SMs run one after another, without clusters.
  const int tiles = (a.d + BN - 1) / BN, sms = sm_count();
  a.stage_bytes = W_BYTES + PIECES * ((a.T + 7) / 8 * 1024);
  auto low_bytes = [&](int split) {
    return ((a.T + split - 1) / split * a.rank * 4 + 15) / 16 * 16;
  };
  auto fixed = [&](int split) { return 1024 + (int)sizeof(Tail) + low_bytes(split); };
  auto two = [&](int split) { return SMEM_TWO - fixed(split) >= 2 * a.stage_bytes; };
  auto at_once = [&](int split) { return split * tiles <= (two(split) ? 2 : 1) * sms - 16; };
  a.split = 1;
  for (int n = 2; n <= 4 && 2 * n <= a.kb; n *= 2)  // every CTA has two stages at least
    if (at_once(n)) a.split = n;
  a.low_bytes = low_bytes(a.split);
  a.stages = ((a.split * tiles <= sms - 16 ? SMEM_ONE : SMEM_TWO) - fixed(a.split)) / a.stage_bytes;
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  // one CTA an SM then; a single stage where low (64 KB at most) leaves no more
  if (a.stages < 2) a.stages = SMEM_MAX - fixed(a.split) >= 2 * a.stage_bytes ? 2 : 1;
  a.ring_bytes = a.stages * a.stage_bytes;
  const int smem = fixed(a.split) + a.ring_bytes;
  a.status = device_status_ptr();
  a.limit_ns = kWaitLimitNs;
  CUtensorMap mx, mw;
  if (!make_piece_map(&mx, x, a.T, d_in, 1, (uint32_t)(a.T + 7) / 8 * 8, PIECES) ||
      !make_piece_map(&mw, w, d_in, a.d, 1, BK, BN / 64))
    return MOE_ERR_CUDA;
  auto kern = adapter_few_kernel<BN>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  launch_begin(K_ADAPTER_FEW, st);
  launch_kernel(kern, dim3((unsigned)(a.split * tiles)), dim3(THREADS), (size_t)smem, st,
                (unsigned)a.split, mx, mw, a);
  return launch_end(K_ADAPTER_FEW, st);
}

}  // namespace

moe_status launch_adapter_few(const AdapterFewArgs& a, int d_in, const void* x, const void* w,
                              cudaStream_t st) {
  // 128 columns a tile where clusters of four then give most SMs a CTA, else 64
  return (a.d + 127) / 128 * 4 >= 100 ? run_bn<128>(a, d_in, x, w, st)
                                      : run_bn<64>(a, d_in, x, w, st);
}

}  // namespace moe
