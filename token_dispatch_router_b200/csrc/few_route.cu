// Router of the few-token layer: logits = x W_r (+ bias), softmax and top-K for at most 128
// tokens, with any E and K that the layer takes. It also clears the control words of the
// kernel that follows it.
//
// A latency-bound step (W_r is a few hundred KB): a cluster of 8 CTAs takes 1 to 8 tokens, as
// many as keep the clusters of all tokens on the SMs at once, and splits d. A CTA copies its
// rows of W_r to shared memory with all of its cp.async in flight together (one round trip),
// and every thread sums one expert over its share of the rows, for all the cluster's tokens,
// in fp32. The partials of a CTA are added through shared memory, those of the cluster through
// distributed shared memory in rank order (the sums do not depend on timing), by the rank that
// owns the token; one warp then ranks it (K rounds of a warp arg-max).
#include "few.cuh"
#include "tc_ptx.cuh"
#include "topk.cuh"

namespace moe {

namespace {

using namespace ptx;

constexpr int THREADS = 256;
constexpr int RANKS = 8;
constexpr int W_SMEM = 128 * 1024;  // rows of W_r held at a time

struct FewRouteArgs {
  const bf16* x;
  const bf16* w_r;
  const float* bias;
  const float* logits_in;
  int32_t* ids;
  float* w;
  uint32_t* clear;
  int n_clear;
  int T, d, E, K, renorm;
  int ec;    // E rounded up to a power of two (at least 8): threads side by side on a row
  int rows;  // rows of W_r per pass (a multiple of 8)
};

// TG tokens a cluster; VPL logits a lane when a token is ranked.
template <int TG, int VPL>
__global__ void __launch_bounds__(THREADS) few_route_kernel(const FewRouteArgs g) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ float part[TG * 32 * VPL];
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = (int)cluster_rank(), t0 = (int)cluster_id_x() * TG;
  pdl_wait();  // the previous kernel in the stream has completed
  pdl_trigger();
  for (int i = blockIdx.x * THREADS + tid; i < g.n_clear; i += gridDim.x * THREADS) g.clear[i] = 0u;

  if (g.logits_in == nullptr) {
    bf16* wsm = reinterpret_cast<bf16*>(smem_raw);
    float* xs = reinterpret_cast<float*>(smem_raw + (size_t)g.rows * g.E * 2);  // [rows][TG]
    float* red = xs + (size_t)g.rows * TG;                                     // [256][TG]
    const int k0 = (int)((long long)rank * (g.d / 8) / RANKS) * 8;
    const int k1 = (int)((long long)(rank + 1) * (g.d / 8) / RANKS) * 8;
    const int e = tid & (g.ec - 1), ks = tid / g.ec, nks = THREADS / g.ec;
    float acc[TG];
#pragma unroll
    for (int j = 0; j < TG; ++j) acc[j] = 0.f;
    for (int kc = k0; kc < k1; kc += g.rows) {
      const int nr = min(g.rows, k1 - kc);
      __syncthreads();  // the buffers of the pass before are free
      const uint8_t* src = reinterpret_cast<const uint8_t*>(g.w_r + (size_t)kc * g.E);
      for (int i = tid; i < nr * g.E / 8; i += THREADS) cp_async16(saddr(wsm) + i * 16, src + (size_t)i * 16);
      for (int i = tid; i < TG * (nr / 8); i += THREADS) {
        const int j = i / (nr / 8), r = (i % (nr / 8)) * 8;
        float f[8];
        if (t0 + j < g.T) {
          unpack16(*reinterpret_cast<const uint4*>(g.x + (size_t)(t0 + j) * g.d + kc + r), f, bf16());
        } else {
#pragma unroll
          for (int v = 0; v < 8; ++v) f[v] = 0.f;
        }
#pragma unroll
        for (int v = 0; v < 8; ++v) xs[(r + v) * TG + j] = f[v];
      }
      cp_async_wait_all();
      __syncthreads();
      if (e < g.E) {
#pragma unroll 4
        for (int k = ks; k < nr; k += nks) {
          const float wv = to_f32(wsm[k * g.E + e]);
#pragma unroll
          for (int j = 0; j < TG; ++j) acc[j] = fmaf(xs[k * TG + j], wv, acc[j]);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TG; ++j) red[tid * TG + j] = acc[j];
    __syncthreads();
    for (int i = tid; i < TG * g.E; i += THREADS) {
      const int j = i / g.E, ee = i % g.E;
      float s = 0.f;
      for (int q = 0; q < nks; ++q) s += red[(q * g.ec + ee) * TG + j];
      part[j * 32 * VPL + ee] = s;
    }
    cluster_sync();  // every rank's partial is in its shared memory
  }

  if (tid < 32) {  // this rank's token
    const int t = t0 + rank;
    if (rank < TG && t < g.T) {
      float v[VPL];
      if (g.logits_in != nullptr) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const int e = lane + 32 * j;
          v[j] = e < g.E ? g.logits_in[(size_t)t * g.E + e] : -INFINITY;
        }
      } else {
        uint32_t base[RANKS];
#pragma unroll
        for (int q = 0; q < RANKS; ++q) base[q] = map_rank(saddr(part), (uint32_t)q);
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const int e = lane + 32 * j;
          float p[RANKS];
          const int at = (rank * 32 * VPL + min(e, g.E - 1)) * 4;
#pragma unroll
          for (int q = 0; q < RANKS; ++q) p[q] = ld_dsmem_f32(base[q] + at);
          float s = p[0];
#pragma unroll
          for (int q = 1; q < RANKS; ++q) s += p[q];
          if (g.bias != nullptr && e < g.E) s += g.bias[e];
          v[j] = e < g.E ? s : -INFINITY;
        }
      }
      int id;
      float w;
      warp_route_token<VPL, TOPK_ROUNDS>(v, g.E, g.K, g.renorm, id, w);
      if (lane < g.K) {
        g.ids[(size_t)t * g.K + lane] = id;
        g.w[(size_t)t * g.K + lane] = w;
      }
    }
  }
  __syncwarp();
  if (g.logits_in == nullptr) cluster_sync();  // no rank leaves while its partial may be read
}

template <int TG, int VPL>
moe_status run(const FewRouteArgs& a, cudaStream_t st) {
  auto kern = few_route_kernel<TG, VPL>;
  size_t smem = 16;
  if (a.logits_in == nullptr)
    smem = (size_t)a.rows * a.E * 2 + (size_t)a.rows * TG * 4 + (size_t)THREADS * TG * 4;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  launch_begin(K_FEW_ROUTE, st);
  launch_kernel(kern, dim3((unsigned)((a.T + TG - 1) / TG * RANKS)), dim3(THREADS), smem, st,
                RANKS, a);
  return launch_end(K_FEW_ROUTE, st);
}

template <int TG>
moe_status run_tg(const FewRouteArgs& a, cudaStream_t st) {
  if (a.E <= 32) return run<TG, 1>(a, st);
  if (a.E <= 64) return run<TG, 2>(a, st);
  if (a.E <= 128) return run<TG, 4>(a, st);
  return run<TG, 8>(a, st);
}

}  // namespace

moe_status launch_few_route(const moe_shape& s, const void* x, const void* w_r, const float* bias,
                            const float* logits_in, int32_t* ids, float* w, uint32_t* clear,
                            int n_clear, cudaStream_t st) {
  FewRouteArgs a = {};
  a.x = (const bf16*)x;
  a.w_r = (const bf16*)w_r;
  a.bias = bias;
  a.logits_in = logits_in;
  a.ids = ids;
  a.w = w;
  a.clear = clear;
  a.n_clear = n_clear;
  a.T = s.T;
  a.d = s.d;
  a.E = s.E;
  a.K = s.K;
  a.renorm = s.renormalize;
  a.ec = 8;
  while (a.ec < s.E) a.ec *= 2;
  const int most = (s.d / 8 + RANKS - 1) / RANKS * 8;  // rows of a rank
  a.rows = W_SMEM / (2 * s.E) / 8 * 8;
  if (a.rows > 1024) a.rows = 1024;
  if (a.rows > most) a.rows = most;
  // one token a cluster while the clusters of all tokens fit the SMs, then 2, 4, 8
  const int fit = sm_count() / RANKS;
  if (s.T <= fit) return run_tg<1>(a, st);
  if (s.T <= 2 * fit) return run_tg<2>(a, st);
  if (s.T <= 4 * fit) return run_tg<4>(a, st);
  return run_tg<8>(a, st);
}

}  // namespace moe
