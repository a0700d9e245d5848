// What the kernels for a few tokens share: the size limit, the token masks of the experts, and
// the small wrappers that they have in common.
#pragma once

#include "tc_ptx.cuh"

namespace moe {

constexpr int kFewMaxTokens = 128;  // one 128-lane MMA tile of tokens
constexpr int kFewMaxExperts = 256;

// Which tokens each expert keeps, and which experts have any.
struct FewMasks {
  unsigned mask[kFewMaxExperts][4];  // bit t of an expert's 128: token t is routed to it and kept
  short act[kFewMaxExperts];         // the experts with a kept token, ascending
  int n_act, most;                   // how many, and the most tokens of one
  unsigned bad[4];                   // tokens with an id that is no expert (NaN logits)
};

// few_clear_masks, then few_build_masks, by every thread of the block (n_threads): the masks are
// complete for all of them when the second returns. Over the capacity the first `cap` tokens of
// an expert stay. Clearing needs no global memory, so it can come before a wait.
__device__ __forceinline__ void few_clear_masks(FewMasks& m, int E, int n_threads) {
  for (int i = threadIdx.x; i < 4 * E; i += n_threads) (&m.mask[0][0])[i] = 0u;
  if (threadIdx.x < 4) m.bad[threadIdx.x] = 0u;
  __syncthreads();
}
__device__ __forceinline__ void few_build_masks(FewMasks& m, const int32_t* ids, int T, int K,
                                                int E, int cap, int n_threads) {
  const int tid = threadIdx.x, lane = tid & 31;
  for (int a = tid; a < T * K; a += n_threads) {
    const int e = ids[a], t = a / K;
    if (e >= 0 && e < E) atomicOr(&m.mask[e][t >> 5], 1u << (t & 31));
    else atomicOr(&m.bad[t >> 5], 1u << (t & 31));
  }
  __syncthreads();
  if (tid < 32) {
    int n = 0, most = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      int c = 0;
      if (e < E) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          unsigned b = m.mask[e][w];
          while (c + __popc(b) > cap) b &= ~(0x80000000u >> __clz(b));
          m.mask[e][w] = b;
          c += __popc(b);
        }
      }
      const unsigned has = __ballot_sync(0xffffffffu, c > 0);
      if (c > 0) m.act[n + __popc(has & lanemask_lt())] = (short)e;
      n += __popc(has);
      most = max(most, c);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      m.n_act = n;
      m.most = most;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int few_count(const unsigned (&m)[4]) {
  return __popc(m[0]) + __popc(m[1]) + __popc(m[2]) + __popc(m[3]);
}
// A line of `total` blocks cut into equal pieces, one per CTA, at least `least` blocks each (the
// first ones a block longer): where piece c begins, and the piece that holds block b.
struct FewPieces {
  int n, q, r;
  __device__ __forceinline__ FewPieces(int total, int least, int ctas) {
    n = max(1, min(ctas, total / least));
    q = total / n;
    r = total - q * n;
  }
  __device__ __forceinline__ int begin(int c) const { return c * q + min(c, r); }
  __device__ __forceinline__ int of(int b) const {
    const int longer = r * (q + 1);
    return b < longer ? b / (q + 1) : r + (b - longer) / q;
  }
};

}  // namespace moe
