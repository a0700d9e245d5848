// Shared pieces of the adapter kernels: the table of adapters by row tile, warp-level matrix instructions on 16 x 8
// tiles (used where a product is too thin for the tensor-core pipeline through TMEM) and the
// split of an fp32 value into bf16 terms.
#pragma once

#include "tc_ptx.cuh"

namespace moe {

// The adapters that have rows in a 256-row tile of the large product, and for each the rows
// (bit r % 32 of word r / 32) that are NOT its own.
constexpr int kAdapterTileRows = 256;
struct AdapterTile {
  int n;
  int pad[3];
  int id[kAdapterTileRows];
  uint32_t off[kAdapterTileRows][8];
};

// D[16 x 8] += A[16 x 16] B[16 x 8], bf16 operands, fp32 sums.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
// 16 bytes global -> shared, zeros when `on` is false (nothing is read then).
__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// (a, b) as bf16 pairs hi + lo (+ what is left, returned in a and b): 8 bits of mantissa each.
__device__ __forceinline__ uint32_t take_bf16x2(float& a, float& b) {
  const uint32_t h = pack_bf16x2(a, b);
  a -= __uint_as_float(h << 16);
  b -= __uint_as_float(h & 0xffff0000u);
  return h;
}

}  // namespace moe
