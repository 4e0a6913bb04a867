// Copies into shared memory and matrix operands of one warp, as the attention
// kernels over few rows use them.
#pragma once

#include "attend_common.cuh"

namespace hc {
namespace {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes));
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two fp32 as pairs of bf16, high and low: the upper halves as they stand,
// and what is left of them rounded to bf16: 16 bits in all.
__device__ __forceinline__ void split_bf16(float2 v, uint32_t& high, uint32_t& low) {
  const uint32_t ux = __float_as_uint(v.x), uy = __float_as_uint(v.y);
  high = __byte_perm(ux, uy, 0x7632);
  const float2 kept = make_float2(__uint_as_float(high * 65536u), __uint_as_float(high & 0xffff0000u));
  const __nv_bfloat162 rest = __float22bfloat162_rn(__ffma2_rn(kept, make_float2(-1.f, -1.f), v));
  memcpy(&low, &rest, 4);
}

}  // namespace
}  // namespace hc
