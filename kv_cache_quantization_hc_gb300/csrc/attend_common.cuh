// Pieces shared by the two attention kernels over the 4-bit cache: requests,
// the keys that a run of query rows sees, and small conversions.
#pragma once

#include "serve.cuh"

namespace hc {
namespace {

constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// (w & mask) ^ flip in one LOP3: left to itself the compiler makes two, each
// with its constant, and the integer pipe is what the loops are bound by.
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t mask, uint32_t flip) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(d) : "r"(w), "r"(mask), "r"(flip));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
// 2^e as a float, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Two 16-bit elements as floats.
__device__ __forceinline__ float2 widen(uint32_t u, int bf16) {
  return bf16 ? u32_to_float2(u, static_cast<const __nv_bfloat16*>(nullptr))
              : u32_to_float2(u, static_cast<const __half*>(nullptr));
}

// A request as the call sees it; n = 0 where there is nothing to write.
struct Request {
  int q0, n, kv;
};
__device__ __forceinline__ Request load_request(const AttendParams& p, int r, int& bad) {
  Request q;
  q.q0 = __ldg(p.q_starts + r);
  q.n = __ldg(p.q_starts + r + 1) - q.q0;
  q.kv = __ldg(p.kv_lens + r);
  const bool ok = q.n >= 0 && q.n <= p.max_new && q.q0 >= 0 && q.q0 <= p.n_tokens - q.n && q.kv >= 0 &&
                  q.kv <= (static_cast<int64_t>(p.table_width) << p.B_log2);
  if (!ok) {
    bad |= HC_DEVERR_LENGTH;
    q.q0 = q.n = q.kv = 0;
  }
  return q;
}

// Keys [lo, hi) that some of the rows [row0, row1) see, and their tiles of kTile keys.
struct Range {
  int lo, hi, tile0, tiles;
};
template <int kTile>
__device__ __forceinline__ Range visible(const AttendParams& p, const Request& q, int row0, int row1) {
  const int i0 = static_cast<int>(p.by_group.div(row0)), i1 = static_cast<int>(p.by_group.div(row1 - 1));
  Range v;
  v.hi = p.causal ? min(q.kv, q.kv - q.n + i1 + 1) : q.kv;
  v.lo = p.window ? max(0, q.kv - q.n + i0 - p.window + 1) : 0;
  if (v.lo >= v.hi) v.lo = v.hi = 0;
  v.tile0 = v.lo / kTile;
  v.tiles = max(1, (v.hi + kTile - 1) / kTile - v.tile0);  // rows without keys are still written
  return v;
}

}  // namespace
}  // namespace hc
