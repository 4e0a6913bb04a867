// Pieces shared by the two attention kernels over the paged buffer: requests,
// the keys that a query and a run of query rows see, and scores.
#pragma once

#include "attend_common.cuh"
#include "paged.cuh"

namespace hc {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A request as the call sees it; n = 0 where there is nothing to write.
struct PagedRequest {
  int q0, n, kv, prefix;
};
__device__ __forceinline__ PagedRequest load_request(const AttendPagedParams& p, int r, int& bad) {
  PagedRequest q;
  q.q0 = __ldg(p.q_starts + r);
  q.n = __ldg(p.q_starts + r + 1) - q.q0;
  q.kv = __ldg(p.kv_lens + r);
  q.prefix = p.prefix_lens ? max(__ldg(p.prefix_lens + r), 0) : 0;
  const bool ok = q.n >= 0 && q.n <= p.max_new && q.q0 >= 0 && q.q0 <= p.n_tokens - q.n && q.kv >= 0 &&
                  q.kv <= p.most_keys;
  if (!ok) {
    bad |= HC_DEVERR_LENGTH;
    q.q0 = q.n = q.kv = 0;
  }
  return q;
}

// Position of the request's query i; any negative one (more queries than keys) is -1.
__device__ __forceinline__ int position(const AttendPagedParams& p, const PagedRequest& q, int i) {
  return max(p.positions ? __ldg(p.positions + q.q0 + i) : q.kv - q.n + i, -1);
}
// Keys [lo, hi) that a query at this position sees; hi <= lo: none.
__device__ __forceinline__ int last_key(const AttendPagedParams& p, const PagedRequest& q, int pos) {
  return p.causal ? max(min(pos, q.kv - 1) + 1, min(q.prefix, q.kv)) : q.kv;
}
__device__ __forceinline__ int first_key(const AttendPagedParams& p, int pos) {
  return p.window ? max(0, pos - p.window + 1) : 0;
}

// Keys [lo, hi) that some of the rows [row0, row1) see, and their tiles of
// kTile keys.  Positions do not fall within a request, so the first row's
// window starts first and the last row sees furthest.
template <int kTile>
__device__ __forceinline__ Range visible(const AttendPagedParams& p, const PagedRequest& q, int row0, int row1) {
  Range v;
  v.hi = last_key(p, q, position(p, q, static_cast<int>(p.by_group.div(row1 - 1))));
  v.lo = first_key(p, position(p, q, static_cast<int>(p.by_group.div(row0))));
  if (v.lo >= v.hi) v.lo = v.hi = 0;
  v.tile0 = v.lo / kTile;
  v.tiles = max(1, (v.hi + kTile - 1) / kTile - v.tile0);  // rows without keys are still written
  return v;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tanh(y) to 2^-22 of 1 and of y.  Up to 1/2, where 1 - 2 / (e^2y + 1) would
// cancel, an odd polynomial: the minimax fit of tanh(y) / y in y^2 by Remez'
// exchange, off by 1.3e-8.  Above, that formula.
__device__ __forceinline__ float tanh_of(float y) {
  const float u = y * y;
  const float small =
      y * fmaf(u, fmaf(u, fmaf(u, fmaf(u, 0.0171350182863f, -0.0529860809237f), 0.133247793996f), -0.333330693977f),
               0.999999986872f);
  const float large = fmaf(-2.f, rcp(ex2(y * (2.f * kLog2e)) + 1.f), 1.f);
  return fabsf(y) < 0.5f ? small : large;
}

}  // namespace
}  // namespace hc
