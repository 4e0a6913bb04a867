// Rotary positions with several axes: y = x with the pairs of its rows turned.
// Memory-bound (each element read and written once).  A warp takes one
// token's rows, or a part of its heads where there are few tokens, and gathers
// the token's (cos, sin) once, from as many rows of the table as there are
// axes: into registers where a row's pieces divide the warp (whole rotations of
// 64 or 128 channels among them), into shared memory where they do not.
// 1369 tokens of 40 heads of 128 bf16 channels on 3 axes: 8.1 us (28.8 MB; by
// way of shared memory 12.0; element by element, for rows that 16-byte pieces
// do not fit, 13.1).  20011 tokens of 32 heads in fp32: 99.4 us, 6.7 TB/s (105,
// 105.4).
#include "rope.cuh"

namespace hc {
namespace {

template <typename T, int kPairing, int V, bool kInLanes>
__global__ void __launch_bounds__(kRopeWarps * 32) k_rope_axes(const __grid_constant__ RopeAxesParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t tok, part;
  p.parts.divmod(blockIdx.x * kRopeWarps + warp, tok, part);
  if (tok >= static_cast<uint32_t>(p.n_tokens)) return;
  const int64_t t = tok;
  const int h0 = static_cast<int>(part) * p.heads_per_warp;
  const int h1 = min(h0 + p.heads_per_warp, p.n_heads);
  const T* x = static_cast<const T*>(p.x) + t * p.x_token;
  T* y = static_cast<T*>(p.y) + t * p.y_token;
  bool ok;
  if constexpr (kInLanes) {
    ok = rotate_rows_in_lanes<T, kPairing, V>(p.rope, static_cast<int>(t), x, p.x_head, y, p.y_head, h0, h1,
                                              static_cast<int>(p.items_per_row.d), lane, [] { return true; });
  } else {
    __shared__ float2 cs[kRopeWarps][128];
    ok = stage_cos_sin(p.rope, static_cast<int>(t), lane, cs[warp]);
    if (ok)
      rotate_rows<T, kPairing, V, 4>(x, p.x_head, y, p.y_head, h0, h1, p.rope.half, cs[warp], p.items_per_row, lane);
  }
  if (!ok && lane == 0) flag_error(p.err, HC_DEVERR_POS);
}

template <typename T, int kPairing, int V>
cudaError_t launch(RopeAxesParams p, cudaStream_t s) {
  const int items = rope_items<kPairing, V>(p.rope.half, p.d);
  p.items_per_row = FastDivmod(static_cast<uint32_t>(items));
  const bool in_lanes = V * sizeof(T) == 16 && items <= 32 && 32 % items == 0;
  p.heads_per_warp = heads_per_warp(p.n_tokens, p.n_heads, items, false);
  p.parts = FastDivmod(static_cast<uint32_t>((p.n_heads + p.heads_per_warp - 1) / p.heads_per_warp));
  const int64_t warps = static_cast<int64_t>(p.n_tokens) * p.parts.d;
  const unsigned grid = static_cast<unsigned>((warps + kRopeWarps - 1) / kRopeWarps);
  if (in_lanes)
    k_rope_axes<T, kPairing, V, V * sizeof(T) == 16><<<grid, kRopeWarps * 32, 0, s>>>(p);
  else
    k_rope_axes<T, kPairing, V, false><<<grid, kRopeWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_dtype(int pairing, bool pieces16, const RopeAxesParams& p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  if (pairing == HC_PAIR_HALF_SPLIT)
    return pieces16 ? launch<T, HC_PAIR_HALF_SPLIT, V>(p, s) : launch<T, HC_PAIR_HALF_SPLIT, 1>(p, s);
  return pieces16 ? launch<T, HC_PAIR_INTERLEAVED, V>(p, s) : launch<T, HC_PAIR_INTERLEAVED, 2>(p, s);
}

}  // namespace

cudaError_t launch_rope_axes(int dtype, int pairing, bool pieces16, const RopeAxesParams& p,
                             cudaStream_t s) {
  switch (dtype) {
    case HC_F32: return launch_dtype<float>(pairing, pieces16, p, s);
    case HC_F16: return launch_dtype<__half>(pairing, pieces16, p, s);
    default: return launch_dtype<__nv_bfloat16>(pairing, pieces16, p, s);
  }
}

}  // namespace hc
