// The new tokens into the paged buffer: queries and keys rotated, values
// copied, in one launch.  Memory-bound: q, k, v read once, q_out and the
// buffer's rows written once.
//
// A warp takes some heads of a token: of its queries, its keys or its values.
// Rotated rows go as k_rope_axes takes them, (cos, sin) in registers where a
// row's pieces divide the warp and in shared memory where they do not; a row of
// the buffer is a token's heads side by side.
#include "paged.cuh"
#include "rope.cuh"

namespace hc {
namespace {

// Whether the token's positions are in the table (a lane per axis).
__device__ __forceinline__ bool positions_exist(const RopeParams& p, int64_t t, int lane) {
  bool ok = true;
  if (p.table != nullptr && (p.axes >> lane & 1u)) {
    const int pos = __ldg(p.positions + lane * p.position_stride + t);
    ok = pos >= 0 && pos < p.n_positions;
  }
  return __all_sync(0xffffffffu, ok);
}

template <typename T, int kPairing, bool kInLanes>
__global__ void __launch_bounds__(kRopeWarps * 32) k_append_paged(const __grid_constant__ AppendPagedParams p) {
  constexpr int V = 16 / sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t tok, part_of;
  p.parts.divmod(blockIdx.x * kRopeWarps + warp, tok, part_of);
  if (tok >= static_cast<uint32_t>(p.n_tokens)) return;
  const int64_t t = tok;
  int part = static_cast<int>(part_of);
  // asked after the data is on its way: what is read is there whatever the row says
  const int64_t row = __ldg(p.token_rows + t);
  const bool row_ok = row >= -1 && row < p.n_rows;
  const T *x;
  T* y;
  int64_t x_head, y_head;
  int heads;
  if (part < p.q_parts) {
    x = static_cast<const T*>(p.q) + t * p.q_token;
    y = static_cast<T*>(p.q_out) + t * p.o_token;
    x_head = p.q_head;
    y_head = p.o_head;
    heads = p.n_q_heads;
  } else {
    part -= p.q_parts;
    const bool keys = part < p.kv_parts;
    if (!keys) part -= p.kv_parts;
    x = keys ? static_cast<const T*>(p.k) + t * p.k_token : static_cast<const T*>(p.v) + t * p.v_token;
    x_head = keys ? p.k_head : p.v_head;
    y_head = p.d;
    heads = p.H;
    // rows that are not there (and a padding token's) are not written: see below
    const int64_t slot = row >> p.B_log2, in_slot = row & ((1 << p.B_log2) - 1);
    y = static_cast<T*>(keys ? p.k_pages : p.v_pages) + slot * p.slot_stride + in_slot * (static_cast<int64_t>(p.H) * p.d);
    if (!keys) {
      const int h0 = part * p.heads_per_warp, h1 = min(h0 + p.heads_per_warp, heads);
      const int pieces = p.d / V, total = (h1 - h0) * pieces;  // pieces of a row: a power of two
      constexpr int kUnroll = 4;
      bool allowed = false, asked = false;
      for (int first = lane; first < total + lane; first += 32 * kUnroll) {  // the same for all lanes
        Piece<T, V> a[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int i = first + u * 32;
          if (i < total) a[u] = load_piece<T, V>(x + (h0 + i / pieces) * x_head + (i & (pieces - 1)) * V);
        }
        if (!asked) {
          const bool pos_ok = positions_exist(p.rope, t, lane);
          allowed = pos_ok && row_ok && row >= 0;
          asked = true;
          if (lane == 0) flag_error(p.err, (pos_ok ? 0 : HC_DEVERR_POS) | (row_ok ? 0 : HC_DEVERR_SLOT));
        }
        if (!allowed) return;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int i = first + u * 32;
          if (i < total) store_piece<T, V>(y + (h0 + i / pieces) * y_head + (i & (pieces - 1)) * V, a[u]);
        }
      }
      return;
    }
  }
  const bool writes = row_ok && (part_of < static_cast<uint32_t>(p.q_parts) || row >= 0);
  if (!row_ok && lane == 0) flag_error(p.err, HC_DEVERR_SLOT);
  const int h0 = part * p.heads_per_warp, h1 = min(h0 + p.heads_per_warp, heads);
  bool ok;
  if constexpr (kInLanes) {
    ok = rotate_rows_in_lanes<T, kPairing, V>(p.rope, static_cast<int>(t), x, x_head, y, y_head, h0, h1,
                                              static_cast<int>(p.items_per_row.d), lane, [&] { return writes; });
  } else {
    __shared__ float2 cs[kRopeWarps][64];
    ok = stage_cos_sin(p.rope, static_cast<int>(t), lane, cs[warp]);
    if (ok && writes)
      rotate_rows<T, kPairing, V, 4>(x, x_head, y, y_head, h0, h1, p.rope.half, cs[warp], p.items_per_row, lane);
  }
  if (!ok && lane == 0) flag_error(p.err, HC_DEVERR_POS);
}

template <typename T, int kPairing>
cudaError_t launch(AppendPagedParams p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int items = rope_items<kPairing, V>(p.rope.half, p.d);
  p.items_per_row = FastDivmod(static_cast<uint32_t>(items));
  const bool in_lanes = items <= 32 && 32 % items == 0;
  p.heads_per_warp = heads_per_warp(p.n_tokens, p.n_q_heads + 2 * p.H, items, in_lanes);
  p.q_parts = (p.n_q_heads + p.heads_per_warp - 1) / p.heads_per_warp;
  p.kv_parts = (p.H + p.heads_per_warp - 1) / p.heads_per_warp;
  p.parts = FastDivmod(static_cast<uint32_t>(p.q_parts + 2 * p.kv_parts));
  const int64_t warps = static_cast<int64_t>(p.n_tokens) * p.parts.d;
  const unsigned grid = static_cast<unsigned>((warps + kRopeWarps - 1) / kRopeWarps);
  if (in_lanes)
    k_append_paged<T, kPairing, true><<<grid, kRopeWarps * 32, 0, s>>>(p);
  else
    k_append_paged<T, kPairing, false><<<grid, kRopeWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_dtype(int pairing, const AppendPagedParams& p, cudaStream_t s) {
  return pairing == HC_PAIR_HALF_SPLIT ? launch<T, HC_PAIR_HALF_SPLIT>(p, s) : launch<T, HC_PAIR_INTERLEAVED>(p, s);
}

}  // namespace

cudaError_t launch_append_paged(int dtype, int pairing, const AppendPagedParams& p, cudaStream_t s) {
  switch (dtype) {
    case HC_F32: return launch_dtype<float>(pairing, p, s);
    case HC_F16: return launch_dtype<__half>(pairing, p, s);
    default: return launch_dtype<__nv_bfloat16>(pairing, p, s);
  }
}

}  // namespace hc
