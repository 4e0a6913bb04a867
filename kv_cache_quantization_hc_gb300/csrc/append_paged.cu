// The new tokens into the paged buffer: queries and keys rotated, values
// copied, in one launch.  Memory-bound: q, k, v read once, q_out and the
// buffer's rows written once.
//
// A warp takes some heads of a token's queries, keys or values, and the same
// heads of later tokens.  A lane has the same pieces of every row (lanes are
// left over where a partial rotation's pieces are no power of two), so what it
// needs of (cos, sin) is in registers, and the next token's rows are on their
// way while this one's are turned.
//
// 8197 tokens of 32 query and 8 cache heads of 128 channels, of 30 us that the bytes
// take at the copy rate (fp32 60):
//                                 fp16   bf16   fp32
//   interleaved pairs               43     56     72
//   half a rotation apart           53     59     72
//   the same, 96 channels of 128    83     91    106
// fp16 is bound by latency: a token's positions, then its (cos, sin), then 400
// instructions, by 16 warps an SM (122 and 124 registers; 24 warps at 80 spill: 57 us
// instead of 43; half as many rows in hand, 46 to 75).  A warp for each token,
// without the next one's rows on their way: 45 us.  bf16 has the same loads but takes
// all 128 registers and spills 40 and 44 bytes; fp32 takes 108 and 104.
#include <algorithm>

#include "paged.cuh"
#include "rope.cuh"

namespace hc {
namespace {

// Rows that a lane has in hand of a token: 16 registers of them, as many again of the next token's.
template <int kPairing>
constexpr int kRowsInHand = kPairing == HC_PAIR_HALF_SPLIT ? 2 : 4;

// Some heads of the queries, keys or values: where they are, where they go, and whether they turn.
template <typename T>
struct Part {
  const T* from;
  T* to;
  int64_t from_token, from_head, to_head;
  int h0, h1;
  bool queries, turns;
};
template <typename T>
__device__ __forceinline__ Part<T> part_of(const AppendPagedParams& p, int part) {
  Part<T> w;
  w.queries = part < p.q_parts;
  const bool keys = !w.queries && part < p.q_parts + p.kv_parts;
  w.turns = p.rope.table != nullptr && (w.queries || keys);
  part -= w.queries ? 0 : keys ? p.q_parts : p.q_parts + p.kv_parts;
  w.h0 = part * p.heads_per_warp;
  w.h1 = min(w.h0 + p.heads_per_warp, w.queries ? p.n_q_heads : p.H);
  w.from = static_cast<const T*>(w.queries ? p.q : keys ? p.k : p.v);
  w.to = static_cast<T*>(w.queries ? p.q_out : keys ? p.k_pages : p.v_pages);
  w.from_token = w.queries ? p.q_token : keys ? p.k_token : p.v_token;
  w.from_head = w.queries ? p.q_head : keys ? p.k_head : p.v_head;
  w.to_head = w.queries ? p.o_head : p.d;
  return w;
}
// Where a token's rows of a part go, given its row in the pages, which exists.
template <typename T>
__device__ __forceinline__ T* destination(const AppendPagedParams& p, const Part<T>& w, int64_t t, int64_t row) {
  if (w.queries) return w.to + t * p.o_token;
  return w.to + (row >> p.B_log2) * p.slot_stride + (row & ((1 << p.B_log2) - 1)) * (static_cast<int64_t>(p.H) * p.d);
}

template <typename T, int kPairing>
__global__ void __launch_bounds__(kRopeWarps * 32, 2) k_append_paged(const __grid_constant__ AppendPagedParams p) {
  constexpr int V = 16 / sizeof(T), R = kRowsInHand<kPairing>;
  constexpr bool kSplit = kPairing == HC_PAIR_HALF_SPLIT;
  using Item = LaneItem<T, kPairing, V>;
  const int lane = threadIdx.x & 31;
  uint32_t first, part;
  p.parts.divmod(blockIdx.x * kRopeWarps + (threadIdx.x >> 5), first, part);
  if (first >= static_cast<uint32_t>(p.token_step)) return;
  const Part<T> w = part_of<T>(p, static_cast<int>(part));
  const Item item(lane, p.lanes_per_row, p.rope.half);
  const PairAxes<Item::kPairs> axes(p.rope, item.first_pair(), item.rotates);
  const T* const from = w.from + (w.h0 + item.sub) * w.from_head + item.c;
  const int heads = item.it < p.items ? w.h1 - w.h0 - item.sub : 0;  // of this lane, every at_once-th
  struct {
    Piece<T, V> a[R], b[R];
    int64_t row;
    int pos;
  } in[2];
  auto fetch = [&](auto& to, int64_t t) {
    const T* x = from + t * w.from_token;
#pragma unroll
    for (int u = 0; u < R; ++u)
      if (u * item.at_once < heads) {
        to.a[u] = load_piece<T, V>(x + u * item.at_once * w.from_head);
        if (kSplit && item.rotates) to.b[u] = load_piece<T, V>(x + u * item.at_once * w.from_head + item.half);
      }
    to.row = __ldg(p.token_rows + t);
    to.pos = p.rope.table != nullptr ? lane_position(p.rope, static_cast<int>(t), lane) : 0;
  };
  int64_t t = first;
  fetch(in[0], t);
  for (;;) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      auto& now = in[s];
      if (t + p.token_step < p.n_tokens) fetch(in[s ^ 1], t + p.token_step);
      const bool known = p.rope.table == nullptr || positions_exist(p.rope, now.pos, lane);
      const bool exists = now.row >= -1 && now.row < p.n_rows;
      if (lane == 0) flag_error(p.err, (known ? 0 : HC_DEVERR_POS) | (exists ? 0 : HC_DEVERR_SLOT));
      if (known && exists && (w.queries || now.row >= 0)) {
        float2 cs[Item::kPairs];
        if (w.turns) turns_at(p.rope, axes, now.pos, item.first_pair(), item.rotates, cs);
        T* y = destination(p, w, t, now.row) + (w.h0 + item.sub) * w.to_head + item.c;
#pragma unroll
        for (int u = 0; u < R; ++u)
          if (u * item.at_once < heads) {
            T* to = y + u * item.at_once * w.to_head;
            if (w.turns && item.rotates) {
              float x[V], x2[V];
              widen_piece(now.a[u], x);
              if (kSplit) widen_piece(now.b[u], x2);
#pragma unroll
              for (int i = 0; i < Item::kPairs; ++i)
                turn(kSplit ? x[i] : x[2 * i], kSplit ? x2[i] : x[2 * i + 1], cs[i]);
              narrow_piece(x, now.a[u]);
              if (kSplit) narrow_piece(x2, now.b[u]);
            }
            store_piece<T, V>(to, now.a[u]);
            if (kSplit && item.rotates) store_piece<T, V>(to + item.half, now.b[u]);
          }
      }
      t += p.token_step;
      if (t >= p.n_tokens) return;
    }
  }
}

template <typename T, int kPairing>
cudaError_t launch(AppendPagedParams p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  p.items = rope_items<kPairing, V>(p.rope.half, p.d);
  p.lanes_per_row = 1;
  while (p.lanes_per_row < p.items) p.lanes_per_row *= 2;  // at most 32: of 128 fp32 channels
  p.heads_per_warp = std::min(std::max(p.n_q_heads, p.H), kRowsInHand<kPairing> * (32 / p.lanes_per_row));
  p.q_parts = (p.n_q_heads + p.heads_per_warp - 1) / p.heads_per_warp;
  p.kv_parts = (p.H + p.heads_per_warp - 1) / p.heads_per_warp;
  p.parts = FastDivmod(static_cast<uint32_t>(p.q_parts + 2 * p.kv_parts));
  // as many warps as the device holds at once, each with every token_step-th token
  static KernelOnDevice kernel;
  int resident = 0;
  const cudaError_t e =
      kernel.resident(reinterpret_cast<const void*>(k_append_paged<T, kPairing>), kRopeWarps * 32, 0, &resident);
  if (e != cudaSuccess) return e;
  p.token_step = static_cast<int32_t>(
      std::min<int64_t>(p.n_tokens, std::max<int64_t>(1, int64_t{resident} * kRopeWarps / p.parts.d)));
  const int64_t warps = static_cast<int64_t>(p.token_step) * p.parts.d;
  const unsigned grid = static_cast<unsigned>((warps + kRopeWarps - 1) / kRopeWarps);
  k_append_paged<T, kPairing><<<grid, kRopeWarps * 32, 0, s>>>(p);
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
