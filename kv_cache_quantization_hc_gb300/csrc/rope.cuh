// Device pieces of the rotation by positions with several axes, shared by
// hc_rope_axes and hc_append_int4.
//
// A pair (x1, x2) turns by (c, s): y1 = x1*c - x2*s, y2 = x1*s + x2*c, each
// product and sum rounded to fp32 on its own (no fused multiply-add), so that
// the result is one definite value per input: the appended codes depend on
// it bit by bit.
#pragma once

#include <algorithm>

#include "serve.cuh"

namespace hc {
namespace {

constexpr int kRopeWarps = 8;

// (cos, sin) of every pair for token t, by one warp into cs[half]; false if
// a position is outside the table (nothing is read for it then).
__device__ __forceinline__ bool stage_cos_sin(const RopeParams& p, int t, int lane, float2* cs) {
  bool ok = true;
  for (int i = lane; i < p.half; i += 32) {
    const int pos = __ldg(p.positions + p.pair_axis[i] * p.position_stride + t);
    const bool in = pos >= 0 && pos < p.n_positions;
    ok = ok && in;
    if (in) {
      float2 v = __ldg(p.table + static_cast<int64_t>(pos) * p.half + i);
      if (p.inverse) v.y = -v.y;
      cs[i] = v;
    }
  }
  ok = __all_sync(0xffffffffu, ok);
  __syncwarp();
  return ok;
}

__device__ __forceinline__ void turn(float& x1, float& x2, float2 cs) {
  const float y1 = __fsub_rn(__fmul_rn(x1, cs.x), __fmul_rn(x2, cs.y));
  const float y2 = __fadd_rn(__fmul_rn(x1, cs.y), __fmul_rn(x2, cs.x));
  x1 = y1;
  x2 = y2;
}

template <typename T>
__device__ __forceinline__ float to_f32(T x) { return static_cast<float>(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// V consecutive elements, moved as one 16-byte word (V * sizeof(T) == 16) or
// one by one (V small).
template <typename T, int V>
struct Piece {
  T e[V];
};
template <typename T, int V>
__device__ __forceinline__ Piece<T, V> load_piece(const T* p) {
  Piece<T, V> r;
  if constexpr (V * sizeof(T) == 16) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    memcpy(&r, &w, 16);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.e[i] = p[i];
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_piece(T* p, const Piece<T, V>& r) {
  if constexpr (V * sizeof(T) == 16) {
    uint4 w;
    memcpy(&w, &r, 16);
    *reinterpret_cast<uint4*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = r.e[i];
  }
}

// A lane's position of token t, of the axis that is its number: as it is
// stored, so positions_exist is asked before turns_at reads the table there.
__device__ __forceinline__ int lane_position(const RopeParams& p, int t, int lane) {
  return p.axes >> lane & 1u ? __ldg(p.positions + lane * p.position_stride + t) : 0;
}
// False if a position that some pair needs is outside the table.  Called by whole warps.
__device__ __forceinline__ bool positions_exist(const RopeParams& p, int pos, int lane) {
  return __all_sync(0xffffffffu, !(p.axes >> lane & 1u) || (pos >= 0 && pos < p.n_positions));
}
// The axes of pairs first..first+N-1, which differ from lane to lane: a kernel
// that takes several tokens looks them up once.  Called by whole warps.
template <int N>
struct PairAxes {
  uint32_t axis[N];
  bool same;  // for every lane, all its pairs have one axis
  __device__ __forceinline__ PairAxes(const RopeParams& p, int first, bool rotates) {
    same = true;
    // 4 bytes at a time (N and first are even, or N is 1)
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint32_t w = rotates ? *reinterpret_cast<const uint32_t*>(p.pair_axis + first + i) : 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) axis[i + j] = __byte_perm(w, 0, 0x4440 + j);
        same = same && w == axis[0] * 0x01010101u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        axis[i] = rotates ? p.pair_axis[first + i] : 0u;
        same = same && axis[i] == axis[0];
      }
    }
    same = N % 2 == 0 && p.pairs16 && __all_sync(0xffffffffu, same);
  }
};
// (cos, sin) of these pairs at the lanes' positions, which exist, in registers.
template <int N>
__device__ __forceinline__ void turns_at(const RopeParams& p, const PairAxes<N>& axes, int pos, int first, bool rotates,
                                         float2 (&cs)[N]) {
  if (axes.same) {
    const int at = __shfl_sync(0xffffffffu, pos, axes.axis[0]);
    if (rotates) {
      const float4* src = reinterpret_cast<const float4*>(p.table + static_cast<int64_t>(at) * p.half + first);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float4 v = __ldg(src + i);
        cs[2 * i] = make_float2(v.x, v.y);
        cs[2 * i + 1] = make_float2(v.z, v.w);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = __shfl_sync(0xffffffffu, pos, axes.axis[i]);
      if (rotates) cs[i] = __ldg(p.table + static_cast<int64_t>(at) * p.half + first + i);
    }
  }
  if (p.inverse) {
#pragma unroll
    for (int i = 0; i < N; ++i) cs[i].y = -cs[i].y;
  }
}
// The same for token t; false if a position is outside the table (nothing is read for it then).
template <int N>
__device__ __forceinline__ bool load_turns(const RopeParams& p, int t, int first, bool rotates, int lane,
                                           float2 (&cs)[N]) {
  const int pos = lane_position(p, t, lane);
  if (!positions_exist(p, pos, lane)) return false;
  turns_at(p, PairAxes<N>(p, first, rotates), pos, first, rotates, cs);
  return true;
}

// A piece's elements as floats, and floats as a piece: 16-bit elements two at a time.
template <typename T, int V>
__device__ __forceinline__ void widen_piece(const Piece<T, V>& a, float (&x)[V]) {
  if constexpr (sizeof(T) == 2 && V % 2 == 0) {
    uint32_t w[V / 2];
    memcpy(w, &a, sizeof w);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 f = u32_to_float2(w[i], static_cast<const T*>(nullptr));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f32(a.e[i]);
  }
}
__device__ __forceinline__ uint32_t narrow2(float a, float b, const __half*) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ uint32_t narrow2(float a, float b, const __nv_bfloat16*) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
template <typename T, int V>
__device__ __forceinline__ void narrow_piece(const float (&x)[V], Piece<T, V>& a) {
  if constexpr (sizeof(T) == 2 && V % 2 == 0) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = narrow2(x[2 * i], x[2 * i + 1], static_cast<const T*>(nullptr));
    memcpy(&a, w, sizeof w);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) a.e[i] = from_f32<T>(x[i]);
  }
}

// Items of one row: its rotated pieces (half split: the piece of V pairs at
// channels V*i.. and half+V*i..; interleaved: V channels, V/2 pairs), then
// the pieces that are copied.
template <int kPairing, int V>
__host__ __device__ constexpr int rope_items(int half, int d) {
  return (kPairing == HC_PAIR_HALF_SPLIT ? half / V : 2 * half / V) + (d - 2 * half) / V;
}

// The rows of heads [h0, h1) of one token, by one warp.  kUnroll items per
// lane are loaded before the first is stored.
template <typename T, int kPairing, int V, int kUnroll>
__device__ __forceinline__ void rotate_rows(const T* x, int64_t x_head, T* y, int64_t y_head, int h0,
                                            int h1, int half, const float2* cs,
                                            const FastDivmod& items_per_row, int lane) {
  const int turned = kPairing == HC_PAIR_HALF_SPLIT ? half / V : 2 * half / V;
  const int total = (h1 - h0) * static_cast<int>(items_per_row.d);
  for (int base = lane; base < total; base += 32 * kUnroll) {
    Piece<T, V> a[kUnroll], b[kUnroll];
    int item[kUnroll];
    int64_t yo[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int idx = base + 32 * u;
      item[u] = -1;
      if (idx < total) {
        uint32_t h, it;
        items_per_row.divmod(static_cast<uint32_t>(idx), h, it);
        item[u] = static_cast<int>(it);
        const int c = item[u] < turned || kPairing != HC_PAIR_HALF_SPLIT ? item[u] * V
                                                                         : 2 * half + (item[u] - turned) * V;
        const int64_t head = h0 + static_cast<int>(h);
        yo[u] = head * y_head + c;
        a[u] = load_piece<T, V>(x + head * x_head + c);
        if (kPairing == HC_PAIR_HALF_SPLIT && item[u] < turned)
          b[u] = load_piece<T, V>(x + head * x_head + c + half);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (item[u] < 0) continue;
      if (item[u] < turned) {
        if constexpr (kPairing == HC_PAIR_HALF_SPLIT) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float x1 = to_f32(a[u].e[i]), x2 = to_f32(b[u].e[i]);
            turn(x1, x2, cs[item[u] * V + i]);
            a[u].e[i] = from_f32<T>(x1);
            b[u].e[i] = from_f32<T>(x2);
          }
          store_piece<T, V>(y + yo[u] + half, b[u]);
        } else {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            float x1 = to_f32(a[u].e[2 * i]), x2 = to_f32(a[u].e[2 * i + 1]);
            turn(x1, x2, cs[item[u] * (V / 2) + i]);
            a[u].e[2 * i] = from_f32<T>(x1);
            a[u].e[2 * i + 1] = from_f32<T>(x2);
          }
        }
      }
      store_piece<T, V>(y + yo[u], a[u]);
    }
  }
}

// Passes over rows that a warp loads at once, and heads for a warp to take:
// where the rows are in lanes, one such load, so that nothing waits twice.
// hc_append_int4's queries gain by that (76 us to 72 with their read-back);
// hc_rope_axes, which has nothing else to do meanwhile, asks for as many heads as
// keep the SMs busy (1369 x 40 rows: 8.1 us, 10.2 with one load).
constexpr int kRowsAhead = 4;
inline int heads_per_warp(int n_tokens, int heads, int items, bool in_lanes) {
  if (heads < 1) return 1;
  int most = heads;
  if (in_lanes) most = std::min(heads, kRowsAhead * (32 / items));
  // few tokens: shared out until the GPU has the 16 warps per SM that k_rope_axes' registers let in (24: 8.8 us
  // instead of 8.1 for 1369 x 40 rows), or a warp has no more than an item per lane
  const int64_t enough = int64_t{device_sm_count()} * 16;
  while (most > 1 && static_cast<int64_t>(most) * items > 32 &&
         static_cast<int64_t>(n_tokens) * ((heads + most - 1) / most) < enough)
    most = (most + 1) / 2;
  return most;
}

// Rows whose items divide a warp's lanes: a lane has the same item of every
// row it takes, so its (cos, sin) stay in registers.
template <typename T, int kPairing, int V>
struct LaneItem {
  static constexpr bool kHalfSplit = kPairing == HC_PAIR_HALF_SPLIT;
  static constexpr int kPairs = kHalfSplit ? V : V / 2;  // of an item
  int it, sub, at_once;  // the item, the row among those of a pass, rows of a pass
  bool rotates;
  int c, half;           // the item's first channel; half-split: its second piece is `half` further on

  __device__ __forceinline__ LaneItem(int lane, int items, int half_) {
    it = lane & (items - 1);
    at_once = 32 / items;
    sub = lane / items;
    half = half_;
    const int turned = kHalfSplit ? half / V : 2 * half / V;
    rotates = it < turned;
    c = rotates || !kHalfSplit ? it * V : 2 * half + (it - turned) * V;
  }
  __device__ __forceinline__ int first_pair() const { return it * kPairs; }
  __device__ __forceinline__ void load(const T* row, Piece<T, V>& a, Piece<T, V>& b) const {
    a = load_piece<T, V>(row + c);
    if (kHalfSplit && rotates) b = load_piece<T, V>(row + c + half);
  }
  __device__ __forceinline__ void turn_and_store(T* row, Piece<T, V>& a, Piece<T, V>& b, const float2 (&cs)[kPairs]) const {
    if (rotates) {
      float x[V], x2[V];
      widen_piece(a, x);
      if (kHalfSplit) widen_piece(b, x2);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) turn(kHalfSplit ? x[i] : x[2 * i], kHalfSplit ? x2[i] : x[2 * i + 1], cs[i]);
      narrow_piece(x, a);
      if (kHalfSplit) {
        narrow_piece(x2, b);
        store_piece<T, V>(row + c + half, b);
      }
    }
    store_piece<T, V>(row + c, a);
  }
};

// The rows of heads [h0, h1) of token t.  The first rows are on their way
// before the positions and the table are read, and before `allowed` is asked
// whether to go on.  False: a position outside.
template <typename T, int kPairing, int V, typename Allowed>
__device__ __forceinline__ bool rotate_rows_in_lanes(const RopeParams& rope, int t, const T* x, int64_t x_head, T* y,
                                                     int64_t y_head, int h0, int h1, int items, int lane,
                                                     const Allowed& allowed) {
  constexpr int kUnroll = kRowsAhead;
  using Item = LaneItem<T, kPairing, V>;
  const Item item(lane, items, rope.half);
  Piece<T, V> a[kUnroll], b[kUnroll];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + u * item.at_once < h1) item.load(x + (h + u * item.at_once) * x_head, a[u], b[u]);
  };
  int h = h0 + item.sub;
  load(h);
  float2 cs[Item::kPairs];
  if (rope.table != nullptr && !load_turns<Item::kPairs>(rope, t, item.first_pair(), item.rotates, lane, cs)) return false;
  if (!allowed()) return true;
  for (;;) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + u * item.at_once < h1) item.turn_and_store(y + (h + u * item.at_once) * y_head, a[u], b[u], cs);
    h += kUnroll * item.at_once;
    if (h0 + (h - h0 - item.sub) >= h1) return true;  // the same for all lanes
    load(h);
  }
}

}  // namespace
}  // namespace hc
