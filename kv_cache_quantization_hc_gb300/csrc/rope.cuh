// Device pieces of the rotation by positions with several axes, shared by
// hc_rope_axes and hc_append_int4.
//
// A pair (x1, x2) turns by (c, s): y1 = x1*c - x2*s, y2 = x1*s + x2*c, each
// product and sum rounded to fp32 on its own (no fused multiply-add), so that
// the result is one definite value per input: the appended codes depend on
// it bit by bit.
#pragma once

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

// (cos, sin) of pairs first..first+N-1 for token t, in registers; false if a
// position that some pair needs is outside the table (nothing is read for it).
// Called by whole warps with N pairs for each lane.
template <int N>
__device__ __forceinline__ bool load_turns(const RopeParams& p, int t, int first, bool rotates, int lane,
                                           float2 (&cs)[N]) {
  int pos = 0;
  bool ok = true;
  if (p.axes >> lane & 1u) {  // a lane per axis
    pos = __ldg(p.positions + lane * p.position_stride + t);
    ok = pos >= 0 && pos < p.n_positions;
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) return false;
  uint8_t axis[N];
  bool same = true;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    axis[i] = rotates ? p.pair_axis[first + i] : 0;
    same = same && axis[i] == axis[0];
  }
  if (N % 2 == 0 && p.pairs16 && __all_sync(0xffffffffu, same)) {
    const int at = __shfl_sync(0xffffffffu, pos, axis[0]);
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
      const int at = __shfl_sync(0xffffffffu, pos, axis[i]);
      if (rotates) cs[i] = __ldg(p.table + static_cast<int64_t>(at) * p.half + first + i);
    }
  }
  if (p.inverse) {
#pragma unroll
    for (int i = 0; i < N; ++i) cs[i].y = -cs[i].y;
  }
  return true;
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
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        T& e1 = kHalfSplit ? a.e[i] : a.e[2 * i];
        T& e2 = kHalfSplit ? b.e[i] : a.e[2 * i + 1];
        float x1 = to_f32(e1), x2 = to_f32(e2);
        turn(x1, x2, cs[i]);
        e1 = from_f32<T>(x1);
        e2 = from_f32<T>(x2);
      }
      if (kHalfSplit) store_piece<T, V>(row + c + half, b);
    }
    store_piece<T, V>(row + c, a);
  }
};

// The rows of heads [h0, h1) of token t.  The first rows are on their way
// before the positions and the table are read.  False: a position outside.
template <typename T, int kPairing, int V, int kUnroll>
__device__ __forceinline__ bool rotate_rows_in_lanes(const RopeParams& rope, int t, const T* x, int64_t x_head, T* y,
                                                     int64_t y_head, int h0, int h1, int items, int lane) {
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
