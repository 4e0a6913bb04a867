// The new tokens into the 4-bit cache: queries rotated, keys rotated and
// quantized, values quantized, in one launch.  Memory-bound: q, k, v read
// once, q_out and the 4-bit rows written once.
//
// A warp takes either some query heads of a token (as k_rope_axes) or some of
// its cache heads.  Where all channels rotate (or none), a lane has whole
// pieces of 16 bytes of a row before and after the rotation (channels i.. and
// i + half..): it quantizes them where they are, the group's maximum found by
// shuffles.  A partial rotation shifts pieces against groups; such keys go
// through shared memory in fp32 first, which takes 62 us where this takes 49
// (the case below).
//
// A code is fp32(x / s) rounded: the quotient as x * r corrected by its exact
// residual, r = fp32(1 / s) correctly rounded (Markstein, IBM J. Res. Dev.
// 34(1), 1990), which gives the IEEE quotient where nothing under- or overflows;
// scales outside 2^-100..2^100 are divided by.
//
// 8197 tokens of 32 query and 8 cache heads of 128 fp16 channels: 48 us of 17
// that the bytes take; about 3500 instructions a token, 24 warps an SM.
#include <algorithm>
#include <type_traits>

#include "div7.cuh"
#include "rope.cuh"

namespace hc {
namespace {

// Cache heads per warp: a row of values takes 8 to 32 lanes, a row of keys as
// many or half of that.
template <int D>
constexpr int kKvHeads = 512 / D;

// The codes of N values, a nibble each from the lowest on.
template <int N>
__device__ __forceinline__ uint32_t codes_of(const float (&x)[N], float s) {
  uint32_t packed = 0;
  float q[N];
  if (s >= 0x1p-100f && s <= 0x1p100f) {
    const float r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      q[i] = x[i] * r;
      q[i] = fmaf(fmaf(-q[i], s, x[i]), r, q[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = s != 0.f ? __fdiv_rn(x[i], s) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    // 1.5 * 2^23 more: rounded to even, the two's complement in the low bits
    const uint32_t n = __float_as_uint(fminf(fmaxf(q[i], -7.f), 7.f) + 12582912.f);
    packed |= (n & 0xfu) << (4 * i);
  }
  return packed;
}

// `wire`: the encoders' amax / 7, which differs from the product in the last bit of some fp32 scales.
template <bool kScaleF16>
__device__ __forceinline__ float scale_of(float amax, int wire) {
  const float s = wire ? div7(amax) : __fmul_rn(amax, 0x1.24924ap-3f);  // fp32(1/7)
  return kScaleF16 ? __half2float(__float2half_rn(s)) : s;
}
template <bool kScaleF16>
__device__ __forceinline__ void store_scale(void* scales, int64_t i, float s) {
  if (kScaleF16)
    static_cast<__half*>(scales)[i] = __float2half_rn(s);
  else
    static_cast<float*>(scales)[i] = s;
}
template <int N>
__device__ __forceinline__ float amax_of(const float (&x)[N]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, fabsf(x[i]));
  return m;
}
// The largest over runs of `lanes` lanes (a power of two).
__device__ __forceinline__ float amax_over(float m, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* codes, int channel, uint32_t packed) {
  if (N == 8)
    *reinterpret_cast<uint32_t*>(codes + channel / 2) = packed;
  else
    *reinterpret_cast<uint16_t*>(codes + channel / 2) = static_cast<uint16_t>(packed);
}

// A row's codes and scales in the cache.
struct CacheRow {
  uint8_t* codes;
  int64_t scale;  // index of its first scale
};
template <int D>
__device__ __forceinline__ CacheRow cache_row(const AppendParams& p, int64_t row, int kv, int h) {
  const int64_t at = ((((row >> p.B_log2) * 2 + kv) * p.H + h) << p.B_log2) + (row & ((1 << p.B_log2) - 1));
  return {p.codes + at * (D / 2), at * (D >> p.group_log2)};
}

// One piece of V channels per lane, D / V lanes to a row; `live`: the lane's row is there.
template <int D, bool kScaleF16, int V>
__device__ __forceinline__ void quantize_pieces(const AppendParams& p, const float (&x)[V], int channel, CacheRow to,
                                                bool live) {
  const float s = scale_of<kScaleF16>(amax_over(amax_of(x), (1 << p.group_log2) / V), p.wire_scales);
  const uint32_t packed = codes_of(x, s);
  if (!live) return;
  store_codes<V>(to.codes, channel, packed);
  if ((channel & ((1 << p.group_log2) - 1)) == 0) store_scale<kScaleF16>(p.scales, to.scale + (channel >> p.group_log2), s);
}

template <typename T, int D>
struct AppendShared {
  float2 cs[kRopeWarps][D / 2];
  alignas(16) float rows[kRopeWarps][512];
};
struct NoShared {};

// Three CTAs an SM (80 registers) cover the latency of a chunk's loads better
// than two with the 96 or more registers that some variants would take.
template <typename T, int D, int kPairing, bool kScaleF16, bool kInLanes>
__global__ void __launch_bounds__(kRopeWarps * 32, 3) k_append_int4(const __grid_constant__ AppendParams p) {
  constexpr int V = 16 / sizeof(T);
  __shared__ std::conditional_t<kInLanes, NoShared, AppendShared<T, D>> sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t tok, part_of;
  p.parts.divmod(blockIdx.x * kRopeWarps + warp, tok, part_of);
  if (tok >= static_cast<uint32_t>(p.n_tokens)) return;
  const int64_t t = tok;
  const int part = static_cast<int>(part_of);
  // asked after the data is on its way: what is read is there whatever the row says
  const int64_t row = __ldg(p.token_rows + t);
  auto row_exists = [&] {
    const bool ok = row >= -1 && row < p.n_rows;
    if (!ok && lane == 0) flag_error(p.err, HC_DEVERR_SLOT);
    return ok;
  };
  if (part < p.q_parts) {
    const int h0 = part * p.q_heads_per_warp, h1 = min(h0 + p.q_heads_per_warp, p.n_q_heads);
    const T* q = static_cast<const T*>(p.q) + t * p.q_token;
    T* q_out = static_cast<T*>(p.q_out) + t * p.o_token;
    bool ok;
    if constexpr (kInLanes) {
      ok = rotate_rows_in_lanes<T, kPairing, V>(p.rope, static_cast<int>(t), q, p.q_head, q_out, p.o_head, h0, h1,
                                                static_cast<int>(p.items_per_row.d), lane, row_exists);
    } else {
      ok = stage_cos_sin(p.rope, static_cast<int>(t), lane, sh.cs[warp]);
      if (ok && row_exists())
        rotate_rows<T, kPairing, V, 4>(q, p.q_head, q_out, p.o_head, h0, h1, p.rope.half, sh.cs[warp], p.items_per_row, lane);
    }
    if (!ok && lane == 0) flag_error(p.err, HC_DEVERR_POS);
    return;
  }
  const int h0 = (part - p.q_parts) * kKvHeads<D>, nh = min(kKvHeads<D>, p.H - h0);
  const T* k = static_cast<const T*>(p.k) + t * p.k_token + h0 * p.k_head;
  const T* v = static_cast<const T*>(p.v) + t * p.v_token + h0 * p.v_head;
  constexpr int kLanes = D / V, kAt = 32 / kLanes;  // lanes of a row of values, rows at a time
  const int piece = lane % kLanes;
  // values: on their way before the keys are worked on (rows past the last repeat it and are not stored)
  Piece<T, V> vp[kKvHeads<D> / kAt];
#pragma unroll
  for (int u = 0; u < kKvHeads<D> / kAt; ++u)
    vp[u] = load_piece<T, V>(v + min(u * kAt + lane / kLanes, nh - 1) * p.v_head + piece * V);

  if constexpr (kInLanes) {
    using Item = LaneItem<T, kPairing, V>;
    const Item item(lane, static_cast<int>(p.items_per_row.d), p.rope.half);
    constexpr int kItemLanes = kPairing == HC_PAIR_HALF_SPLIT ? D / 2 / V : D / V, kRowsAt = 32 / kItemLanes;
    constexpr bool kSplit = kPairing == HC_PAIR_HALF_SPLIT;
    if (p.rope.table != nullptr) {
      Piece<T, V> a[(kKvHeads<D> + kRowsAt - 1) / kRowsAt], b[(kKvHeads<D> + kRowsAt - 1) / kRowsAt];
#pragma unroll
      for (int u = 0; u < (kKvHeads<D> + kRowsAt - 1) / kRowsAt; ++u)
        item.load(k + min(u * kRowsAt + item.sub, nh - 1) * p.k_head, a[u], b[u]);
      float2 cs[Item::kPairs];
      if (!load_turns<Item::kPairs>(p.rope, static_cast<int>(t), item.first_pair(), true, lane, cs)) {
        if (lane == 0) flag_error(p.err, HC_DEVERR_POS);
        return;
      }
      if (!row_exists() || row < 0) return;
#pragma unroll
      for (int u = 0; u < (kKvHeads<D> + kRowsAt - 1) / kRowsAt; ++u) {
        const int r = u * kRowsAt + item.sub;
        const bool live = r < nh;
        const CacheRow to = cache_row<D>(p, row, 0, h0 + (live ? r : 0));
        float x[V], x2[V];
        widen_piece(a[u], x);
        if (kSplit) widen_piece(b[u], x2);
#pragma unroll
        for (int i = 0; i < Item::kPairs; ++i) {
          if (kSplit)
            turn(x[i], x2[i], cs[i]);
          else
            turn(x[2 * i], x[2 * i + 1], cs[i]);
        }
        if (!kSplit) {
          quantize_pieces<D, kScaleF16, V>(p, x, item.c, to, live);
        } else {
          // channels c.. and c + D/2..: in groups of their own, or the same one
          const bool one = (1 << p.group_log2) > D / 2;
          const int lanes = one ? kItemLanes : (1 << p.group_log2) / V;
          float m1 = amax_of(x), m2 = amax_of(x2);
          if (one) m1 = fmaxf(m1, m2);
          m1 = amax_over(m1, lanes);
          m2 = one ? m1 : amax_over(m2, lanes);
          const float s1 = scale_of<kScaleF16>(m1, p.wire_scales), s2 = one ? s1 : scale_of<kScaleF16>(m2, p.wire_scales);
          const uint32_t c1 = codes_of(x, s1), c2 = codes_of(x2, s2);
          if (live) {
            store_codes<V>(to.codes, item.c, c1);
            store_codes<V>(to.codes, item.c + D / 2, c2);
            if ((item.it & (lanes - 1)) == 0) {
              store_scale<kScaleF16>(p.scales, to.scale + (item.c >> p.group_log2), s1);
              if (!one) store_scale<kScaleF16>(p.scales, to.scale + ((item.c + D / 2) >> p.group_log2), s2);
            }
          }
        }
      }
    } else {
      if (!row_exists() || row < 0) return;
#pragma unroll
      for (int u = 0; u < kKvHeads<D> / kAt; ++u) {
        const int r = u * kAt + lane / kLanes;
        const bool live = r < nh;
        float x[V];
        widen_piece(load_piece<T, V>(k + min(r, nh - 1) * p.k_head + piece * V), x);
        quantize_pieces<D, kScaleF16, V>(p, x, piece * V, cache_row<D>(p, row, 0, h0 + (live ? r : 0)), live);
      }
    }
  } else {
    // rotated in fp32 into shared memory, converted on the way
    if (!stage_cos_sin(p.rope, static_cast<int>(t), lane, sh.cs[warp])) {
      if (lane == 0) flag_error(p.err, HC_DEVERR_POS);
      return;
    }
    if (!row_exists() || row < 0) return;
    const int total = nh * static_cast<int>(p.items_per_row.d);
    const int half = p.rope.half;
    const int turned = kPairing == HC_PAIR_HALF_SPLIT ? half / V : 2 * half / V;
    for (int idx = lane; idx < total; idx += 32) {
      uint32_t h, it;
      p.items_per_row.divmod(static_cast<uint32_t>(idx), h, it);
      const int item = static_cast<int>(it);
      const int c = item < turned || kPairing != HC_PAIR_HALF_SPLIT ? item * V : 2 * half + (item - turned) * V;
      const T* src = k + h * p.k_head + c;
      float* dst = sh.rows[warp] + h * D + c;
      const Piece<T, V> a = load_piece<T, V>(src);
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = to_f32(a.e[i]);
      if (item < turned) {
        if constexpr (kPairing == HC_PAIR_HALF_SPLIT) {
          const Piece<T, V> b = load_piece<T, V>(src + half);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float x2 = to_f32(b.e[i]);
            turn(f[i], x2, sh.cs[warp][item * V + i]);
            dst[half + i] = x2;
          }
        } else {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) turn(f[2 * i], f[2 * i + 1], sh.cs[warp][item * (V / 2) + i]);
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) dst[i] = f[i];
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < kKvHeads<D> / kAt; ++u) {
      const int r = u * kAt + lane / kLanes;
      const bool live = r < nh;
      float x[V];
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = live ? sh.rows[warp][r * D + piece * V + i] : 0.f;
      quantize_pieces<D, kScaleF16, V>(p, x, piece * V, cache_row<D>(p, row, 0, h0 + (live ? r : 0)), live);
    }
  }
#pragma unroll
  for (int u = 0; u < kKvHeads<D> / kAt; ++u) {
    const int r = u * kAt + lane / kLanes;
    const bool live = r < nh;
    float x[V];
    widen_piece(vp[u], x);
    quantize_pieces<D, kScaleF16, V>(p, x, piece * V, cache_row<D>(p, row, 1, h0 + (live ? r : 0)), live);
  }
}

template <typename T, int D, int kPairing>
cudaError_t launch(AppendParams p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int items = rope_items<kPairing, V>(p.rope.half, D);
  p.items_per_row = FastDivmod(static_cast<uint32_t>(items));
  p.kv_parts = (p.H + kKvHeads<D> - 1) / kKvHeads<D>;
  const bool in_lanes = p.rope.half == 0 || 2 * p.rope.half == D;
  p.q_heads_per_warp = heads_per_warp(p.n_tokens, p.n_q_heads, items, in_lanes);
  p.q_parts = (p.n_q_heads + p.q_heads_per_warp - 1) / p.q_heads_per_warp;
  p.parts = FastDivmod(static_cast<uint32_t>(p.q_parts + p.kv_parts));
  const int64_t warps = static_cast<int64_t>(p.n_tokens) * p.parts.d;
  const unsigned grid = static_cast<unsigned>((warps + kRopeWarps - 1) / kRopeWarps);
  if (in_lanes && p.scale_f16)
    k_append_int4<T, D, kPairing, true, true><<<grid, kRopeWarps * 32, 0, s>>>(p);
  else if (in_lanes)
    k_append_int4<T, D, kPairing, false, true><<<grid, kRopeWarps * 32, 0, s>>>(p);
  else if (p.scale_f16)
    k_append_int4<T, D, kPairing, true, false><<<grid, kRopeWarps * 32, 0, s>>>(p);
  else
    k_append_int4<T, D, kPairing, false, false><<<grid, kRopeWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_dtype(int d, int pairing, const AppendParams& p, cudaStream_t s) {
  if (d == 64)
    return pairing == HC_PAIR_HALF_SPLIT ? launch<T, 64, HC_PAIR_HALF_SPLIT>(p, s)
                                         : launch<T, 64, HC_PAIR_INTERLEAVED>(p, s);
  return pairing == HC_PAIR_HALF_SPLIT ? launch<T, 128, HC_PAIR_HALF_SPLIT>(p, s)
                                       : launch<T, 128, HC_PAIR_INTERLEAVED>(p, s);
}

}  // namespace

cudaError_t launch_append_int4(int dtype, int d, int pairing, const AppendParams& p, cudaStream_t s) {
  switch (dtype) {
    case HC_F32: return launch_dtype<float>(d, pairing, p, s);
    case HC_F16: return launch_dtype<__half>(d, pairing, p, s);
    default: return launch_dtype<__nv_bfloat16>(d, pairing, p, s);
  }
}

}  // namespace hc
