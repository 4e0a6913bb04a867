// The new tokens into the 4-bit cache: queries rotated, keys rotated and
// quantized, values quantized, in one launch.  Memory-bound: q, k, v read
// once, q_out and the 4-bit rows written once.
//
// A warp takes either some query heads of a token (as k_rope_axes) or two
// cache heads of it: their rotated keys go to shared memory in fp32, because
// the rotation's lanes hold channels i and i + half while a quantization
// group is a run of 32 to 128 channels; each lane then quantizes 8 adjacent
// channels, the group's maximum found by shuffles.
#include <algorithm>

#include "rope.cuh"

namespace hc {
namespace {

// Cache heads per warp: as many rows as its lanes hold at 8 channels each.
template <int D>
constexpr int kKvHeads = 256 / D;

// One row of 8 channels per lane (D / 8 lanes): scale and codes.
template <int D, bool kScaleF16>
__device__ __forceinline__ void quantize_row(const float (&x)[8], int lane, int group_log2, uint8_t* codes,
                                             void* scales) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
  for (int o = 1; o < (1 << (group_log2 - 3)); o <<= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  float s = __fmul_rn(amax, 0x1.24924ap-3f);  // fp32(1/7)
  if (kScaleF16) s = __half2float(__float2half_rn(s));
  uint32_t packed = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = s != 0.f ? __fdiv_rn(x[i], s) : 0.f;
    const int n = static_cast<int>(fminf(fmaxf(rintf(q), -7.f), 7.f));
    packed |= (static_cast<uint32_t>(n) & 0xfu) << (4 * i);
  }
  const int piece = lane & (D / 8 - 1);
  reinterpret_cast<uint32_t*>(codes)[piece] = packed;
  if ((piece & ((1 << (group_log2 - 3)) - 1)) == 0) {
    const int g = piece >> (group_log2 - 3);
    if (kScaleF16)
      static_cast<__half*>(scales)[g] = __float2half_rn(s);
    else
      static_cast<float*>(scales)[g] = s;
  }
}

template <typename T, int D, int kPairing, bool kScaleF16>
__global__ void __launch_bounds__(kRopeWarps * 32) k_append_int4(const __grid_constant__ AppendParams p) {
  constexpr int V = 16 / sizeof(T);
  __shared__ float2 cs[kRopeWarps][D / 2];
  __shared__ __align__(16) float rows[kRopeWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp;
  const int parts = p.q_parts + p.kv_parts;
  const int64_t t = w / parts;
  if (t >= p.n_tokens) return;
  const int part = static_cast<int>(w - t * parts);
  const int64_t row = __ldg(p.token_rows + t);
  int bad = row < -1 || row >= p.n_rows ? HC_DEVERR_SLOT : 0;
  if (p.rope.table != nullptr && !stage_cos_sin(p.rope, static_cast<int>(t), lane, cs[warp]))
    bad |= HC_DEVERR_POS;
  if (bad) {
    if (lane == 0) flag_error(p.err, bad);
    return;
  }
  if (part < p.q_parts) {
    const int h0 = part * p.q_heads_per_warp;
    rotate_rows<T, kPairing, V, 4>(static_cast<const T*>(p.q) + t * p.q_token, p.q_head,
                                   static_cast<T*>(p.q_out) + t * p.o_token, p.o_head, h0,
                                   min(h0 + p.q_heads_per_warp, p.n_q_heads), p.rope.half, cs[warp],
                                   p.items_per_row, lane);
    return;
  }
  if (row < 0) return;
  const int h0 = (part - p.q_parts) * kKvHeads<D>, nh = min(kKvHeads<D>, p.H - h0);
  const int64_t slot = row >> p.B_log2;
  const int64_t in_block = row & ((1 << p.B_log2) - 1);
  constexpr int kLanes = D / 8;
  const int groups = D >> p.group_log2;

  // keys: rotated in fp32 into shared memory, converted on the way
  const T* k = static_cast<const T*>(p.k) + t * p.k_token + h0 * p.k_head;
  const int total = nh * static_cast<int>(p.items_per_row.d);
  const int half = p.rope.half;
  const int turned = kPairing == HC_PAIR_HALF_SPLIT ? half / V : 2 * half / V;
  for (int idx = lane; idx < total; idx += 32) {
    uint32_t h, it;
    p.items_per_row.divmod(static_cast<uint32_t>(idx), h, it);
    const int item = static_cast<int>(it);
    const int c = item < turned || kPairing != HC_PAIR_HALF_SPLIT ? item * V : 2 * half + (item - turned) * V;
    const T* src = k + h * p.k_head + c;
    float* dst = rows[warp] + h * D + c;
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
          turn(f[i], x2, cs[warp][item * V + i]);
          dst[half + i] = x2;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) turn(f[2 * i], f[2 * i + 1], cs[warp][item * (V / 2) + i]);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) dst[i] = f[i];
  }
  __syncwarp();

  // every lane 8 channels of a row; lanes past the last row repeat it
  const int h = min(lane / kLanes, nh - 1), c = (lane & (kLanes - 1)) * 8;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float x[8];
    if (kv == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = rows[warp][h * D + c + i];
    } else {
      const T* src = static_cast<const T*>(p.v) + t * p.v_token + (h0 + h) * p.v_head + c;
#pragma unroll
      for (int j = 0; j < 8 / V; ++j) {
        const Piece<T, V> a = load_piece<T, V>(src + j * V);
#pragma unroll
        for (int i = 0; i < V; ++i) x[j * V + i] = to_f32(a.e[i]);
      }
    }
    const int64_t at = (((slot * 2 + kv) * p.H + h0 + h) << p.B_log2) + in_block;
    quantize_row<D, kScaleF16>(x, lane, p.group_log2, p.codes + at * (D / 2),
                               static_cast<uint8_t*>(p.scales) + at * groups * (kScaleF16 ? 2 : 4));
  }
}

template <typename T, int D, int kPairing>
cudaError_t launch(AppendParams p, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int items = rope_items<kPairing, V>(p.rope.half, D);
  p.items_per_row = FastDivmod(static_cast<uint32_t>(items));
  p.kv_parts = (p.H + kKvHeads<D> - 1) / kKvHeads<D>;
  p.q_heads_per_warp = std::max(1, p.n_q_heads);
  constexpr int64_t enough = 152 * 24;
  while (p.q_heads_per_warp > 1 && static_cast<int64_t>(p.q_heads_per_warp) * items > 32 &&
         static_cast<int64_t>(p.n_tokens) *
                 (p.kv_parts + (p.n_q_heads + p.q_heads_per_warp - 1) / p.q_heads_per_warp) < enough)
    p.q_heads_per_warp = (p.q_heads_per_warp + 1) / 2;
  p.q_parts = (p.n_q_heads + p.q_heads_per_warp - 1) / p.q_heads_per_warp;
  const int64_t warps = static_cast<int64_t>(p.n_tokens) * (p.q_parts + p.kv_parts);
  const unsigned grid = static_cast<unsigned>((warps + kRopeWarps - 1) / kRopeWarps);
  if (p.scale_f16)
    k_append_int4<T, D, kPairing, true><<<grid, kRopeWarps * 32, 0, s>>>(p);
  else
    k_append_int4<T, D, kPairing, false><<<grid, kRopeWarps * 32, 0, s>>>(p);
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
