// Attention of the new tokens over the 4-bit cache, rows of few queries:
// tensor-core products on the codes as they are, split over the keys.
//
// For a request and a cache head, the query rows are its new tokens times the
// query heads that share the cache head.  A piece of work is up to 8 * NT of
// those rows against all their keys.  The pieces of a call, laid end to end in
// tiles of 128 keys, are cut into equal runs, one per CTA (4 warps, 32 keys
// of a tile each), so requests of any lengths load the SMs alike; a CTA ends
// a piece, starts the next, or does both.  A piece that one CTA holds whole
// is written at once; otherwise each CTA leaves its partial sums in the
// workspace and the last to arrive (a counter per piece) joins them, in the
// order of the CTAs, so the result does not depend on which came last.
//
// Mathematics, per row, over tiles of keys with a reference m:
//   x_j = c * sum_g s_jg * (q_g . n_jg - corr_g),  p_j = 2^(x_j - m),
//   l = sum p_j,  O = sum (p_j * sv_jg) * nv_jg
// with n the codes, s the scales of their groups and c = softmax_scale *
// log2(e) * the power of two that the row's queries were scaled by.
// * Keys as fp16 without conversion: the nibble u = code + 8, in the low
//   bits of an fp16, is the subnormal u * 2^-24 exactly, so one AND-XOR makes
//   two operands; the "+ 8" is the same for all keys, and corr_g = 8 * sum of
//   q over the group, the products' starting value, takes it off again.
//   Nibbles 1 and 5 of a word stay 4 bits up (16 u) against queries divided
//   by 16.
// * Queries as fp16: each row times a power of two that brings its largest
//   value near 2^14, so that bf16's range fits and only values below 2^-28
//   of the row's largest lose bits (2^-24 in the channels of nibbles 1 and 5,
//   whose queries are divided by 16).
// * Values as exact bf16 whole numbers.  Their scales go into the
//   probabilities, and those into two bf16 (16 bits of mantissa, fp32's
//   range) for two products: an fp16 would flush what is below 2^-39 of the
//   largest, which a channel keeps where the larger keys' values are zero,
//   and its rounding is as large as that of an fp16 output.
// * S = Q K^T, then O^T = V^T P^T: a thread's results of the first product are
//   where the second wants them, and channels are the 16 rows of the second.
//   The first has room for 16 query rows; where there are up to 8, the others
//   hold the queries of a word's other four channels, so that both products of
//   a word read the same operand.
// * The reference m is the largest score of the first keys; it moves when a
//   sum passes 2^40 (fp32 and bf16 hold 2^-126 to 2^127), so most tiles need
//   no maximum, and no lanes' agreement but one vote.
//
// Bound: the cache's bytes when rows are few; in fact the issue of about 740
// instructions per 32 keys of 128 channels, half of them the codes' conversion.
// 64 requests of 200 to 25000 keys, 8 cache heads of 128 channels, groups of
// 32: 107 us, 3.6 TB/s; 8 of 131000 keys, one group per head: 252 us, 4.4 TB/s.
// Splitting the keys into equal runs rather than per request keeps every SM
// busy whatever the lengths; copies run two tiles ahead (three: the same).
#include <algorithm>

#include "attend_common.cuh"
#include "warp_mma.cuh"

namespace hc {
namespace {

constexpr int kWarpsA = 4;
constexpr int kKeysWarp = 32;                      // keys of one warp in a tile
constexpr int kTile = kWarpsA * kKeysWarp;         // keys of a tile
// What a piece's start and end take, in tiles: 64 requests of 200 to 25000 keys
// took 137 us where it was not counted (short requests crowded on one CTA),
// 117 us with 2, 120 us with 4.
constexpr int kPieceCost = 2;
constexpr int kStages = 3;
// Per SM, up to 8 query rows: 64 ragged requests took 110 us with 3, 117 us
// with 4, whose 128 registers do not hold the loop.  16 rows: 2.
constexpr int kCtasPerSm = 3;
constexpr int kMaxCtas = 1024;                     // counters in the workspace
constexpr int kMaxRows = 16;                       // rows of a piece
constexpr float kMostSum = 0x1p40f;                // of a lane's probabilities against a reference
constexpr int kPartialFloats = kMaxRows * (128 + 2);

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                        const float* c) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// Signed codes of nibbles 0 and 4 of w as bf16: 128 + u in the mantissa,
// u = code + 8, less 136.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
  const uint32_t m = and_xor(w, 0x000f000fu, 0x43084308u);
  __nv_bfloat162 h;
  memcpy(&h, &m, 4);
  h = __hsub2(h, __bfloat162bfloat162(__ushort_as_bfloat16(0x4308)));
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
template <int kRows>
__device__ __forceinline__ int request_units(const AttendParams& p, const Request& q) {
  int units = 0;
  if (q.n * p.G > p.rows_above) return 0;  // k_attend_tiles does these
  for (int r0 = 0, rows = q.n * p.G; r0 < rows; r0 += kRows)
    units += visible<kTile>(p, q, r0, min(r0 + kRows, rows)).tiles + p.piece_cost;
  return units * p.H;
}

template <int D, int GROUP, bool kScaleF16>
struct Layout {
  static constexpr int kRowBytes = D / 2;
  static constexpr int kRowChunks = kRowBytes / 16;
  static constexpr int kGroups = D / GROUP;
  static constexpr int kScaleBytes = kGroups * (kScaleF16 ? 2 : 4);  // of one key
  static constexpr int kCodeBytes = kKeysWarp * kRowBytes;           // K or V of a stage
  static constexpr int kScaleStage = kKeysWarp * kScaleBytes;
  static constexpr int kStageBytes = 2 * kCodeBytes + 2 * kScaleStage;
  static constexpr int kWarpBytes = kStages * kStageBytes;
};

// A 16-byte piece's place in a row of codes: rows that ldmatrix reads
// together fall into different banks.
template <int D>
__device__ __forceinline__ int swizzled(int key, int chunk) {
  return D == 128 ? chunk ^ ((key >> 1) & 3) : chunk ^ ((key >> 2) & 1);
}

// The scales of keys key and key + 1 (key even), by group.
template <int kGroups, bool kScaleF16>
__device__ __forceinline__ void load_scales(float2 (&s)[kGroups], const unsigned char* base, int key) {
  constexpr int kWords = kGroups * (kScaleF16 ? 1 : 2);  // of both keys
  uint32_t w[kWords];
  const unsigned char* at = base + key / 2 * (kWords * 4);
  if constexpr (kWords % 4 == 0) {
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(at + i * 4);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  } else if constexpr (kWords == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  }
  if constexpr (!kScaleF16) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) s[g] = make_float2(__uint_as_float(w[g]), __uint_as_float(w[kGroups + g]));
  } else if constexpr (kGroups == 1) {
    s[0] = u32_to_float2(w[0], static_cast<const __half*>(nullptr));
  } else {
#pragma unroll
    for (int g = 0; g < kGroups; g += 2) {
      const float2 a = u32_to_float2(w[g / 2], static_cast<const __half*>(nullptr));
      const float2 b = u32_to_float2(w[kGroups / 2 + g / 2], static_cast<const __half*>(nullptr));
      s[g] = make_float2(a.x, b.x);
      s[g + 1] = make_float2(a.y, b.y);
    }
  }
}

struct Shared {
  int32_t r, off;  // the request and the offset in it where the CTA's run starts
  uint32_t warp[kWarpsA];
  int32_t last;
  float m[kWarpsA][kMaxRows], l[kWarpsA][kMaxRows];
  float wt[kMaxRows], inv[kMaxRows];
};

template <int D, int GROUP, bool kScaleF16, int NT>
__global__ void __launch_bounds__(kWarpsA * 32, NT == 1 ? kCtasPerSm : 2)
    k_attend_rows(const __grid_constant__ AttendParams p) {
  using L = Layout<D, GROUP, kScaleF16>;
  constexpr int kRows = 8 * NT;
  constexpr int kChunks = D / 32;                 // 16-byte pieces of a row: 32 channels each
  constexpr int kGroups = L::kGroups;
  constexpr int kChunksPerGroup = GROUP / 32;
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  unsigned char* stages = dyn + warp * L::kWarpBytes;
  const uint32_t stages_addr = smem_addr(stages);
  int bad = 0;

  // ---- this CTA's run of tiles
  const int per = (p.n_req + kWarpsA * 32 - 1) / (kWarpsA * 32);
  const int r_first = tid * per, r_last = min(r_first + per, p.n_req);
  uint32_t mine = 0;
  for (int r = r_first; r < r_last; ++r) mine += request_units<kRows>(p, load_request(p, r, bad));
  uint32_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sh.warp[warp] = inc;
  if (tid == 0) sh.r = -1;
  __syncthreads();
  uint32_t before = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarpsA; ++w) {
    if (w < warp) before += sh.warp[w];
    total += sh.warp[w];
  }
  const uint32_t ctas = gridDim.x, b = blockIdx.x;
  const uint32_t share = total / ctas, extra = total - share * ctas;
  const uint32_t begin = b * share + min(b, extra), end = begin + share + (b < extra ? 1u : 0u);
  if (b == 0) flag_error(p.err, bad);
  bad = 0;
  if (begin == end) return;
  if (before <= begin && begin < before + mine) {
    uint32_t at = before;
    for (int r = r_first; r < r_last; ++r) {
      const uint32_t u = request_units<kRows>(p, load_request(p, r, bad));
      if (begin < at + u) {
        sh.r = r;
        sh.off = static_cast<int>(begin - at);
        break;
      }
      at += u;
    }
  }
  __syncthreads();
  bad = 0;

  // ---- the pieces of the run
  int r = sh.r, off = sh.off, row0 = 0, head = 0;
  if (r < 0) return;
  Request rq = load_request(p, r, bad);
  int rows_all = rq.n * p.G;
  Range vis = visible<kTile>(p, rq, 0, min(kRows, rows_all));
  for (;;) {  // to the piece that holds `off`: rows outermost, then heads
    const int cost = vis.tiles + p.piece_cost;
    if (off < cost * p.H) {
      head = off / cost;
      off -= head * cost;
      break;
    }
    off -= cost * p.H;
    row0 += kRows;
    if (row0 >= rows_all) return;  // never, unless the lengths change under the kernel
    vis = visible<kTile>(p, rq, row0, min(row0 + kRows, rows_all));
  }

  for (uint32_t unit = begin; unit < end;) {
    // units [off, off + taken) of the piece: its start, then its tiles
    const int taken = static_cast<int>(min(end - unit, static_cast<uint32_t>(vis.tiles + p.piece_cost - off)));
    const int first = max(off - p.piece_cost, 0), seg = max(off + taken - p.piece_cost, 0) - first;
    if (seg > 0) {
      const int rows = min(kRows, rows_all - row0);

      // -- the first tiles on their way
      const int32_t* table = p.tables + static_cast<int64_t>(r) * p.table_stride;
      const int key_first = (vis.tile0 + first) * kTile + warp * kKeysWarp;
      const int key_end = min(vis.hi, (vis.tile0 + first + seg) * kTile);
      // the slots of a tile's two runs of 16 keys; -1: no visible key, or no such slot
      auto load_slots = [&](int key0, int (&slot)[2]) {
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
          const int key = key0 + sb * 16;
          slot[sb] = -1;
          if (key < key_end && key + 16 > vis.lo) {
            slot[sb] = __ldg(table + (key >> p.B_log2));
            if (static_cast<uint32_t>(slot[sb]) >= static_cast<uint32_t>(p.num_slots)) {
              bad |= HC_DEVERR_SLOT;
              slot[sb] = -1;
            }
          }
        }
      };
      // A run of 16 keys is contiguous in the cache, codes and scales alike: lane l copies piece l of each 512 bytes
      // of codes, and of the scales K's pieces by the lanes from 0, V's by the lanes after them.
      constexpr int kRunCopies = 16 * L::kRowBytes / 512;
      constexpr int kScalePieces = 16 * L::kScaleBytes / 16;  // of a run, of K; as many of V
      const int run_bits = p.B_log2 - 4;                       // runs of a block
      const uint32_t to_v = static_cast<uint32_t>(p.H) << run_bits;
      const int64_t v_bytes = static_cast<int64_t>(to_v) * (16 * L::kRowBytes);
      const uint8_t* code_src = p.codes + lane * 16;
      const bool scales_v = lane >= kScalePieces;
      const int scale_piece = scales_v ? lane - kScalePieces : lane;
      const uint8_t* scale_src = static_cast<const uint8_t*>(p.scales) + scale_piece * 16 +
                                 (scales_v ? static_cast<int64_t>(to_v) * (16 * L::kScaleBytes) : 0);
      const uint32_t code_dst = stages_addr + (lane / L::kRowChunks) * L::kRowBytes +
                                swizzled<D>(lane / L::kRowChunks, lane % L::kRowChunks) * 16;
      const uint32_t scale_dst = stages_addr + 2 * L::kCodeBytes + (scales_v ? L::kScaleStage : 0) + scale_piece * 16;
      auto run_at = [&](int key, int slot) {
        return ((static_cast<uint32_t>(slot) * 2 * p.H + head) << run_bits) + ((key & ((1 << p.B_log2) - 1)) >> 4);
      };
      auto load_tile = [&](int key0, uint32_t stage, const int (&slot)[2]) {
        if (slot[0] >= 0 && slot[1] >= 0 && key0 + kKeysWarp <= vis.hi) {  // all there
#pragma unroll
          for (int sb = 0; sb < 2; ++sb) {
            const uint32_t run = run_at(key0 + sb * 16, slot[sb]);
            const uint8_t* src = code_src + static_cast<uint64_t>(run) * (16 * L::kRowBytes);
            const uint8_t* v_src = src + v_bytes;
            const uint32_t dst = code_dst + stage + sb * 16 * L::kRowBytes;
#pragma unroll
            for (int it = 0; it < kRunCopies; ++it) {
              // rows that ldmatrix reads together differ by less than the 512 bytes, so the swizzle repeats
              cp_async16(dst + it * 512, src + it * 512, 16);
              cp_async16(dst + it * 512 + L::kCodeBytes, v_src + it * 512, 16);
            }
            if (lane < 2 * kScalePieces)
              cp_async16(scale_dst + stage + sb * kScalePieces * 16,
                         scale_src + static_cast<uint64_t>(run) * (16 * L::kScaleBytes), 16);
          }
          return;
        }
#pragma unroll 1
        for (int sb = 0; sb < 2; ++sb) {
          const int key = key0 + sb * 16, at = sb ? slot[1] : slot[0];
          const int keys = at < 0 ? 0 : min(16, vis.hi - key);  // to copy; zeros after them
          const uint32_t run = at < 0 ? 0 : run_at(key, at);
          const uint8_t* src = code_src + static_cast<uint64_t>(run) * (16 * L::kRowBytes);
          const uint32_t dst = code_dst + stage + sb * 16 * L::kRowBytes;
          for (int it = 0; it < kRunCopies; ++it) {
            const bool in = it * (16 / kRunCopies) + lane / L::kRowChunks < keys;
            cp_async16(dst + it * 512, in ? src + it * 512 : p.codes, in ? 16 : 0);
            cp_async16(dst + it * 512 + L::kCodeBytes, in ? src + it * 512 + v_bytes : p.codes, in ? 16 : 0);
          }
          if (lane < 2 * kScalePieces) {
            const int left = min(16, max(0, keys * L::kScaleBytes - scale_piece * 16));
            const uint8_t* from = static_cast<const uint8_t*>(p.scales);
            if (left > 0) from = scale_src + static_cast<uint64_t>(run) * (16 * L::kScaleBytes);
            cp_async16(scale_dst + stage + sb * kScalePieces * 16, from, left);
          }
        }
      };
      int slot[2];
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) {
        load_slots(key_first + i * kTile, slot);
        if (i < seg) load_tile(key_first + i * kTile, i * L::kStageBytes, slot);
        cp_async_commit();
      }
      load_slots(key_first + (kStages - 1) * kTile, slot);
      uint32_t stage_to = (kStages - 1) * L::kStageBytes, stage_at = 0;  // copied to, read from

      // -- queries: fragments, the correction of the codes' offset, row factors
      // As A operands.  Up to 8 rows: rows 0 to 7 for nibbles 0, 4, 1, 5 of a word, rows 8 to 15 (the same queries)
      // for 2, 6, 3, 7.  Up to 16 rows: one operand for the first four nibbles, one for the others.
      uint32_t qf[NT][kChunks][4];
      // the products' starting values; up to 8 rows, two groups to an operand as their queries are
      constexpr int kStarts = NT == 1 ? (kGroups + 1) / 2 : kGroups;
      float factor[NT], corr[kStarts][4] = {};  // of row g (and g + 8)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = row0 + nt * 8 + g;
        const bool live = row < rows_all;
        float f[kChunks][8];
        float amax = 0.f;
        const int i = static_cast<int>(p.by_group.div(live ? row : 0));
        const int64_t at = static_cast<int64_t>(rq.q0 + i) * p.q_token +
                           static_cast<int64_t>(head * p.G + (live ? row : 0) - i * p.G) * p.q_head;
#pragma unroll
        for (int cc = 0; cc < kChunks; ++cc) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (live)
            w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at + cc * 32 + t * 8);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = widen(u[k], p.bf16);
            f[cc][2 * k] = v.x;
            f[cc][2 * k + 1] = v.y;
            amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^e <= amax < 2^(e+1); queries times 2^(14-e)
        const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);  // at most 127: finite
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
        float sum[kGroups];
#pragma unroll
        for (int k = 0; k < kGroups; ++k) sum[k] = 0.f;
#pragma unroll
        for (int cc = 0; cc < kChunks; ++cc) {
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = f[cc][k] * up * ((k & 1) ? 0.0625f : 1.f);
          const uint32_t pairs[4] = {pack_f16(x[0], x[4]), pack_f16(x[1], x[5]), pack_f16(x[2], x[6]),
                                     pack_f16(x[3], x[7])};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (NT == 1)
              qf[0][cc][k % 2 * 2 + k / 2] = pairs[k];
            else
              qf[k / 2][cc][k % 2 * 2 + nt] = pairs[k];
            const float2 v = u32_to_float2(pairs[k], static_cast<const __half*>(nullptr));
            sum[cc / kChunksPerGroup] += (v.x + v.y) * ((k & 1) ? 16.f : 1.f);
          }
        }
        factor[nt] = p.scale_log2 * 1024.f * pow2(e);  // 2^(24-14+e), which fp32 does not hold by itself from e = 118 on
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
          sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
          sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
          const float start = sum[k] * (-8.f * 0x1p-24f);
          if (NT == 1)
            corr[k / 2][k % 2 * 2] = corr[k / 2][k % 2 * 2 + 1] = start;
          else
            corr[k][2 * nt] = corr[k][2 * nt + 1] = start;
        }
      }
      // keys that every row sees: no mask needed inside
      int all_lo, all_hi;
      {
        const int i0 = static_cast<int>(p.by_group.div(row0)), i1 = static_cast<int>(p.by_group.div(row0 + rows - 1));
        all_hi = p.causal ? min(rq.kv, rq.kv - rq.n + i0 + 1) : rq.kv;
        all_lo = p.window ? max(0, rq.kv - rq.n + i1 - p.window + 1) : 0;
      }

      float o[NT][D / 16][4], m[NT];
      float2 l[NT];  // of even and odd keys
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[nt][c][j] = 0.f;
        m[nt] = kNegInf;
        l[nt] = make_float2(0.f, 0.f);
      }

      // Rows before the window came along with their run of 16 and may hold anything.  Their probabilities are 0, but
      // 0 times a value scale that is infinite or NaN is not (scores are replaced, whatever they are).  Only the first
      // tile has such rows; inside the loop this took 250 us to 253 (8 requests of 131000 keys, no window).
      if (key_first < vis.lo) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        if (key_first + lane < vis.lo) {
          uint16_t* hidden = reinterpret_cast<uint16_t*>(stages + 2 * L::kCodeBytes + L::kScaleStage + lane * L::kScaleBytes);
#pragma unroll
          for (int i = 0; i < L::kScaleBytes / 2; ++i) hidden[i] = 0;
        }
      }
      for (int i = 0; i < seg; ++i) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        const int key0 = key_first + i * kTile;
        if (i + kStages - 1 < seg) load_tile(key0 + (kStages - 1) * kTile, stage_to, slot);
        cp_async_commit();
        load_slots(key0 + kStages * kTile, slot);
        const unsigned char* stage = stages + stage_at;
        stage_to = stage_at;
        stage_at = stage_at == (kStages - 1) * L::kStageBytes ? 0 : stage_at + L::kStageBytes;
        if (key0 >= vis.hi || key0 + kKeysWarp <= vis.lo) continue;
        const uint32_t ks = smem_addr(stage), vs = ks + L::kCodeBytes;
        const unsigned char* k_scale = stage + 2 * L::kCodeBytes;
        const unsigned char* v_scale = k_scale + L::kScaleStage;

        // -- scores: S[row][key], keys 2t and 2t + 1 of each run of 8
        float2 s[NT][kKeysWarp / 8];
        [[maybe_unused]] uint32_t kw2[4];  // 64 channels: of two runs
#pragma unroll
        for (int n = 0; n < kKeysWarp / 8; ++n) {
          uint32_t kw[kChunks];  // of key g: word t of each 16-byte piece
          if constexpr (D == 128) {
            const int key = n * 8 + (lane & 7);
            ldmatrix4(kw, ks + key * L::kRowBytes + swizzled<D>(key, lane >> 3) * 16);
          } else {
            if (n % 2 == 0) {
              const int key = n * 8 + ((lane >> 4) & 1) * 8 + (lane & 7);
              ldmatrix4(kw2, ks + key * L::kRowBytes + swizzled<D>(key, (lane >> 3) & 1) * 16);
            }
            kw[0] = kw2[n % 2 * 2], kw[1] = kw2[n % 2 * 2 + 1];
          }
          float2 sk[kGroups];
          load_scales<kGroups, kScaleF16>(sk, k_scale, n * 8 + 2 * t);
#pragma unroll
          for (int gr = 0; gr < kGroups; ++gr) {
            float a0[4], a1[4];  // of the two halves of the codes
            constexpr float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = gr * kChunksPerGroup; c < (gr + 1) * kChunksPerGroup; ++c) {
              const uint32_t w = kw[c], x = w >> 8;
              const uint32_t b0 = and_xor(w, 0x000f000fu, 0x00080008u), b1 = and_xor(w, 0x00f000f0u, 0x00800080u);
              const uint32_t b2 = and_xor(x, 0x000f000fu, 0x00080008u), b3 = and_xor(x, 0x00f000f0u, 0x00800080u);
              const bool starts = c == gr * kChunksPerGroup;
              if constexpr (NT == 1) {
                // one A operand for both: its rows from 8 on are the queries of the second half, so the first
                // product's upper rows and the second's lower rows mean nothing
                mma_f16(a0, qf[0][c], b0, b1, starts ? (gr % 2 == 0 ? corr[gr / 2] : zero) : a0);
                mma_f16(a1, qf[0][c], b2, b3, starts ? (gr % 2 == 1 ? corr[gr / 2] : zero) : a1);
              } else {
                mma_f16(a0, qf[0][c], b0, b1, starts ? corr[gr] : a0);
                mma_f16(a0, qf[1][c], b2, b3, a0);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float2 v = NT == 1 ? __fadd2_rn(make_float2(a0[0], a0[1]), make_float2(a1[2], a1[3]))
                                       : make_float2(a0[2 * nt], a0[2 * nt + 1]);
              s[nt][n] = gr == 0 ? __fmul2_rn(v, sk[gr]) : __ffma2_rn(v, sk[gr], s[nt][n]);
            }
          }
        }

        // the first values' codes on their way to registers
        uint32_t vw[kChunks / 2][4];
#pragma unroll
        for (int cp = 0; cp < kChunks / 2; ++cp) {
          const int key = ((lane >> 3) & 1) * 8 + (lane & 7);
          ldmatrix4_trans(vw[cp], vs + key * L::kRowBytes + swizzled<D>(key, cp * 2 + (lane >> 4)) * 16);
        }
        // -- probabilities against the reference that the rows have, kept while the sums stay small
        bool done = !(key0 < all_lo || key0 + kKeysWarp > all_hi);
        float2 e[NT][kKeysWarp / 8];
        if (done) {
          bool small = true;
          float2 sum[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 f = make_float2(factor[nt], factor[nt]), less = make_float2(-m[nt], -m[nt]);
            sum[nt] = l[nt];
#pragma unroll
            for (int n = 0; n < kKeysWarp / 8; ++n) {
              const float2 x = __ffma2_rn(s[nt][n], f, less);
              e[nt][n] = make_float2(ex2(x.x), ex2(x.y));
              sum[nt] = __fadd2_rn(sum[nt], e[nt][n]);
            }
            small = small && sum[nt].x + sum[nt].y <= kMostSum;
          }
          done = __all_sync(0xffffffffu, small);
          if (done) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) l[nt] = sum[nt];
          }
        }
        if (!done) {  // the first keys, keys that some row does not see, a reference to move
          float alpha[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int row = min(row0 + nt * 8 + g, rows_all - 1);
            const int pos = rq.kv - rq.n + static_cast<int>(p.by_group.div(row));
            const int last = p.causal ? min(rq.kv, pos + 1) : rq.kv, first = p.window ? pos - p.window + 1 : 0;
            float top = kNegInf;
#pragma unroll
            for (int n = 0; n < kKeysWarp / 8; ++n) {
              const int key = key0 + n * 8 + 2 * t;
              s[nt][n].x = key < first || key >= last ? kNegInf : s[nt][n].x * factor[nt];
              s[nt][n].y = key + 1 < first || key + 1 >= last ? kNegInf : s[nt][n].y * factor[nt];
              top = fmaxf(top, fmaxf(s[nt][n].x, s[nt][n].y));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float to = fmaxf(m[nt], top), ref = to == kNegInf ? 0.f : to;
            // nothing seen so far: l and O are 0, whatever they are multiplied by
            alpha[nt] = m[nt] == kNegInf ? 0.f : ex2(m[nt] - to);
            m[nt] = to;
            l[nt].x *= alpha[nt];
            l[nt].y *= alpha[nt];
#pragma unroll
            for (int n = 0; n < kKeysWarp / 8; ++n) {
              e[nt][n] = make_float2(ex2(s[nt][n].x - ref), ex2(s[nt][n].y - ref));
              l[nt] = __fadd2_rn(l[nt], e[nt][n]);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float a = __shfl_sync(0xffffffffu, alpha[nt], (2 * t + j) * 4);
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                o[nt][c][j] *= a;
                o[nt][c][2 + j] *= a;
              }
            }
        }

        // -- O^T += V^T P^T, 16 keys at a time
#pragma unroll
        for (int mt = 0; mt < kKeysWarp / 16; ++mt) {
          const int key = mt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
          float2 sv[2][kGroups];
          load_scales<kGroups, kScaleF16>(sv[0], v_scale, mt * 16 + 2 * t);
          load_scales<kGroups, kScaleF16>(sv[1], v_scale, mt * 16 + 2 * t + 8);
          uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
          for (int cp = 0; cp < kChunks / 2; ++cp) {  // two 16-byte pieces: 64 channels
            uint32_t w[4];
            if (mt == 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = vw[cp][i];
            } else {
              ldmatrix4_trans(w, vs + key * L::kRowBytes + swizzled<D>(key, cp * 2 + (lane >> 4)) * 16);
            }
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              const int c = cp * 2 + h2;
              if (c % kChunksPerGroup == 0) {
                const int gr = c / kChunksPerGroup;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf)
                    split_bf16(__fmul2_rn(e[nt][mt * 2 + hf], sv[hf][gr]), ph[nt][hf], pl[nt][hf]);
              }
              const uint32_t w0 = w[h2 * 2], w1 = w[h2 * 2 + 1];
              const uint32_t a0 = codes_bf16(w0), a1 = codes_bf16(w0 >> 4), a2 = codes_bf16(w1), a3 = codes_bf16(w1 >> 4);
              const uint32_t b0 = codes_bf16(w0 >> 8), b1 = codes_bf16(w0 >> 12), b2 = codes_bf16(w1 >> 8),
                             b3 = codes_bf16(w1 >> 12);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_bf16(o[nt][2 * c], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
                mma_bf16(o[nt][2 * c + 1], b0, b1, b2, b3, ph[nt][0], ph[nt][1]);
                mma_bf16(o[nt][2 * c], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
                mma_bf16(o[nt][2 * c + 1], b0, b1, b2, b3, pl[nt][0], pl[nt][1]);
              }
            }
          }
        }
      }
      cp_async_wait<0>();

      __syncthreads();

      // ---- the warps' sums joined: O in shared memory, [warp][row][channel]
      float* so = reinterpret_cast<float*>(dyn);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float sum = l[nt].x + l[nt].y;
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (t == 0) {
          sh.m[warp][nt * 8 + g] = m[nt];
          sh.l[warp][nt * 8 + g] = sum;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = nt * 8 + 2 * t + j;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const int ch = (c >> 1) * 32 + 4 * g + 2 * (c & 1);
            *reinterpret_cast<float2*>(so + (warp * kRows + row) * D + ch) = make_float2(o[nt][c][j], o[nt][c][2 + j]);
          }
        }
      }
      __syncthreads();
      const bool whole = seg == vis.tiles;
      float* ws = reinterpret_cast<float*>(p.workspace + kMaxCtas * sizeof(int32_t));
      int32_t* counters = reinterpret_cast<int32_t*>(p.workspace);
      float* partial = ws + (static_cast<int64_t>(b) * 2 + (first > 0 ? 0 : 1)) * kPartialFloats;

      auto write_row = [&](int row, int ch, float4 v, float mref, float sum) {
        // v: unnormalised sums of 4 channels
        const int rr = row0 + row, i = static_cast<int>(p.by_group.div(rr)), h = head * p.G + rr - i * p.G;
        const int64_t tok = rq.q0 + i;
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        uint2 w;
        w.x = p.bf16 ? pack_bf16(v.x * inv, v.y * inv) : pack_f16(v.x * inv, v.y * inv);
        w.y = p.bf16 ? pack_bf16(v.z * inv, v.w * inv) : pack_f16(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + tok * p.o_token + h * p.o_head + ch) = w;
        if (p.lse && ch == 0)
          p.lse[tok * (static_cast<int64_t>(p.H) * p.G) + h] =
              sum > 0.f ? (mref + log2f(sum)) * 0.6931471805599453f : kNegInf;
      };

      for (int id = tid; id < rows * (D / 4); id += kWarpsA * 32) {
        const int row = id / (D / 4), ch = (id % (D / 4)) * 4;
        float top = kNegInf, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarpsA; ++w) top = fmaxf(top, sh.m[w][row]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarpsA; ++w) {
          const float wt = sh.m[w][row] == kNegInf ? 0.f : ex2(sh.m[w][row] - top);
          const float4 v = *reinterpret_cast<const float4*>(so + (w * kRows + row) * D + ch);
          sum += wt * sh.l[w][row];
          acc.x += wt * v.x, acc.y += wt * v.y, acc.z += wt * v.z, acc.w += wt * v.w;
        }
        if (whole) {
          write_row(row, ch, acc, top, sum);
        } else {
          __stcg(reinterpret_cast<float4*>(partial + 2 * kMaxRows + row * D + ch), acc);
          if (ch == 0) {
            __stcg(partial + row, top);
            __stcg(partial + kMaxRows + row, sum);
          }
        }
      }
      if (!whole) {
        // the CTAs that hold a part of this piece: first to last
        const uint32_t u0 = unit - off + p.piece_cost, u1 = u0 + vis.tiles - 1;
        auto owner = [&](uint32_t u) {
          const uint32_t big = extra * (share + 1);
          return u < big ? u / (share + 1) : extra + (u - big) / share;
        };
        const uint32_t c0 = owner(u0), c1 = owner(u1);
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          const int arrived = atomicAdd(counters + c0, 1);
          sh.last = arrived == static_cast<int>(c1 - c0);
          if (sh.last) counters[c0] = 0;
          __threadfence();
        }
        __syncthreads();
        if (sh.last) {
          auto part = [&](uint32_t c) { return ws + (static_cast<int64_t>(c) * 2 + (c == c0 ? 1 : 0)) * kPartialFloats; };
          for (int row = warp; row < rows; row += kWarpsA) {
            float top = kNegInf, sum = 0.f;
            for (uint32_t c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, __ldcg(part(c) + row));
#pragma unroll
            for (int o2 = 16; o2 > 0; o2 >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o2));
            for (uint32_t c = c0 + lane; c <= c1; c += 32) {
              const float mc = __ldcg(part(c) + row);
              if (mc != kNegInf) sum += ex2(mc - top) * __ldcg(part(c) + kMaxRows + row);
            }
#pragma unroll
            for (int o2 = 16; o2 > 0; o2 >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o2);
            if (lane == 0) {
              sh.wt[row] = top;
              sh.inv[row] = sum;
            }
          }
          __syncthreads();
          for (int id = tid; id < rows * (D / 4); id += kWarpsA * 32) {
            const int row = id / (D / 4), ch = (id % (D / 4)) * 4;
            const float top = sh.wt[row];
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (uint32_t c = c0; c <= c1; ++c) {
              const float mc = __ldcg(part(c) + row);
              const float4 v = __ldcg(reinterpret_cast<const float4*>(part(c) + 2 * kMaxRows + row * D + ch));
              const float wt = mc == kNegInf ? 0.f : ex2(mc - top);
              acc.x += wt * v.x, acc.y += wt * v.y, acc.z += wt * v.z, acc.w += wt * v.w;
            }
            write_row(row, ch, acc, top, sh.inv[row]);
          }
        }
      }

    }

    // ---- the next piece
    unit += taken;
    off = 0;
    if (unit < end) {
      if (++head == p.H) {
        head = 0;
        row0 += kRows;
        while (row0 >= rows_all) {
          if (++r >= p.n_req) return;  // likewise
          rq = load_request(p, r, bad);
          bad &= ~HC_DEVERR_LENGTH;  // CTA 0 reports these
          rows_all = rq.n * p.G <= p.rows_above ? rq.n * p.G : 0;
          row0 = rows_all > 0 ? 0 : 1;
        }
        vis = visible<kTile>(p, rq, row0, min(row0 + kRows, rows_all));
      }
    }
    __syncthreads();
  }
  if (lane == 0) flag_error(p.err, bad & HC_DEVERR_SLOT);
}

template <int D, int GROUP, bool kScaleF16, int NT>
cudaError_t launch_rows(AttendParams p, cudaStream_t s) {
  using L = Layout<D, GROUP, kScaleF16>;
  const int smem = std::max(kWarpsA * L::kWarpBytes, kWarpsA * 8 * NT * D * 4);
  static KernelOnDevice kernel;
  int resident = 0;
  const cudaError_t e = kernel.resident(reinterpret_cast<const void*>(k_attend_rows<D, GROUP, kScaleF16, NT>),
                                        kWarpsA * 32, smem, &resident);
  if (e != cudaSuccess) return e;
  // one CTA per resident place, or per tile where there are fewer (as far as the host can tell)
  const int64_t rows =
      (std::min<int64_t>(static_cast<int64_t>(p.max_new) * p.G, p.rows_above) + 8 * NT - 1) / (8 * NT);
  const int64_t keys = static_cast<int64_t>(p.table_width) << p.B_log2;
  const int64_t tiles = std::max<int64_t>(1, (keys + kTile - 1) / kTile);
  int64_t grid = std::min(kMaxCtas, resident);
  p.piece_cost = kPieceCost;
  if (static_cast<double>(p.n_req) * p.H * rows * tiles < static_cast<double>(grid))
{
    grid = p.n_req * p.H * rows * tiles;
    p.piece_cost = 0;
  }
  k_attend_rows<D, GROUP, kScaleF16, NT><<<static_cast<unsigned>(grid), kWarpsA * 32, smem, s>>>(p);
  return cudaGetLastError();
}

// Pieces of 8 rows where no request has more: 64 ragged requests of 4 rows took
// 106 us, 144 us in pieces of 16, which need twice the products.
template <int D, int GROUP, bool kScaleF16>
cudaError_t launch_nt(const AttendParams& p, cudaStream_t s) {
  const int64_t rows = std::min<int64_t>(static_cast<int64_t>(p.max_new) * p.G, p.rows_above);
  return rows <= 8 ? launch_rows<D, GROUP, kScaleF16, 1>(p, s) : launch_rows<D, GROUP, kScaleF16, 2>(p, s);
}

template <int D, int GROUP>
cudaError_t launch_scale(bool scale_f16, const AttendParams& p, cudaStream_t s) {
  return scale_f16 ? launch_nt<D, GROUP, true>(p, s) : launch_nt<D, GROUP, false>(p, s);
}

}  // namespace

int64_t attend_workspace_bytes() {
  return kMaxCtas * static_cast<int64_t>(sizeof(int32_t)) +
         static_cast<int64_t>(kMaxCtas) * 2 * kPartialFloats * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_attend_rows(int d, int group, bool scale_f16, const AttendParams& p, cudaStream_t s) {
  if (d == 64) return group == 32 ? launch_scale<64, 32>(scale_f16, p, s) : launch_scale<64, 64>(scale_f16, p, s);
  if (group == 32) return launch_scale<128, 32>(scale_f16, p, s);
  return group == 64 ? launch_scale<128, 64>(scale_f16, p, s) : launch_scale<128, 128>(scale_f16, p, s);
}

}  // namespace hc
