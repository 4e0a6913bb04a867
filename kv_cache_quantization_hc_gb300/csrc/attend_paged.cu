// Attention of the new tokens over the paged buffer, rows of few queries:
// split over the keys, one pass over them.
//
// For a request and a cache head, the query rows are its new tokens times the
// query heads that share the cache head.  A piece of work is up to 8 * NT of
// those rows against all their keys.  For each cache head the pieces of a call,
// laid end to end in tiles of keys, are cut into equal runs, one per CTA (4
// warps, an equal part of a tile's keys each).  CTAs of the same run and
// neighbouring heads are neighbours: a token's heads lie side by side in the
// buffer, so they are read at about the same time.  A piece that one CTA holds
// whole is written at once; otherwise each CTA leaves its partial sums in the
// workspace and the last to arrive (a counter per piece) joins them, in the
// order of the CTAs, so the result does not depend on which came last.
//
// Mathematics, per row, over tiles of keys with the running maximum m:
//   x_j = the score of key j in units of log2, p_j = 2^(x_j - m + up),
//   l = sum p_j,  O = sum p_j v_j,  out = O / l
// * Queries and keys enter the products as they are stored; scores are fp32.
// * S = Q K^T, then O^T = V^T P^T: a thread's results of the first product are
//   where the second wants them, and channels are the 16 rows of the second.
// * Probabilities go into the second product as a high and a low part of the
//   values' type, 16 bits (bf16) or 22 (fp16) in all: a single one would be
//   rounded as coarsely as the output.  fp16 ends at 65504 and 2^-24, so there
//   up = 15: what is below 2^-39 of a row's largest is lost.
//
// Bound: the cache's bytes.  64 requests of 200 to 25000 keys, 32 query and 8
// cache heads of 128 bf16 channels: 204 us, 6.6 TB/s, 97% of the measured copy
// rate; 8 requests of 131000 keys, 8 query heads a cache head: 600 us, 7.2 TB/s.
// With few keys a CTA, latency: one request of 1000 keys 10 us (lengths, slots,
// keys, partial sums: a chain of reads).  Several pieces of a request each read
// its keys: 37 requests, 14 to 49 rows, 20.6 us of 4.9.
#include <algorithm>

#include "attend_paged_common.cuh"
#include "warp_mma.cuh"

namespace hc {
namespace {

constexpr int kWarpsA = 4;
constexpr int kPieceCost = 2;   // what a piece's start and end take, in tiles
// A run has this many units at least: a partial sum more takes longer than a tile more (5 requests of 84 to 5360 keys, 14
// to 49 rows: 20.0 us with 1, 15.4 with 2, 14.9 with 3, 16.8 with 4; one of 1000 keys, 4 rows: 10.6, 10.6, 11.0, 11.7).
constexpr uint32_t kLeastUnits = 2;
constexpr int kStages = 3;
constexpr int kCtasPerSm = 2;
constexpr int kMaxCtas = 1024;  // counters in the workspace
constexpr int kMaxRows = 16;    // rows of a piece
constexpr int kPartialFloats = kMaxRows * (128 + 2);

// A warp's part of a tile: 4 KiB of keys and 4 KiB of values.
template <int D>
struct Layout {
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kRowChunks = kRowBytes / 16;
  static constexpr int kKeys = 4096 / kRowBytes;  // of one warp in a tile
  static constexpr int kTile = kWarpsA * kKeys;
  static constexpr int kStageBytes = 2 * 4096;
  static constexpr int kWarpBytes = kStages * kStageBytes;
};

// A 16-byte piece's place in a row: the 8 rows that ldmatrix reads together
// fall into different banks.
__device__ __forceinline__ int swizzled(int key, int chunk) { return chunk ^ (key & 7); }

// D (+)= A B with 16-bit operands of type T, 16 x 8 x 16.
template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>)
    mma_bf16(c, a0, a1, a2, a3, b0, b1);
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two fp32 as a high and a low pair of T.
template <typename T>
__device__ __forceinline__ void split(float2 v, uint32_t& high, uint32_t& low) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    split_bf16(v, high, low);
  } else {
    high = pack_f16(v.x, v.y);
    const float2 kept = u32_to_float2(high, static_cast<const __half*>(nullptr));
    low = pack_f16(v.x - kept.x, v.y - kept.y);
  }
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) return pack_bf16(lo, hi);
  return pack_f16(lo, hi);
}

template <int kRows, int kTile>
__device__ __forceinline__ int request_units(const AttendPagedParams& p, const PagedRequest& q) {
  int units = 0;
  if (q.n * p.G > p.rows_above) return 0;  // k_attend_paged_tiles does these
  for (int r0 = 0, rows = q.n * p.G; r0 < rows; r0 += kRows)
    units += visible<kTile>(p, q, r0, min(r0 + kRows, rows)).tiles + p.piece_cost;
  return units;
}

struct Shared {
  int32_t r, off;  // the request and the offset in it where the CTA's run starts
  uint32_t warp[kWarpsA];
  int32_t last;
  float m[kWarpsA][kMaxRows], l[kWarpsA][kMaxRows];
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarpsA * 32, kCtasPerSm) k_attend_paged_rows(const __grid_constant__ AttendPagedParams p) {
  using L = Layout<D>;
  constexpr bool kBf16 = std::is_same_v<T, __nv_bfloat16>;
  constexpr float kUp = kBf16 ? 0.f : 15.f;
  constexpr int kRows = 8 * NT, kTile = L::kTile, kKeys = L::kKeys;
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t stages_addr = smem_addr(dyn + warp * L::kWarpBytes);
  uint32_t b, head_of;
  p.by_heads.divmod(blockIdx.x, b, head_of);
  const int head = static_cast<int>(head_of);
  int bad = 0;

  // ---- this CTA's run of tiles
  const int per = (p.n_req + kWarpsA * 32 - 1) / (kWarpsA * 32);
  const int r_first = tid * per, r_last = min(r_first + per, p.n_req);
  uint32_t mine = 0;
  for (int r = r_first; r < r_last; ++r) mine += request_units<kRows, kTile>(p, load_request(p, r, bad));
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
  if (blockIdx.x == 0) flag_error(p.err, bad);
  bad = 0;
  const uint32_t runs = max(1u, min(gridDim.x / p.H, total / kLeastUnits));  // of each head
  if (b >= runs) return;
  const uint32_t share = total / runs, extra = total - share * runs;
  const uint32_t begin = b * share + min(b, extra), end = begin + share + (b < extra ? 1u : 0u);
  if (begin == end) return;
  if (before <= begin && begin < before + mine) {
    uint32_t at = before;
    for (int r = r_first; r < r_last; ++r) {
      const uint32_t u = request_units<kRows, kTile>(p, load_request(p, r, bad));
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
  int r = sh.r, off = sh.off, row0 = 0;
  if (r < 0) return;
  PagedRequest rq = load_request(p, r, bad);
  int rows_all = rq.n * p.G;
  Range vis = visible<kTile>(p, rq, 0, min(kRows, rows_all));
  for (;;) {  // to the piece that holds `off`
    const int cost = vis.tiles + p.piece_cost;
    if (off < cost) break;
    off -= cost;
    row0 += kRows;
    if (row0 >= rows_all) return;  // never, unless the lengths change under the kernel
    vis = visible<kTile>(p, rq, row0, min(row0 + kRows, rows_all));
  }

  // A lane's 16-byte pieces of a run of 16 keys: piece `chunk` of keys lane / kRowChunks, and of every
  // 32 / kRowChunks-th after it.
  constexpr int kAt = 32 / L::kRowChunks;       // keys of a copy
  constexpr int kCopies = 16 / kAt;             // of a run of 16 keys
  const int lane_key = lane / L::kRowChunks;
  const int64_t key_bytes = static_cast<int64_t>(p.H) * L::kRowBytes;  // from a key to the next
  const int64_t lane_off = lane_key * key_bytes + static_cast<int64_t>(head) * L::kRowBytes + (lane % L::kRowChunks) * 16;
  const unsigned char* k_src = static_cast<const unsigned char*>(p.k_pages) + lane_off;
  const unsigned char* v_src = static_cast<const unsigned char*>(p.v_pages) + lane_off;

  for (uint32_t unit = begin; unit < end;) {
    // units [off, off + taken) of the piece: its start, then its tiles
    const int taken = static_cast<int>(min(end - unit, static_cast<uint32_t>(vis.tiles + p.piece_cost - off)));
    const int first = max(off - p.piece_cost, 0), seg = max(off + taken - p.piece_cost, 0) - first;
    if (seg > 0) {
      const int rows = min(kRows, rows_all - row0);

      // -- the first tiles on their way
      const int32_t* table = p.tables + static_cast<int64_t>(r) * p.table_stride;
      const int key_first = (vis.tile0 + first) * kTile + warp * kKeys;
      const int key_end = min(vis.hi, (vis.tile0 + first + seg) * kTile);
      // the slots of a warp's runs of 16 keys; -1: no visible key, or no such slot
      constexpr int kRuns = kKeys / 16;
      auto load_slots = [&](int key0, int (&slot)[kRuns]) {
#pragma unroll
        for (int sb = 0; sb < kRuns; ++sb) {
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
      // Rows that no query of the piece sees are not read: zeros take their place, as 0 times what they hold (an
      // infinity, a NaN) need not be 0.
      auto load_tile = [&](int key0, uint32_t stage, const int (&slot)[kRuns]) {
#pragma unroll
        for (int sb = 0; sb < kRuns; ++sb) {
          const int key = key0 + sb * 16;
          const uint32_t dst = stages_addr + stage + sb * 16 * L::kRowBytes;
          const int64_t at = slot[sb] < 0 ? 0
                                          : slot[sb] * p.slot_stride * 2 +
                                                static_cast<int64_t>(key & ((1 << p.B_log2) - 1)) * key_bytes;
          const bool whole = slot[sb] >= 0 && key >= vis.lo && key + 16 <= vis.hi;
          const int lo = vis.lo - key, hi = slot[sb] < 0 ? 0 : vis.hi - key;  // rows of the run that are seen
#pragma unroll
          for (int it = 0; it < kCopies; ++it) {
            const int row = it * kAt + lane_key;
            const uint32_t to = dst + row * L::kRowBytes + swizzled(row, lane % L::kRowChunks) * 16;
            const bool in = whole || (row >= lo && row < hi);
            const int64_t from = at + (it * kAt) * key_bytes;
            cp_async16(to, in ? k_src + from : p.k_pages, in ? 16 : 0);
            cp_async16(to + 4096, in ? v_src + from : p.v_pages, in ? 16 : 0);
          }
        }
      };
      int slot[kRuns];
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) {
        load_slots(key_first + i * kTile, slot);
        if (i < seg) load_tile(key_first + i * kTile, i * L::kStageBytes, slot);
        cp_async_commit();
      }
      load_slots(key_first + (kStages - 1) * kTile, slot);
      uint32_t stage_to = (kStages - 1) * L::kStageBytes, stage_at = 0;  // copied to, read from

      // -- queries as A operands (rows 8 to 15 are there for NT = 2 only), and what each row sees
      uint32_t qf[NT][D / 16][2];
      int lo[NT], hi[NT];
      int pos[NT];
      float slope[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = row0 + nt * 8 + g;
        const bool live = row < rows_all;
        const int i = static_cast<int>(p.by_group.div(live ? row : 0));
        const int h = head * p.G + (live ? row : 0) - i * p.G;
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + static_cast<int64_t>(rq.q0 + i) * p.q_token +
                              static_cast<int64_t>(h) * p.q_head + 2 * t;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          qf[nt][s][0] = live ? *reinterpret_cast<const uint32_t*>(src + s * 16) : 0u;
          qf[nt][s][1] = live ? *reinterpret_cast<const uint32_t*>(src + s * 16 + 8) : 0u;
        }
        lo[nt] = 0;
        hi[nt] = 0x7fffffff;
        pos[nt] = 0;
        slope[nt] = 0.f;
        if (live) {
          pos[nt] = position(p, rq, i);
          lo[nt] = first_key(p, pos[nt]);
          hi[nt] = last_key(p, rq, pos[nt]);
          if (p.slopes) slope[nt] = __ldg(p.slopes + h) * kLog2e;
          if (p.positions && i > 0 && __ldg(p.positions + rq.q0 + i - 1) > pos[nt]) bad |= HC_DEVERR_POS;
        }
      }

      float o[NT][D / 16][4], m[NT], l[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[nt][c][j] = 0.f;
        m[nt] = kNegInf;
        l[nt] = 0.f;
      }

      for (int i = 0; i < seg; ++i) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        const int key0 = key_first + i * kTile;
        if (i + kStages - 1 < seg) load_tile(key0 + (kStages - 1) * kTile, stage_to, slot);
        cp_async_commit();
        load_slots(key0 + kStages * kTile, slot);
        const uint32_t ks = stages_addr + stage_at, vs = ks + 4096;
        stage_to = stage_at;
        stage_at = stage_at == (kStages - 1) * L::kStageBytes ? 0 : stage_at + L::kStageBytes;
        if (key0 >= vis.hi || key0 + kKeys <= vis.lo) continue;

        // -- scores: S[row][key], keys 2t and 2t + 1 of each run of 8
        float s[NT][kKeys / 8][2];
#pragma unroll
        for (int n = 0; n < kKeys / 8; ++n) {
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          const int key = n * 8 + (lane & 7);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {  // 32 channels: 4 pieces of 16 bytes
            uint32_t kb[4];
            ldmatrix4(kb, ks + key * L::kRowBytes + swizzled(key, c * 4 + (lane >> 3)) * 16);
#pragma unroll
            for (int u = 0; u < 2; ++u)
              mma16<T>(acc, qf[0][c * 2 + u][0], NT == 2 ? qf[NT - 1][c * 2 + u][0] : 0u, qf[0][c * 2 + u][1],
                       NT == 2 ? qf[NT - 1][c * 2 + u][1] : 0u, kb[2 * u], kb[2 * u + 1]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            s[nt][n][0] = acc[2 * nt];
            s[nt][n][1] = acc[2 * nt + 1];
          }
        }

        // -- in units of log2; capped, less the bias, hidden where the row does not see the key
        float top[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (p.cap_log2 != 0.f) {
#pragma unroll
            for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
              for (int j = 0; j < 2; ++j) s[nt][n][j] = tanh_of(s[nt][n][j] * p.cap_in) * p.cap_log2;
          } else {
#pragma unroll
            for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
              for (int j = 0; j < 2; ++j) s[nt][n][j] *= p.scale_log2;
          }
          if (p.slopes) {
            const float away = static_cast<float>(pos[nt] - key0);  // positions themselves pass fp32's 24 bits
#pragma unroll
            for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                s[nt][n][j] = fmaf(-slope[nt], fabsf(away - static_cast<float>(n * 8 + 2 * t + j)), s[nt][n][j]);
          }
          if (key0 < lo[nt] || key0 + kKeys > hi[nt]) {
#pragma unroll
            for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int key = key0 + n * 8 + 2 * t + j;
                if (key < lo[nt] || key >= hi[nt]) s[nt][n][j] = kNegInf;
              }
          }
          top[nt] = kNegInf;
#pragma unroll
          for (int n = 0; n < kKeys / 8; ++n) top[nt] = fmaxf(top[nt], fmaxf(s[nt][n][0], s[nt][n][1]));
          top[nt] = fmaxf(top[nt], __shfl_xor_sync(0xffffffffu, top[nt], 1));
          top[nt] = fmaxf(top[nt], __shfl_xor_sync(0xffffffffu, top[nt], 2));
        }
        bool moves = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) moves = moves || top[nt] > m[nt];
        if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float to = fmaxf(m[nt], top[nt]);
            // nothing seen so far: l and O are 0, whatever they are multiplied by
            const float alpha = m[nt] == kNegInf ? 0.f : ex2(m[nt] - to);
            m[nt] = to;
            l[nt] *= alpha;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float a = __shfl_sync(0xffffffffu, alpha, (2 * t + j) * 4);
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                o[nt][c][j] *= a;
                o[nt][c][2 + j] *= a;
              }
            }
          }
        }
        uint32_t ph[NT][kKeys / 8], pl[NT][kKeys / 8];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float ref = m[nt] == kNegInf ? 0.f : m[nt] - kUp;
#pragma unroll
          for (int n = 0; n < kKeys / 8; ++n) {
            const float2 e = make_float2(ex2(s[nt][n][0] - ref), ex2(s[nt][n][1] - ref));
            l[nt] += e.x + e.y;
            split<T>(e, ph[nt][n], pl[nt][n]);
          }
        }

        // -- O^T += V^T P^T, 16 keys at a time
#pragma unroll
        for (int mt = 0; mt < kKeys / 16; ++mt) {
          const int key = mt * 16 + ((lane >> 4) & 1) * 8 + (lane & 7);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t va[4];
            ldmatrix4_trans(va, vs + key * L::kRowBytes + swizzled(key, c * 2 + ((lane >> 3) & 1)) * 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16<T>(o[nt][c], va[0], va[1], va[2], va[3], ph[nt][2 * mt], ph[nt][2 * mt + 1]);
              mma16<T>(o[nt][c], va[0], va[1], va[2], va[3], pl[nt][2 * mt], pl[nt][2 * mt + 1]);
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
        float sum = l[nt];
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
            so[(warp * kRows + row) * D + c * 16 + g] = o[nt][c][j];
            so[(warp * kRows + row) * D + c * 16 + 8 + g] = o[nt][c][2 + j];
          }
        }
      }
      __syncthreads();
      const bool whole = seg == vis.tiles;
      float* ws = reinterpret_cast<float*>(p.workspace + kMaxCtas * sizeof(int32_t));
      int32_t* counters = reinterpret_cast<int32_t*>(p.workspace);
      auto part_of = [&](uint32_t run, bool starts) {  // partial sums of a run: of the piece that starts in it, or goes on
        return ws + ((static_cast<int64_t>(run) * p.H + head) * 2 + (starts ? 1 : 0)) * kPartialFloats;
      };
      float* partial = part_of(b, first == 0);

      auto write_row = [&](int row, int ch, float4 v, float mref, float sum) {
        // v: unnormalised sums of 4 channels
        const int rr = row0 + row, i = static_cast<int>(p.by_group.div(rr)), h = head * p.G + rr - i * p.G;
        const int64_t tok = rq.q0 + i;
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        uint2 w;
        w.x = pack<T>(v.x * inv, v.y * inv);
        w.y = pack<T>(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + tok * p.o_token + h * p.o_head + ch) = w;
        if (p.lse && ch == 0)
          p.lse[tok * (static_cast<int64_t>(p.H) * p.G) + h] = sum > 0.f ? (mref - kUp + log2f(sum)) * kLn2 : kNegInf;
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
        // the runs that hold a part of this piece: first to last
        const uint32_t u0 = unit - off + p.piece_cost, u1 = u0 + vis.tiles - 1;
        auto owner = [&](uint32_t u) {
          const uint32_t big = extra * (share + 1);
          return u < big ? u / (share + 1) : extra + (u - big) / share;
        };
        const uint32_t c0 = owner(u0), c1 = owner(u1);
        int32_t* counter = counters + c0 * p.H + head;
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          const int arrived = atomicAdd(counter, 1);
          sh.last = arrived == static_cast<int>(c1 - c0);
          if (sh.last) *counter = 0;
          __threadfence();
        }
        __syncthreads();
        if (sh.last) {
          // in the order of the CTAs, kAtOnce partial sums on their way together
          auto part = [&](uint32_t c) { return part_of(min(c, c1), min(c, c1) == c0); };
          constexpr int kAtOnce = 8;
          for (int id = tid; id < rows * (D / 4); id += kWarpsA * 32) {
            const int row = id / (D / 4), ch = (id % (D / 4)) * 4;
            float top = kNegInf, sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (uint32_t c = c0; c <= c1; c += kAtOnce) {
              float m_part[kAtOnce], l_part[kAtOnce];
              float4 v[kAtOnce];
#pragma unroll
              for (int u = 0; u < kAtOnce; ++u) {
                const float* from = part(c + u);
                m_part[u] = __ldcg(from + row);
                l_part[u] = __ldcg(from + kMaxRows + row);
                v[u] = __ldcg(reinterpret_cast<const float4*>(from + 2 * kMaxRows + row * D + ch));
              }
#pragma unroll
              for (int u = 0; u < kAtOnce; ++u) {
                if (c + u > c1 || m_part[u] == kNegInf) continue;
                const float to = fmaxf(top, m_part[u]), old = ex2(top - to), wt = ex2(m_part[u] - to);  // top -inf: old 0
                top = to;
                sum = sum * old + wt * l_part[u];
                acc.x = acc.x * old + wt * v[u].x, acc.y = acc.y * old + wt * v[u].y;
                acc.z = acc.z * old + wt * v[u].z, acc.w = acc.w * old + wt * v[u].w;
              }
            }
            write_row(row, ch, acc, top, sum);
          }
        }
      }
    }

    // ---- the next piece
    unit += taken;
    off = 0;
    if (unit < end) {
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
    __syncthreads();
  }
  flag_error(p.err, bad & (HC_DEVERR_SLOT | HC_DEVERR_POS));
}

template <typename T, int D, int NT>
cudaError_t launch_rows(AttendPagedParams p, cudaStream_t s) {
  using L = Layout<D>;
  const int smem = std::max(kWarpsA * L::kWarpBytes, kWarpsA * 8 * NT * D * 4);
  static KernelOnDevice kernel;
  int resident = 0;
  const cudaError_t e =
      kernel.resident(reinterpret_cast<const void*>(k_attend_paged_rows<T, D, NT>), kWarpsA * 32, smem, &resident);
  if (e != cudaSuccess) return e;
  // one CTA per resident place, or per tile where there are fewer (as far as the host can tell), the same
  // number for every head; with more heads than places each head is one CTA's, and nothing is joined
  const int64_t rows = (std::min<int64_t>(static_cast<int64_t>(p.max_new) * p.G, p.rows_above) + 8 * NT - 1) / (8 * NT);
  const int64_t keys = static_cast<int64_t>(p.table_width) << p.B_log2;
  const int64_t tiles = std::max<int64_t>(1, (keys + L::kTile - 1) / L::kTile);
  int64_t runs = std::max(1, std::min(kMaxCtas, resident) / p.H);
  p.piece_cost = kPieceCost;
  if (static_cast<double>(p.n_req) * rows * tiles < static_cast<double>(runs)) {
    runs = p.n_req * rows * tiles;
    p.piece_cost = 0;
  }
  k_attend_paged_rows<T, D, NT><<<static_cast<unsigned>(runs * p.H), kWarpsA * 32, smem, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_type(const AttendPagedParams& p, cudaStream_t s) {
  const bool few = std::min<int64_t>(static_cast<int64_t>(p.max_new) * p.G, p.rows_above) <= 8;
  if (p.bf16) return few ? launch_rows<__nv_bfloat16, D, 1>(p, s) : launch_rows<__nv_bfloat16, D, 2>(p, s);
  return few ? launch_rows<__half, D, 1>(p, s) : launch_rows<__half, D, 2>(p, s);
}

}  // namespace

int64_t attend_paged_counter_bytes() { return kMaxCtas * static_cast<int64_t>(sizeof(int32_t)); }

int64_t attend_paged_rows_bytes() {
  return attend_paged_counter_bytes() +
         static_cast<int64_t>(kMaxCtas) * 2 * kPartialFloats * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_attend_paged_rows(int d, const AttendPagedParams& p, cudaStream_t s) {
  return d == 64 ? launch_type<64>(p, s) : launch_type<128>(p, s);
}

}  // namespace hc
