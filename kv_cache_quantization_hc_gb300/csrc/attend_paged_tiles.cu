// Attention of the new tokens over the paged buffer, many query rows: tiles of
// 256 rows (new tokens times the query heads of one cache head) against tiles
// of 128 keys on the 5th-generation tensor cores.
//
// One CTA per SM takes runs of 256 rows one after another, the longest first
// (k-th run: number k * CTAs + i, or the mirror of it for odd k, which evens
// the sums out).  Its 12 warps each go through the runs by themselves, so that
// one's keys are loaded while the last one's result is still written:
//   warps 0-3, 4-7  the softmax of rows 0-127 and 128-255, a thread per row;
//   warp 8          keys and values by TMA, a block of the buffer at a time;
//   warp 9          one thread issues the products: S = Q K^T into tensor
//                   memory, O += P V with P from tensor memory;
//   warp 10         finds the runs, up to four ahead;
//   warp 11         zeros in place of values that no row sees.
// While one half's softmax runs, the other half's products do: per half the
// order is S(j), softmax(j), O += P(j) V(j), S(j + 1).  Tensor memory is full:
// two S of 128 columns, over which P is written, and two O of d.
//
// Mathematics, per row, over tiles of keys from the last to the first:
//   x_j = the score of key j in units of log2, p_j = 2^(x_j - m + top),
//   l = sum p_j,  O = sum p_j v_j,  out = O / l
// * Queries, keys and values enter the products as they are stored, scores and
//   sums are fp32, and probabilities enter in the values' type: one of 8 bits
//   (bf16) or 11 (fp16), as the output is, whose sum over keys is as exact as
//   one output's rounding.
// * From the last tile to the first: the tile that rows see partly, which takes
//   two passes, is also the one that sets the reference m, which takes two as
//   well; and a bias by distance has its largest scores there.
// * bf16 has fp32's range, so m is the maximum of the first tile and moves only
//   when a tile's probabilities sum up to 2^40; no maximum is looked for
//   otherwise.  fp16 ends at 65504: top = 11.5, m is 3 above the maximum and
//   moves when that exceeds m by 3.5 or a tile's sum passes 60000; a
//   probability keeps 11 bits down to 2^-22 of the largest.  Rows that see n
//   keys in all, fewer than a tile, have m 128 / n times lower.
//
// Bound: the tensor cores (4 d flops per row and key).
#include <algorithm>
#include <climits>
#include <cuda.h>

#include "attend_paged_common.cuh"
#include "mbarrier.cuh"
#include "tcgen05.cuh"

namespace hc {
namespace {

constexpr int kKeys = 128;       // keys of a tile
constexpr int kHalf = 128;       // rows of a half
constexpr int kRowsTile = 2 * kHalf;
constexpr int kSoftmaxWarps = 8, kLoadWarp = 8, kProductWarp = 9, kWorkWarp = 10, kEdgeWarp = 11;
constexpr int kThreadsTiles = 12 * 32;
constexpr int kWorksAhead = 4;   // found before they are begun
constexpr int kBlockBytes = kKeys * 128;  // 128 rows of 64 channels, swizzled in 128-byte rows

// p = 2^(x - m + kTop); see above.
template <bool kBf16>
struct Softmax;
template <>
struct Softmax<true> {
  static constexpr float kTop = 0.f, kMoveAt = 0.f, kAhead = 0.f, kMostSum = 0x1p40f;
};
template <>
struct Softmax<false> {
  static constexpr float kTop = 11.5f, kMoveAt = 3.5f, kAhead = 3.f, kMostSum = 60000.f;
};

template <int D>
struct TileSmem {
  static constexpr int kTileBytes = D / 64 * kBlockBytes;
  static constexpr int kQ = 0, kK = 2 * kTileBytes, kV = kK + 2 * kTileBytes;
  static constexpr int kBytes = kV + 2 * kTileBytes;
  // with 1 KiB to align, and enough for one CTA per SM: each takes all of tensor memory
  static constexpr int kAsk = (kBytes > 120 * 1024 ? kBytes : 120 * 1024) + 1024;
};

// Work of a CTA: 256 rows of one request and cache head.
struct alignas(16) Work {
  PagedRequest rq;
  int r, head, row0, rows_all, tiles;  // tiles 0: no work, the CTA is done
  Range vis;
};
// Tile j of a work, from the last one on: its first key.
__device__ __forceinline__ int tile_key(const Range& v, int j) { return (v.tile0 + v.tiles - 1 - j) * kKeys; }
// Whether some key of the tile is seen by no row of the work.
__device__ __forceinline__ bool at_edge(const Range& v, int key0) { return key0 < v.lo || key0 + kKeys > v.hi; }

struct TileShared {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], v_edge[2], s_full[2], p_full[2], q_full[2],
      work_full[kWorksAhead], work_empty[kWorksAhead], drain;
  uint32_t tmem;
  int32_t dead;               // some wait ran out
  Work work[kWorksAhead];     // work k at k % kWorksAhead
};

__device__ __forceinline__ void mbar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(mbar_addr(b)), "r"(bytes) : "memory");
}
// Issued by one thread, like the products, while the whole warp goes along.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint64_t* b, int channel, int head, int slot,
                                         uint32_t leader) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.ne.u32 q, %7, 0;\n"
      "@q cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];\n}" ::"r"(
          dst),
      "l"(map), "r"(mbar_addr(b)), "r"(channel), "r"(head), "r"(0), "r"(slot), "r"(leader)
      : "memory");
}

// Number `idx` of the call's works, found by a warp (all lanes get it); false
// past the last.  `c` goes forward only, so idx may not fall.
//
// The order: works whose last rows see the most keys, by powers of two; within
// one, by request and from its last rows.  Each class goes through the requests
// again, so many requests, which even out by themselves, are one class.
constexpr int kFewestKeys = 256, kMostRequests = 256;
struct Cursor {
  int r0 = 0, before = 0;  // first request of 32, works of those before it
  int upto;                // the works of this class see fewer keys
  __device__ __forceinline__ explicit Cursor(const AttendPagedParams& p) {
    const int64_t keys = static_cast<int64_t>(p.table_width) << p.B_log2;
    upto = p.n_req > kMostRequests || keys >= 1 << 30 ? INT_MAX : 1 << (32 - __clz(static_cast<int>(keys)));
  }
};
// Runs of 256 rows of a request, of `runs` in all, whose last row's keys end at
// `key` or later; positions do not fall, so they are the last ones.
__device__ __forceinline__ int runs_seeing(const AttendPagedParams& p, const PagedRequest& q, int runs, int key) {
  if (key <= 0) return runs;
  int lo = 0, hi = runs;  // the first such run
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    const int row = min((mid + 1) * kRowsTile, q.n * p.G) - 1;
    if (last_key(p, q, position(p, q, static_cast<int>(p.by_group.div(row)))) >= key)
      hi = mid;
    else
      lo = mid + 1;
  }
  return runs - lo;
}
__device__ __forceinline__ bool find_work(const AttendPagedParams& p, Cursor& c, int idx, int lane, Work& w) {
  for (;;) {
    const int from = p.n_req > kMostRequests || c.upto <= kFewestKeys ? 0 : c.upto == INT_MAX ? 1 << 30 : c.upto >> 1;
    for (; c.r0 < p.n_req; c.r0 += 32) {
      PagedRequest q{0, 0, 0, 0};
      int bad = 0;  // lengths are reported by k_attend_paged_rows
      if (c.r0 + lane < p.n_req) q = load_request(p, c.r0 + lane, bad);
      const int rows = q.n * p.G > p.rows_above ? q.n * p.G : 0;
      const int runs = (rows + kRowsTile - 1) / kRowsTile;
      const int to_end = runs_seeing(p, q, runs, from);
      // positions that fall, which are flagged, may make this negative
      const int works = max(0, to_end - runs_seeing(p, q, runs, c.upto)) * p.H;
      int inc = works;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const uint32_t upto = __ballot_sync(0xffffffffu, idx < c.before + inc);
      if (upto == 0) {
        c.before += __shfl_sync(0xffffffffu, inc, 31);
        continue;
      }
      const int src = __ffs(static_cast<int>(upto)) - 1;
      w.r = c.r0 + src;
      w.rq = {__shfl_sync(0xffffffffu, q.q0, src), __shfl_sync(0xffffffffu, q.n, src),
              __shfl_sync(0xffffffffu, q.kv, src), __shfl_sync(0xffffffffu, q.prefix, src)};
      w.rows_all = __shfl_sync(0xffffffffu, rows, src);
      const int left = __shfl_sync(0xffffffffu, c.before + inc, src) - 1 - idx;  // the last rows first
      const int run = left / p.H;
      w.head = left - run * p.H;
      w.row0 = (__shfl_sync(0xffffffffu, runs - to_end, src) + run) * kRowsTile;
      w.vis = visible<kKeys>(p, w.rq, w.row0, min(w.row0 + kRowsTile, w.rows_all));
      w.tiles = w.vis.tiles;
      return true;
    }
    if (from == 0) return false;
    c.upto = from;
    c.r0 = 0;
  }
}
__device__ __forceinline__ int work_number(int k) {
  const int g = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
  return k * g + (k & 1 ? g - 1 - b : b);
}

// kMods: scores are capped or have a bias.
template <bool kBf16, int D, bool kMods>
__global__ void __launch_bounds__(kThreadsTiles, 1)
    k_attend_paged_tiles(const __grid_constant__ AttendPagedParams p, const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map) {
  using Smem = TileSmem<D>;
  using Soft = Softmax<kBf16>;
  extern __shared__ unsigned char dyn_raw[];
  __shared__ TileShared sh;
  unsigned char* const dyn = dyn_raw + (1024 - (smem_addr(dyn_raw) & 1023)) % 1024;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  int bad = 0;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_empty[i], 1);
      mbar_init(&sh.v_edge[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], kHalf);
      mbar_init(&sh.q_full[i], kHalf);
    }
    for (int i = 0; i < kWorksAhead; ++i) {
      mbar_init(&sh.work_full[i], 1);
      mbar_init(&sh.work_empty[i], kThreadsTiles / 32 - 1);
    }
    mbar_init(&sh.drain, 1);
    sh.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kProductWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }

  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh.tmem;
  bool ok = true;
  int base = 0;  // tiles of the works so far
  // Work k is read where it is needed, which leaves the registers to the loops.
  auto take_work = [&](int k) {  // false: none left (or a wait ran out)
    const bool there = mbar_wait(&sh.work_full[k % kWorksAhead], (k / kWorksAhead) & 1, &sh.dead);
    ok = __all_sync(0xffffffffu, ok && there);
    return ok && sh.work[k % kWorksAhead].tiles > 0;
  };
  auto leave_work = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.work_empty[k % kWorksAhead]);
  };

  if (warp < kSoftmaxWarps) {
    // ================================================== softmax
    const int half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes of tensor memory per warp
    const uint32_t s_at = tmem + lanes + half * 128, o_at = tmem + lanes + 256 + half * D;
    // A row's 16-byte pieces belong to D / 8 lanes where rows are read and written.
    constexpr int kLanes = D / 8, kRowsAt = 32 / kLanes;
    const int piece = lane % kLanes;
    unsigned char* const rows_smem = dyn + Smem::kQ + half * Smem::kTileBytes + (warp & 3) * 32 * 128;
    auto piece_at = [&](int at, int c) {  // piece c of the warp's row `at`: queries, then the result
      return reinterpret_cast<uint4*>(rows_smem + (c / 8) * kBlockBytes + at * 128 + (((c % 8) ^ (at & 7)) << 4));
    };
    auto pack2 = [](float lo, float hi) { return kBf16 ? pack_bf16(lo, hi) : pack_f16(lo, hi); };
    for (int k = 0; take_work(k); ++k) {
      const Work& work = sh.work[k % kWorksAhead];
      const int tiles = work.tiles, row = work.row0 + tid;
      auto row_offset = [&](int rr, int64_t token, int64_t head_stride) {  // of row rr in q or out
        const int i = static_cast<int>(p.by_group.div(rr));
        return static_cast<int64_t>(work.rq.q0 + i) * token +
               static_cast<int64_t>(work.head * p.G + rr - i * p.G) * head_stride;
      };
      // ---- queries
      const int row_first = work.row0 + warp * 32 + lane / kLanes;
#pragma unroll 1
      for (int r0 = 0; r0 < 32; r0 += 8 * kRowsAt) {
        uint4 raw[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int rr = row_first + r0 + u * kRowsAt;
          raw[u] = make_uint4(0, 0, 0, 0);
          if (rr < work.rows_all)
            raw[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                     row_offset(rr, p.q_token, p.q_head) + piece * 8);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) *piece_at(r0 + u * kRowsAt + lane / kLanes, piece) = raw[u];
      }
      fence_async();
      mbar_arrive(&sh.q_full[half]);
      // keys that the thread's row sees; rows past the last see what the work sees
      int first = work.vis.lo, last = work.vis.hi;
      float pos_f = 0.f, slope = 0.f;
      if (row < work.rows_all) {
        const int i = static_cast<int>(p.by_group.div(row));
        const int pos = position(p, work.rq, i);
        first = first_key(p, pos);
        last = last_key(p, work.rq, pos);
        if (kMods) {
          pos_f = static_cast<float>(pos);
          if (p.slopes) slope = __ldg(p.slopes + work.head * p.G + row - i * p.G) * kLog2e;
        }
      }
      __syncwarp();

      float m = kNegInf, l = 0.f;
      for (int j = 0; j < tiles && ok; ++j) {
        ok = mbar_wait(&sh.s_full[half], (base + j + k) & 1, &sh.dead);
        if (!__all_sync(0xffffffffu, ok)) break;
        fence_after();
        const int key0 = tile_key(work.vis, j);
        // Most tiles: all of it seen, by rows that have a reference, and no score far above that.  One pass then,
        // with P kept in registers until its sum is known, since it goes over the scores.
        const bool masked = __any_sync(0xffffffffu, key0 < first || key0 + kKeys > last || m == kNegInf);
        float sum = 0.f;
        bool done = false, crowded = false;  // crowded: the sum was too large
        if (!kMods && !masked) {
          uint32_t x[2][16], h[2][32];
          const float2 f2 = make_float2(p.scale_log2, p.scale_log2), off2 = make_float2(Soft::kTop - m, Soft::kTop - m);
          float2 part = make_float2(0.f, 0.f);
          tmem_load16(x[0], s_at);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t(&y)[16] = x[c & 1];
            tmem_wait_load16(y);
            if (c < 7) tmem_load16(x[(c & 1) ^ 1], s_at + (c + 1) * 16);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float2 v = __ffma2_rn(make_float2(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), f2, off2);
              v.x = ex2(v.x);
              v.y = ex2(v.y);
              part = __fadd2_rn(part, v);
              h[c / 4][(c % 4) * 8 + i / 2] = pack2(v.x, v.y);
            }
          }
          sum = part.x + part.y;
          done = __all_sync(0xffffffffu, sum < Soft::kMostSum);
          crowded = !done;
          if (done) {
            tmem_store32(s_at, h[0]);
            tmem_store32(s_at + 32, h[1]);
          }
        }
        if (!done) {
          const int lo = first - key0, hi = last - key0;  // columns [lo, hi) count
          sum = 0.f;
          uint32_t a[32];
          float top = kNegInf;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_load32(a, s_at + c * 32);
            tmem_wait_load(a);
            // in units of log2, with what is hidden at -inf, where the scores are
            const int n = min(max(hi - c * 32, 0), 32), skip = min(max(lo - c * 32, 0), 32);
            const uint32_t seen = (n == 32 ? ~0u : (1u << n) - 1u) & (skip == 32 ? 0u : ~0u << skip);
            if (kMods) {
              const float away = pos_f - static_cast<float>(key0 + c * 32);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                float x = __uint_as_float(a[i]);
                x = p.cap_log2 != 0.f ? tanh_of(x * p.cap_in) * p.cap_log2 : x * p.scale_log2;
                x = fmaf(-slope, fabsf(away - static_cast<float>(i)), x);
                a[i] = __float_as_uint(x);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) a[i] = __float_as_uint(__uint_as_float(a[i]) * p.scale_log2);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (!(seen >> i & 1u)) a[i] = __float_as_uint(kNegInf);
              top = fmaxf(top, __uint_as_float(a[i]));
            }
            tmem_store32(s_at + c * 32, a);
          }
          wait_store();
          // the reference of the row, and O with it
          float ahead = Soft::kAhead;
          if (!kBf16) {  // n keys in all, fewer than a tile: 128 / n times lower, as n of them do not pass kMostSum either
            const int n = last - first;
            if (n < kKeys) ahead -= static_cast<float>(__clz(max(n - 1, 0)) - __clz(kKeys - 1));
          }
          const float m_new =
              top > m + (crowded ? -Soft::kAhead : Soft::kMoveAt) || (m == kNegInf && top > m) ? top + ahead : m;
          if (__any_sync(0xffffffffu, m_new != m)) {
            const float by = m == kNegInf ? 0.f : ex2(m - m_new);
            l *= by;
            if (j > 0) {
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                tmem_load32(a, o_at + c * 32);
                tmem_wait_load(a);
#pragma unroll
                for (int i = 0; i < 32; ++i) a[i] = __float_as_uint(__uint_as_float(a[i]) * by);
                tmem_store32(o_at + c * 32, a);
              }
            }
            m = m_new;
          }
          const float off = m == kNegInf ? 0.f : Soft::kTop - m;
          float2 part = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t h[16];
            tmem_load32(a, s_at + c * 32);
            tmem_wait_load(a);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 v = make_float2(ex2(__uint_as_float(a[i]) + off), ex2(__uint_as_float(a[i + 1]) + off));
              part = __fadd2_rn(part, v);
              h[i / 2] = pack2(v.x, v.y);
            }
            tmem_store16(s_at + c * 16, h);  // over columns already read
          }
          sum = part.x + part.y;
        }
        l += sum;
        wait_store();
        fence_before();
        mbar_arrive(&sh.p_full[half]);
      }
      base += tiles;
      // ---- the result, through the queries' place in shared memory, which no product reads any more
      ok = ok && mbar_wait(&sh.s_full[half], (base + k) & 1, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      fence_after();
      const float by = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        tmem_load32(x, o_at + c * 32);
        tmem_wait_load(x);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = pack2(__uint_as_float(x[u * 8 + 2 * i]) * by, __uint_as_float(x[u * 8 + 2 * i + 1]) * by);
          *piece_at(lane, c * 4 + u) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      fence_before();
      if (p.lse && row < work.rows_all)
        p.lse[row_offset(row, static_cast<int64_t>(p.H) * p.G, 1)] =
            l > 0.f ? (m - Soft::kTop + log2f(l)) * kLn2 : kNegInf;
      __syncwarp();
#pragma unroll 4
      for (int r0 = 0; r0 < 32; r0 += kRowsAt) {
        const uint4 w = *piece_at(r0 + lane / kLanes, piece);
        if (row_first + r0 < work.rows_all)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row_offset(row_first + r0, p.o_token, p.o_head) +
                                    piece * 8) = w;
      }
      __syncwarp();
      leave_work(k);
    }
  } else if (warp == kLoadWarp) {
    // ================================================== keys and values
    // A box is 64 channels of the tile's rows in one slot; lane i looks slot i up.  Rows of a slot that does not
    // exist, or that no row sees, come from past the buffer's end, where the copy finds zeros.
    const int block = 1 << p.B_log2, slots = kKeys >> p.B_log2;
    const uint32_t leader = elect_leader(), tiles_at = __shfl_sync(0xffffffffu, smem_addr(dyn), 0);
    // bit st: the parity of v_edge[st]'s next use, and whether the last values into stage st went by it
    uint32_t edges = 0, by_edge = 0;
    int k_sent = 0, v_sent = 0;  // tiles on their way so far
    for (int k = 0; take_work(k); ++k) {
      const Work& work = sh.work[k % kWorksAhead];
      const Range vis = work.vis;
      const int head = work.head, tiles = work.tiles;
      const int32_t* const table = p.tables + static_cast<int64_t>(work.r) * p.table_stride;
      auto slot_of = [&](int j) {
        int slot = p.num_slots;
        if (lane < slots && j < tiles) {
          const int key = tile_key(vis, j) + lane * block;
          if (key < vis.hi && key + block > vis.lo) {
            slot = __ldg(table + (key >> p.B_log2));
            if (static_cast<uint32_t>(slot) >= static_cast<uint32_t>(p.num_slots)) {
              bad |= HC_DEVERR_SLOT;
              slot = p.num_slots;
            }
          }
        }
        return slot;
      };
      auto load = [&](uint32_t dst, const CUtensorMap* map, uint64_t* full, int slot) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i >= slots) break;
          const int s = __shfl_sync(0xffffffffu, slot, i);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load(dst + c * kBlockBytes + i * (block * 128), map, full, c * 64, head, s, leader);
        }
      };
      int slot = slot_of(0);
      for (int j = 0; j < tiles; ++j) {
        const int st = (base + j) & 1, round = (base + j) >> 1;
        const int next = slot_of(j + 1);
        if (base + j >= 2) ok = mbar_wait(&sh.k_empty[st], (round - 1) & 1, &sh.dead);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lane == 0) mbar_expect(&sh.k_full[st], Smem::kTileBytes);
        __syncwarp();
        ++k_sent;
        load(tiles_at + Smem::kK + st * Smem::kTileBytes, &k_map, &sh.k_full[st], slot);
        if (base + j >= 2) ok = mbar_wait(&sh.v_empty[st], (round - 1) & 1, &sh.dead);
        if (!__all_sync(0xffffffffu, ok)) break;
        const bool edge = at_edge(vis, tile_key(vis, j));
        uint64_t* const full = edge ? &sh.v_edge[st] : &sh.v_full[st];
        if (lane == 0) mbar_expect(full, Smem::kTileBytes);
        __syncwarp();
        ++v_sent;
        by_edge = (by_edge & ~(1u << st)) | static_cast<uint32_t>(edge) << st;
        if (edge) edges ^= 1u << st;
        load(tiles_at + Smem::kV + st * Smem::kTileBytes, &v_map, full, slot);
        slot = next;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      base += tiles;
      leave_work(k);
    }
    if (!ok) {  // a wait ran out: copies may still be on their way into shared memory
      int32_t no = 0;
      for (int n = max(k_sent - 2, 0); n < k_sent; ++n) mbar_wait(&sh.k_full[n & 1], (n >> 1) & 1, &no);
      for (int n = max(v_sent - 2, 0); n < v_sent; ++n) {
        const int st = n & 1;
        if (by_edge >> st & 1u)
          mbar_wait(&sh.v_edge[st], ~(edges >> st) & 1u, &no);
        else
          mbar_wait(&sh.v_full[st], (n >> 1) & 1, &no);
      }
      __syncwarp();
    }
  } else if (warp == kEdgeWarp) {
    // ================================================== values that no row sees: 0 times them must be 0
    if (p.positions)  // of the requests r = blockIdx.x mod gridDim.x: whether positions fall
      for (int r = blockIdx.x; r < p.n_req; r += gridDim.x) {
        int dummy = 0;
        const PagedRequest q = load_request(p, r, dummy);
        for (int i = 1 + lane; i < q.n; i += 32)
          if (position(p, q, i) < position(p, q, i - 1)) bad |= HC_DEVERR_POS;
      }
    uint32_t edges = 0;  // bit st: the parity of v_edge[st]'s next use
    for (int k = 0; take_work(k); ++k) {
      const Range vis = sh.work[k % kWorksAhead].vis;
      leave_work(k);
      for (int j = 0; j < vis.tiles && ok; ++j) {
        const int key0 = tile_key(vis, j), st = (base + j) & 1;
        if (!at_edge(vis, key0)) continue;
        ok = mbar_wait(&sh.v_edge[st], edges >> st & 1u, &sh.dead);
        if (!__all_sync(0xffffffffu, ok)) break;
        edges ^= 1u << st;
        unsigned char* const tile = dyn + Smem::kV + st * Smem::kTileBytes;
        for (int i = lane; i < kKeys * (D / 8); i += 32) {
          const int key = (i / 8) % kKeys;
          if (key0 + key < vis.lo || key0 + key >= vis.hi) *reinterpret_cast<uint4*>(tile + i * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.v_full[st]);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      base += vis.tiles;
    }
  } else if (warp == kWorkWarp) {
    // ================================================== works, found ahead of the warps that do them
    Cursor cursor(p);
    Work work;
    for (int k = 0;; ++k) {
      const bool more = find_work(p, cursor, work_number(k), lane, work);
      if (!more) work.tiles = 0;
      if (k >= kWorksAhead)
        ok = mbar_wait(&sh.work_empty[k % kWorksAhead], (k / kWorksAhead - 1) & 1, &sh.dead);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) {
        sh.work[k % kWorksAhead] = work;
        mbar_arrive(&sh.work_full[k % kWorksAhead]);
      }
      if (!more) break;
    }
    __syncwarp();
  } else {
    // ================================================== products
    const uint32_t leader = elect_leader();
    const uint32_t at = __shfl_sync(0xffffffffu, tmem, 0), tiles_at = __shfl_sync(0xffffffffu, smem_addr(dyn), 0);
    auto scores = [&](int i, int j) {  // S_i = Q_i K(j)^T
      const uint64_t q = smem_desc(tiles_at + Smem::kQ + i * Smem::kTileBytes, 16);
      const uint64_t k = smem_desc(tiles_at + Smem::kK + (j & 1) * Smem::kTileBytes, 16);
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const uint64_t step = ((s / 4) * kBlockBytes + (s % 4) * 32) >> 4;
        mma_smem(at + i * 128, q + step, k + step, instr_desc(kKeys, false, kBf16), s > 0, leader);
      }
      commit(&sh.s_full[i], leader);
    };
    auto values = [&](int i, int j, bool add) {  // O_i (+)= P_i(j) V(j)
      const uint64_t v = smem_desc(tiles_at + Smem::kV + (j & 1) * Smem::kTileBytes, kBlockBytes);
#pragma unroll
      for (int s = 0; s < kKeys / 16; ++s)
        mma_tmem(at + 256 + i * D, at + i * 128 + s * 8, v + s * (2048 >> 4), instr_desc(D, true, kBf16), add || s > 0, leader);
    };
    for (int k = 0; ok && take_work(k); ++k) {
      const int tiles = sh.work[k % kWorksAhead].tiles;
      leave_work(k);
      for (int j = 0; j <= tiles && ok; ++j) {
        const int jj = base + j;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (j > 0) {
            ok = ok && mbar_wait(&sh.v_full[(jj - 1) & 1], ((jj - 1) >> 1) & 1, &sh.dead) &&
                 mbar_wait(&sh.p_full[i], (jj - 1) & 1, &sh.dead);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            fence_after();
            values(i, jj - 1, j > 1);
            if (i == 1) commit(&sh.v_empty[(jj - 1) & 1], leader);
          }
          if (j < tiles) {
            ok = (j > 0 || mbar_wait(&sh.q_full[i], k & 1, &sh.dead)) &&
                 mbar_wait(&sh.k_full[jj & 1], (jj >> 1) & 1, &sh.dead);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            fence_after();
            scores(i, jj);
            if (i == 1) commit(&sh.k_empty[jj & 1], leader);
          } else {
            commit(&sh.s_full[i], leader);  // O_i is complete
          }
        }
      }
      base += tiles;
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == kProductWarp) {
    if (sh.dead) {  // products may still be on their way: wait for them before their memory goes
      if (lane == 0) flag_error(p.err, HC_DEVERR_WAIT);
      int32_t no = 0;
      commit(&sh.drain, elect_leader());
      mbar_wait(&sh.drain, 0, &no);
      __syncwarp();
    }
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
  if (bad) flag_error(p.err, bad);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// The driver's encoder, found through the runtime, so that the library needs no libcuda to load.
EncodeTiled encode_tiled() {
  static const EncodeTiled found = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult at;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &at);
    return e == cudaSuccess && at == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiled>(f) : nullptr;
  }();
  return found;
}

// Pages as [slot][token][head][channel], copied 64 channels of a head's tokens of one slot at a time into 128-byte
// swizzled rows.
template <bool kBf16>
cudaError_t pages_map(CUtensorMap* map, const void* pages, const AttendPagedParams& p, int d) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t block = cuuint64_t{1} << p.B_log2, row = 2 * static_cast<cuuint64_t>(d);
  const cuuint64_t sizes[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(p.H), block,
                               static_cast<cuuint64_t>(p.num_slots)};
  const cuuint64_t strides[3] = {row, row * p.H, 2 * static_cast<cuuint64_t>(p.slot_stride)};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(std::min<cuuint64_t>(block, kKeys)), 1}, step[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                            const_cast<void*>(pages), sizes, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool kBf16, int D, bool kMods>
cudaError_t launch(const AttendPagedParams& p, cudaStream_t s) {
  static KernelOnDevice kernel;
  int resident = 0;
  cudaError_t e = kernel.resident(reinterpret_cast<const void*>(k_attend_paged_tiles<kBf16, D, kMods>), kThreadsTiles,
                                  TileSmem<D>::kAsk, &resident);
  if (e != cudaSuccess) return e;
  CUtensorMap k_map, v_map;
  e = pages_map<kBf16>(&k_map, p.k_pages, p, D);
  if (e == cudaSuccess) e = pages_map<kBf16>(&v_map, p.v_pages, p, D);
  if (e != cudaSuccess) return e;
  const int64_t runs = (static_cast<int64_t>(p.max_new) * p.G + kRowsTile - 1) / kRowsTile;
  const double works = static_cast<double>(runs) * p.n_req * p.H;
  const int grid = works < resident ? static_cast<int>(works) : resident;
  k_attend_paged_tiles<kBf16, D, kMods><<<grid, kThreadsTiles, TileSmem<D>::kAsk, s>>>(p, k_map, v_map);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_type(const AttendPagedParams& p, cudaStream_t s) {
  const bool mods = p.cap_log2 != 0.f || p.slopes != nullptr;
  if (p.bf16) return mods ? launch<true, D, true>(p, s) : launch<true, D, false>(p, s);
  return mods ? launch<false, D, true>(p, s) : launch<false, D, false>(p, s);
}

}  // namespace

cudaError_t launch_attend_paged_tiles(int d, const AttendPagedParams& p, cudaStream_t s) {
  return d == 64 ? launch_type<64>(p, s) : launch_type<128>(p, s);
}

}  // namespace hc
