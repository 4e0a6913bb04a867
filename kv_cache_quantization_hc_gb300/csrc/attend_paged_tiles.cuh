// Attention of the new tokens over the paged buffer, many query rows: tiles of
// 256 rows (new tokens times the query heads of one cache head) against tiles
// of 128 keys on the 5th-generation tensor cores.
//
// One CTA per SM takes runs of 256 rows as they come, the longest first.  Its 16
// warps each go through the runs by themselves, so that one's keys are loaded
// while the last one's result is still written (runs in a fixed order, and queries
// and results by the softmax's warps: 8192 tokens 334 us, like this 314):
//   warps 0-3, 4-7  the softmax of rows 0-127 and 128-255, a thread per row;
//   warp 8          keys and values by TMA, a block of the buffer at a time,
//                   issued by one thread (by a lane per copy: 387 us);
//   warp 9          one thread issues the products: S = Q K^T into tensor
//                   memory, O += P V with P from tensor memory;
//   warp 10         finds the next run;
//   warp 11         zeros in place of values that no row sees;
//   warps 12-15     the next run's queries, and the last one's result.
// Where a call has few runs, their tiles are shared out as well (SplitRule), and
// the parts' sums joined by a second kernel: 512 tokens over 30000 keys 190 us,
// 64 rows of 16 requests of 200 to 22000 keys 104 us instead of 233.
//
// While one half's softmax runs, the other half's products do: per half the
// order is S(j), softmax(j), O += P(j) V(j), S(j + 1).  Tensor memory is full:
// two S of 128 columns (three with 64 channels), over which P is written, and
// two O of d.
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
//   otherwise.  fp16 ends at 65504: top = 11.5, m is 5 above the maximum and
//   moves when a tile's sum passes 60000 and one of it 65504; a probability keeps
//   11 bits down to 2^-20 of the largest.  Rows that see n keys in all, fewer than
//   a tile, have m 3 above and 128 / n times lower; rows that see n in their first
//   tile and more later, sqrt(128 / n) times higher, and 11 bits down to 2^-17 where
//   n is 1.
// * A move costs a tile 4000 cycles, and one row of 32 is enough.  So in fp16 the
//   last two tiles change places: the first has 128 keys for most rows, whose
//   largest tells more than that of a few (and see kAhead: of 8192 tokens' scores
//   with a few large channels 1.2% of a warp's tiles moved, 0.4% with the tiles in
//   this order, 0.05% with 5 above instead of 3).
//
// Bound: the tensor cores (4 d flops per row and key).  8192 tokens of 32 query
// and 8 cache heads of 128 channels: bf16 320 us, 1.72 PFLOP/s, 89% of a library's
// largest product in a burst, for the first 45 ms of such calls; then 341 us, 1.61
// PFLOP/s, 93% of what that product holds for seconds, as the GPU draws all the power
// that it may and the clock falls (2070 to 1867 MHz), whether inputs repeat or not.
// fp16 344 and 367 us, where the same products draw more power (a library's large
// one runs at 1.71 PFLOP/s against 1.82).  The softmax shows
// with 64 channels, whose tiles are half the products for the same softmax (232 us
// of 142), and with capped scores, whose polynomial is as long as the rest of it
// (516 us; two prompts of 3001 to 4097 tokens: tensor cores 39% active).  A bias
// takes three operations a score, one by one (bf16 383 us beside 341), and with a cap
// as well each tile is gone through twice, with tanh itself (1064 us).  Runs of
// few tiles: a run's first tile takes 1500 to 2300 cycles more.
#pragma once

#include <algorithm>
#include <climits>
#include <cuda.h>
#include <type_traits>

#include "attend_paged_common.cuh"
#include "mbarrier.cuh"
#include "tcgen05.cuh"
#include "warp_mma.cuh"

namespace hc {
namespace {

constexpr int kKeys = 128;       // keys of a tile
constexpr int kHalf = 128;       // rows of a half
constexpr int kRowsTile = 2 * kHalf;
constexpr int kSoftmaxWarps = 8, kLoadWarp = 8, kProductWarp = 9, kWorkWarp = 10, kEdgeWarp = 11, kQueryWarp = 12;
constexpr int kThreadsTiles = 16 * 32;
// Registers of a thread: 128 at launch, shared out anew between the softmax's
// 256 threads and the others (256 * 208 + 256 * 48 = 512 * 128).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 48;
constexpr int kWorksAhead = 2;   // the one in hand and the next
// The next work is taken when this many tiles of the one in hand are not loaded yet: late, as who is done first takes
// the next, but not so late that it is waited for.
constexpr int kDue = 4;
constexpr int kBlockBytes = kKeys * 128;  // 128 rows of 64 channels, swizzled in 128-byte rows

enum Scores { kPlain, kCapped, kBiased };  // kBiased: with or without a cap

// p = 2^(x - m + kTop); see above.
template <bool kBf16>
struct Softmax;
template <>
struct Softmax<true> {
  static constexpr float kTop = 0.f, kMoveAt = 30.f, kAhead = 0.f, kAheadOfAll = 0.f, kMostSum = 0x1p40f;
};
template <>
struct Softmax<false> {
  static constexpr float kTop = 11.5f, kMoveAt = 3.5f, kAhead = 5.f, kAheadOfAll = 3.f, kMostSum = 60000.f;
};

// Tensor memory is full: see above.  A half's next scores wait for its probabilities' product
// where there are two buffers; with 64 channels there is room for a third, and
// they do not.
template <int D>
struct Tiles {
  static constexpr int kBuffers = D == 64 ? 3 : 2, kStages = D == 64 ? 4 : 2;
  static constexpr int kOut = kBuffers * 128;  // column of the first O
  static constexpr int kTileBytes = D / 64 * kBlockBytes;
  static constexpr int kQ = 0, kK = 2 * kTileBytes, kV = kK + kStages * kTileBytes;
  static constexpr int kBytes = kV + kStages * kTileBytes;
  // with 1 KiB to align, and enough for one CTA per SM: each takes all of tensor memory
  static constexpr int kAsk = (kBytes > 120 * 1024 ? kBytes : 120 * 1024) + 1024;
};

// Work of a CTA: 256 rows of one request and cache head.
struct alignas(16) Work {
  PagedRequest rq;
  int r, head, row0, rows_all, tiles;  // tiles 0: no work, the CTA is done
  int parts, part, first_part;  // of the run's tiles, and the places of this one's and the first one's sums (parts 1: the result)
  Range vis;        // its tiles: of this part
};
// Tile j of a work, from the last one on (kFullFirst: the last two change places): its first key.
template <bool kFullFirst>
__device__ __forceinline__ int tile_key(const Range& v, int j) {
  const int at = kFullFirst && j < 2 && v.tiles > 1 ? 1 - j : j;
  return (v.tile0 + v.tiles - 1 - at) * kKeys;
}
// Whether some key of the tile is seen by no row of the work.
__device__ __forceinline__ bool at_edge(const Range& v, int key0) { return key0 < v.lo || key0 + kKeys > v.hi; }

// Scores n = 2 * (tile, counted over all works) + half are in buffer n % kBuffers.
template <int D>
struct TileShared {
  uint64_t k_full[Tiles<D>::kStages], k_empty[Tiles<D>::kStages], v_full[Tiles<D>::kStages], v_empty[Tiles<D>::kStages],
      v_edge[Tiles<D>::kStages], s_full[Tiles<D>::kBuffers], p_full[Tiles<D>::kBuffers], q_full[2], q_empty[2], o_full[2][2], o_empty[2], l_full[2][2],
      work_full[kWorksAhead], work_empty[kWorksAhead], work_due, drain;
  uint32_t tmem;
  int32_t dead;               // some wait ran out
  float2 rows[2][kRowsTile];  // of work k at k & 1: a row's reference and sum
  Work work[kWorksAhead];     // work k at k % kWorksAhead
};

__device__ __forceinline__ __half2 half2_of(uint32_t u) {
  __half2 h;
  memcpy(&h, &u, 4);
  return h;
}
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
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, uint64_t* b, int x, int y, int z,
                                          uint32_t leader) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.ne.u32 q, %6, 0;\n"
      "@q cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];\n}" ::"r"(dst),
      "l"(map), "r"(mbar_addr(b)), "r"(x), "r"(y), "r"(z), "r"(leader)
      : "memory");
}
// Two fp32 in a register pair, kept as one value: left to itself the compiler makes a constant's pair anew for each use.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(float a, float b) {
  Pair d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ Pair fixed_pair(float a) {
  Pair d;
  asm volatile("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(a));
  return d;
}
__device__ __forceinline__ float2 floats_of(Pair p) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float largest(const uint32_t (&y)[32]) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = fmaxf(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]));
#pragma unroll
  for (int i = 8; i < 32; i += 2) m[i / 2 % 4] = max3(m[i / 2 % 4], __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
__device__ __forceinline__ void store32(void* to, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// The order of works: runs of 256 rows whose last rows see the most keys, by
// powers of two; within one such class, by request and from its last rows; and a
// run's parts, from its last tiles.  Each class goes through the requests again,
// so many requests, which even out by themselves, are one class, and so are runs
// that are shared out.
constexpr int kFewestKeys = 256, kMostRequests = 256;
struct Cursor {
  int r0 = 0, before = 0;  // first request of 32, works of those before it
  int upto, from;          // this class' runs see from `from` up to below `upto` keys
  int target = INT_MAX;    // tiles of a part, or a few more
  // the lane's request, of the 32: read once as long as they stay, counted once a class
  bool read = false, counted = false;
  PagedRequest q;
  int rows, runs, parts, to_end, inc;  // parts: of each of its runs
  __device__ __forceinline__ void take_class(const AttendPagedParams& p) {
    from = p.n_req > kMostRequests || upto <= kFewestKeys ? 0 : upto == INT_MAX ? 1 << 30 : upto >> 1;
  }
  __device__ __forceinline__ explicit Cursor(const AttendPagedParams& p) {
    const int64_t keys = static_cast<int64_t>(p.table_width) << p.B_log2;
    upto = p.n_req > kMostRequests || keys >= 1 << 30 ? INT_MAX : 1 << (32 - __clz(static_cast<int>(keys)));
    take_class(p);
  }
  // Short parts need no order, and classes take time (37 requests of 60 to 8400 keys: 36 us in seven, 31 in one); long
  // ones do (64 of 200 to 24000: 277 us and 298).
  __device__ __forceinline__ void share_out(int tiles) {
    target = tiles;
    if (tiles < 16) upto = INT_MAX, from = 0;
  }
};
__device__ __forceinline__ PagedRequest tiled_request(const AttendPagedParams& p, int r, int& rows) {
  int bad = 0;  // lengths are reported by k_attend_paged_rows
  PagedRequest q{0, 0, 0, 0};
  if (r < p.n_req) q = load_request(p, r, bad);
  rows = q.n * p.G > p.rows_above ? q.n * p.G : 0;
  return q;
}
__device__ __forceinline__ int parts_of(int tiles, int target) { return max(1, tiles / target); }
// How long the parts shall be, found by a warp: of one part a run and the rule's
// choices the one of the least time, with a request's runs all as long as its last.
__device__ __forceinline__ int part_tiles(const AttendPagedParams& p, int lane) {
  int best = INT_MAX, runs_here = 0, tiles = 0;  // of the lane's request
  float total = 0.f, time = 0.f;
#pragma unroll 1
  for (int c = -2; c < SplitRule::kChoices; ++c) {  // the first time round for the total
    const int target = c < 0 ? INT_MAX : p.split.target(total, c);
    float works = 0.f, sum = 0.f;
    int longest = 0;
#pragma unroll 1
    for (int r = lane; r - lane < p.n_req; r += 32) {
      if (c == -2 || p.n_req > 32) {  // else it is still there
        int rows;
        const PagedRequest q = tiled_request(p, r, rows);
        runs_here = (rows + kRowsTile - 1) / kRowsTile;
        tiles = rows > 0 ? visible<kKeys>(p, q, (runs_here - 1) * kRowsTile, rows).tiles : 0;
      }
      const int parts = parts_of(tiles, target);
      const float runs = static_cast<float>(runs_here * p.H);
      works = fmaf(runs, static_cast<float>(parts), works);
      sum = fmaf(runs, static_cast<float>(tiles), sum);
      longest = max(longest, (tiles + parts - 1) / parts);
    }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) {
      works += __shfl_xor_sync(0xffffffffu, works, o);
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    total = sum;
    const float t = p.split.time(works, static_cast<float>(__reduce_max_sync(0xffffffffu, longest)), total) +
                    (c < 0 ? 0.f : SplitRule::kJoin);
    if (c < 0 || t < time) {
      time = t;
      best = target;
    }
  }
  return best;
}
// Runs of 256 rows of a request, of `runs` in all, whose last row's keys end at
// `key` or later; positions do not fall, so they are the last ones.  Where they
// do, which is flagged, it is some number that does not rise with `key` either:
// each run is some class's, once.
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
// Work number `idx` of the call, found by a warp (all lanes get it); false past
// the last.  `c` goes forward only, so idx may not fall.  A run's parts have equal
// numbers of tiles but kLeastPartTiles at least; tiles 0 where it has no such part.
template <bool kParts>
__device__ __forceinline__ bool find_work(const AttendPagedParams& p, Cursor& c, int idx, int lane, Work& w) {
  for (;;) {
    if (!c.read) {
      c.q = tiled_request(p, c.r0 + lane, c.rows);
      c.runs = (c.rows + kRowsTile - 1) / kRowsTile;
      if (kParts)
        c.parts = c.rows == 0 ? 1 : parts_of(visible<kKeys>(p, c.q, (c.runs - 1) * kRowsTile, c.rows).tiles, c.target);
      c.read = true;
    }
    if (!c.counted) {
      c.to_end = runs_seeing(p, c.q, c.runs, c.from);
      c.inc = (c.to_end - runs_seeing(p, c.q, c.runs, c.upto)) * p.H * (kParts ? c.parts : 1);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, c.inc, o);
        if (lane >= o) c.inc += v;
      }
      c.counted = true;
    }
    const uint32_t upto = __ballot_sync(0xffffffffu, idx < c.before + c.inc);
    if (upto != 0) {
      const int src = __ffs(static_cast<int>(upto)) - 1;
      w.r = c.r0 + src;
      w.rq = {__shfl_sync(0xffffffffu, c.q.q0, src), __shfl_sync(0xffffffffu, c.q.n, src),
              __shfl_sync(0xffffffffu, c.q.kv, src), __shfl_sync(0xffffffffu, c.q.prefix, src)};
      w.rows_all = __shfl_sync(0xffffffffu, c.rows, src);
      const int most = kParts ? __shfl_sync(0xffffffffu, c.parts, src) : 1;
      const int after = __shfl_sync(0xffffffffu, c.before + c.inc, src) - 1 - idx, left = after / most;  // the last rows first
      const int i = most - 1 - (after - left * most);
      w.part = idx;
      w.first_part = idx - i;
      const int run = static_cast<int>(p.by_heads.div(left));
      w.head = left - run * p.H;
      w.row0 = (__shfl_sync(0xffffffffu, c.runs - c.to_end, src) + run) * kRowsTile;
      w.vis = visible<kKeys>(p, w.rq, w.row0, min(w.row0 + kRowsTile, w.rows_all));
      w.tiles = w.vis.tiles;
      w.parts = 1;
      if (kParts && most > 1) {
        const int each = max((w.vis.tiles + most - 1) / most, kLeastPartTiles), from = i * each;
        w.parts = (w.vis.tiles + each - 1) / each;
        w.tiles = max(0, min(each, w.vis.tiles - from));
        w.vis.tile0 += w.vis.tiles - from - w.tiles;
        w.vis.tiles = w.tiles;
      }
      return true;
    }
    c.before += __shfl_sync(0xffffffffu, c.inc, 31);
    c.counted = false;
    c.r0 += 32;
    c.read = p.n_req <= 32;
    if (c.r0 >= p.n_req) {
      if (c.from == 0) return false;
      c.upto = c.from;
      c.take_class(p);
      c.r0 = 0;
    }
  }
}
// A run whose parts are to be joined.
struct alignas(32) Join {
  int q0, rows_all, head, row0, parts, part;
};
__device__ __forceinline__ Join* joins(const AttendPagedParams& p) { return reinterpret_cast<Join*>(p.part_sums + p.part_bytes); }
// A part's sums in the workspace: O by fours of channels [D / 4][rows], then (reference, sum) [rows].
template <int D>
__device__ __forceinline__ float4* part_sums(const AttendPagedParams& p, int part) {
  return reinterpret_cast<float4*>(p.part_sums + static_cast<int64_t>(part) * p.part_rows * (D * 4 + 8));
}

// kParts: runs may be shared out (the same kernel for calls that do not: 324 us instead of 319 for 8192 tokens).
template <bool kBf16, int D, Scores kScores, bool kParts>
__global__ void __launch_bounds__(kThreadsTiles, 1)
    k_attend_paged_tiles(const __grid_constant__ AttendPagedParams p, const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap q_map) {
  using L = Tiles<D>;
  using Soft = Softmax<kBf16>;
  constexpr int kStages = L::kStages, kBuffers = L::kBuffers;
  constexpr bool kFullFirst = !kBf16 && kScores != kBiased;
  extern __shared__ unsigned char dyn_raw[];
  __shared__ TileShared<D> sh;
  unsigned char* const dyn = dyn_raw + (1024 - (smem_addr(dyn_raw) & 1023)) % 1024;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  int bad = 0;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_empty[i], 1);
      mbar_init(&sh.v_edge[i], 1);
    }
    for (int i = 0; i < kBuffers; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], kHalf);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], p.q_tma ? 1 : 64);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.o_empty[i], 4);
      mbar_init(&sh.l_full[i][0], kHalf);
      mbar_init(&sh.l_full[i][1], kHalf);
      mbar_init(&sh.o_full[i][0], 1);
      mbar_init(&sh.o_full[i][1], 1);
    }
    for (int i = 0; i < kWorksAhead; ++i) {
      mbar_init(&sh.work_full[i], 1);
      mbar_init(&sh.work_empty[i], kThreadsTiles / 32 - 1);
    }
    mbar_init(&sh.work_due, 1);
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
    const bool there = mbar_wait_inline(&sh.work_full[k % kWorksAhead], (k / kWorksAhead) & 1, &sh.dead, p.wait_limit);
    ok = __all_sync(0xffffffffu, ok && there);
    return ok && sh.work[k % kWorksAhead].tiles > 0;
  };
  auto leave_work = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.work_empty[k % kWorksAhead]);
  };

  if (warp < kSoftmaxWarps) {
    // ================================================== softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes of tensor memory per warp
    const uint32_t o_at = tmem + lanes + L::kOut + half * D;
    auto pack2 = [](float lo, float hi) { return kBf16 ? pack_bf16(lo, hi) : pack_f16(lo, hi); };
    for (int k = 0; take_work(k); ++k) {
      const Work& work = sh.work[k % kWorksAhead];
      const int tiles = work.tiles, row = work.row0 + tid;
      const bool live = row < work.rows_all;
      // keys that the thread's row sees; rows past the last see what the work sees
      const int token = static_cast<int>(p.by_group.div(live ? row : 0)), head = work.head * p.G + row - token * p.G;
      int first = work.vis.lo, last = work.vis.hi, pos = 0;
      float slope = 0.f;
      if (live) {
        pos = position(p, work.rq, token);
        first = first_key(p, pos);
        last = last_key(p, work.rq, pos);
        if (kScores == kBiased) slope = p.slopes ? __ldg(p.slopes + head) * kLog2e : 0.f;
      }

      // what a hidden score is overwritten with: -inf once it is multiplied (a factor of 0 would make it NaN, and the
      // smallest that is not, the largest score 2^-21)
      const float factor = p.scale_log2 == 0.f ? 0x1p-149f : p.scale_log2;
      uint32_t hidden = __float_as_uint(kScores == kPlain && factor < 0.f ? -kNegInf : kNegInf);
      // cap * tanh(s * cap_in) up to |s * cap_in| = 3/4 as an odd polynomial in s: the minimax fit of tanh(y) / y in y^2
      // by Remez' exchange, off by 2.9e-8, with the factors in its terms; its last term is negative, so that a score
      // of y = 1000 is one that no probability comes of.  Caps and factors whose products fp32 does not hold do without.
      Pair tanh_terms[6];
      float tanh_reach = -1.f;
      if constexpr (kScores == kCapped) {
        constexpr float kTerms[6] = {0.999999971015f, -0.333329588875f, 0.13325406137f,
                                     -0.0533444364837f, 0.0195829218425f, -0.0047162673917f};
        const float t = p.cap_in * p.cap_in;
        // scale * cap_in^10, of which the last term is made, passes fp32's end within the bounds below (1e39, the least is
        // 1e-35), so 2^-8 of it is counted
        float power = p.scale_log2 * 0x1p-8f;
#pragma unroll
        for (int k = 0; k < 6; ++k) {
          tanh_terms[k] = fixed_pair(kTerms[k] * 0x1p8f * power);
          power *= t;
        }
        if (t >= 1e-6f && t <= 1e6f && p.cap_log2 >= 0.01f && p.cap_log2 <= 1e6f) tanh_reach = 0.5625f / t;
        hidden = __float_as_uint(1000.f / p.cap_in);
      }

      float m = kNegInf, l = 0.f;
      const Range vis = work.vis;
      for (int j = 0; j < tiles && ok; ++j) {
        const int key0 = tile_key<kFullFirst>(vis, j);
        const int n = 2 * (base + j) + half, buffer = n % kBuffers;
        const uint32_t s_at = tmem + lanes + buffer * 128;
        const int lo = first - key0, hi = last - key0;  // columns [lo, hi) count
        // Most tiles: all of it seen, by rows that have a reference.
        const bool partly = live && (lo > 0 || hi < kKeys), fresh = live && m == kNegInf && max(lo, 0) < min(hi, kKeys);
        const bool special = __any_sync(0xffffffffu, partly || fresh);
        ok = mbar_wait_inline(&sh.s_full[buffer], (n / kBuffers) & 1, &sh.dead, p.wait_limit);
        if (!__all_sync(0xffffffffu, ok)) break;
        fence_after();
        // A score in units of log2.
        auto score = [&](float x, int c) {
          if (kScores == kCapped || (kScores == kBiased && p.cap_log2 != 0.f))
            x = tanh_of(x * p.cap_in) * p.cap_log2;
          else
            x *= factor;
          if (kScores == kBiased) x = fmaf(-slope, fabsf(static_cast<float>(pos - key0) - static_cast<float>(c)), x);
          return x;
        };
        // Which of 32 columns count, a bit each.
        auto seen_of = [&](int c) {
          const int count = min(max(hi - c, 0), 32), skip = min(max(lo - c, 0), 32);
          return (count == 32 ? ~0u : (1u << count) - 1u) & (skip == 32 ? 0u : ~0u << skip);
        };
        // The row's reference, given its largest score here, and O with it.
        auto refer = [&](float top, bool crowded) {
          float ahead = Soft::kAhead;
          if (!kBf16) {
            const auto steps = [](int n) { return static_cast<float>(__clz(max(n - 1, 0)) - __clz(kKeys - 1)); };  // log2(128 / n)
            const int all = last - first, here = min(hi, kKeys) - max(lo, 0);
            if (all < kKeys)  // few keys in all: as low as n of them do not pass kMostSum
              ahead = Soft::kAheadOfAll - steps(all);
            else if (here < kKeys)  // few keys here: half as much higher, as larger ones may follow
              ahead += 0.5f * steps(here);
          }
          const float m_new =
              top > m + (crowded ? -Soft::kAhead : Soft::kMoveAt) || (m == kNegInf && top > m) ? top + ahead : m;
          if (__any_sync(0xffffffffu, m_new != m && m != kNegInf)) {  // O of a row without one is 0
            const float by = m == kNegInf ? 0.f : ex2(m - m_new);
            l *= by;
            ok = mbar_wait_inline(&sh.o_full[half][(base + j - 1) & 1], ((base + j - 1) >> 1) & 1, &sh.dead, p.wait_limit) && ok;
            fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_load32(o, o_at + c);
              tmem_wait_load(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
              tmem_store32(o_at + c, o);
            }
          }
          m = m_new;
        };
        // The first keys of a row, or keys that some row does not see: what is hidden is overwritten where it is, and the
        // largest score found (a cap does not change which it is), in a loop that is short in code, as it is seldom in
        // the instruction cache.  With a bias, scores are written as they count.
        float top = kNegInf, most = 0.f;  // most: of the scores' magnitudes
        const bool first_keys = __any_sync(0xffffffffu, fresh);
        bool counted = kScores == kBiased && (special || p.cap_log2 != 0.f);
        if (special || counted) {
#pragma unroll 1
          for (int c = 0; c < kKeys; c += 32) {
            const uint32_t seen = seen_of(c);
            const bool all = __all_sync(0xffffffffu, seen == ~0u || !live);
            if (kScores == kPlain && all && !first_keys) continue;
            uint32_t y[32];
            if (!__any_sync(0xffffffffu, seen != 0)) {
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = hidden;
              tmem_store32(s_at + c, y);
              continue;
            }
            tmem_load32(y, s_at + c);
            tmem_wait_load(y);
            if (kScores == kBiased) {
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(score(__uint_as_float(y[i]), c + i));
            }
            if (kScores == kCapped) {
              uint32_t z[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) z[i] = seen & 1u << i ? y[i] & 0x7fffffffu : 0u;
              most = fmaxf(most, largest(z));
            }
            const uint32_t lowest = __float_as_uint(factor < 0.f ? -kNegInf : kNegInf);
            if (kScores == kCapped && !all) {  // looked through as -inf, written as `hidden`
              uint32_t z[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                z[i] = seen & 1u << i ? y[i] : hidden;
                y[i] = seen & 1u << i ? y[i] : lowest;
              }
              tmem_store32(s_at + c, z);
            } else if (!all) {
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = seen & 1u << i ? y[i] : hidden;
            }
            if (kScores == kBiased || (kScores == kPlain && !all)) tmem_store32(s_at + c, y);
            if (kScores != kBiased && factor < 0.f) {
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] ^= 0x80000000u;
            }
            top = fmaxf(top, largest(y));
          }
          wait_store();
          if (first_keys) {
            if (kScores == kPlain) top *= fabsf(factor);
            if (kScores == kCapped && top != kNegInf) top = score(factor < 0.f ? -top : top, 0);
            refer(top, false);
          }
        }
        // Scores beyond the polynomial's reach: written as they count.
        auto count = [&] {
#pragma unroll 1
          for (int c = 0; c < kKeys; c += 32) {
            const uint32_t seen = seen_of(c);
            uint32_t y[32];
            tmem_load32(y, s_at + c);
            tmem_wait_load(y);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              y[i] = __float_as_uint(seen & 1u << i ? score(__uint_as_float(y[i]), c + i) : kNegInf);
            tmem_store32(s_at + c, y);
          }
          wait_store();
          counted = true;
        };
        if (kScores == kCapped && special && !__all_sync(0xffffffffu, most * most <= tanh_reach || !live)) count();
        // P stays in registers until its sum is known, since it goes over S.
        float sum, reach;
        uint32_t h[2][32];
        auto probabilities = [&](auto as_counted) {
          constexpr bool kCounted = decltype(as_counted)::value;
          const float off = m == kNegInf ? 0.f : Soft::kTop - m;
          [[maybe_unused]] const Pair off2 = kScores == kCapped && !kCounted ? fixed_pair(off) : 0;
          float2 part = make_float2(0.f, 0.f);
          float far[4] = {0.f, 0.f, 0.f, 0.f};  // four, so that one need not wait for the other
          uint32_t x[2][16];
          tmem_load16(x[0], s_at);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t(&y)[16] = x[c & 1];
            tmem_wait_load16(y);
            if (c < 7) tmem_load16(x[(c & 1) ^ 1], s_at + (c + 1) * 16);
            float2 v[8];
            if constexpr (!kCounted && kScores == kCapped) {
              Pair s2[8], u2[8], t2[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                s2[i] = pair_of(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]));
                u2[i] = mul2(s2[i], s2[i]);
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 u = floats_of(u2[i]);
                far[i & 3] = max3(far[i & 3], u.x, u.y);
                t2[i] = fma2(tanh_terms[5], u2[i], tanh_terms[4]);
              }
#pragma unroll
              for (int k = 3; k >= 0; --k)
#pragma unroll
                for (int i = 0; i < 8; ++i) t2[i] = fma2(t2[i], u2[i], tanh_terms[k]);
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = floats_of(fma2(s2[i], t2[i], off2));
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                v[i] = make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]));
                if constexpr (kCounted) {
                  v[i] = __fadd2_rn(v[i], make_float2(off, off));
                } else {
                  v[i] = __ffma2_rn(v[i], make_float2(factor, factor), make_float2(off, off));
                  if (kScores == kBiased) {
                    const float away = static_cast<float>(pos - key0);
                    v[i].x = fmaf(-slope, fabsf(away - static_cast<float>(c * 16 + 2 * i)), v[i].x);
                    v[i].y = fmaf(-slope, fabsf(away - static_cast<float>(c * 16 + 2 * i + 1)), v[i].y);
                  }
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              v[i].x = ex2(v[i].x);
              v[i].y = ex2(v[i].y);
              part = __fadd2_rn(part, v[i]);
              h[c / 4][(c % 4) * 8 + i] = pack2(v[i].x, v[i].y);
            }
          }
          sum = part.x + part.y;
          reach = fmaxf(fmaxf(far[0], far[1]), fmaxf(far[2], far[3]));
        };
        for (bool moved = first_keys;;) {
          if (kScores != kPlain && counted)
            probabilities(std::true_type());
          else
            probabilities(std::false_type());
          if (kScores == kCapped && !special && !counted && !__all_sync(0xffffffffu, reach <= tanh_reach || !live)) {
            count();
            continue;
          }
          if (moved) break;
          bool fits = __all_sync(0xffffffffu, sum < Soft::kMostSum || !live);
          if (!kBf16 && !fits) {  // many keys, or one that fp16 does not hold
            __half2 high = half2_of(h[0][0]);
#pragma unroll
            for (int i = 1; i < 64; ++i) high = __hmax2_nan(high, half2_of(h[i / 32][i % 32]));
            fits = __all_sync(0xffffffffu,
                              __hlt(__hmax_nan(__low2half(high), __high2half(high)), __ushort_as_half(0x7c00)) || !live);
          }
          if (fits) break;
          // scores far above the reference: it moves
          top = kNegInf;
#pragma unroll 1
          for (int c = 0; c < kKeys; c += 32) {
            uint32_t y[32];
            tmem_load32(y, s_at + c);
            tmem_wait_load(y);
            if (kScores == kCapped && !counted) {
              const uint32_t seen = seen_of(c), sign = factor < 0.f ? 0x80000000u : 0u;
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = seen & 1u << i ? y[i] ^ sign : __float_as_uint(kNegInf);
            } else if (kScores == kPlain || !counted) {
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(score(__uint_as_float(y[i]), c + i));
            }
            top = fmaxf(top, largest(y));
          }
          if (kScores == kCapped && !counted && top != kNegInf) top = score(factor < 0.f ? -top : top, 0);
          refer(top, true);
          moved = true;
        }
        tmem_store32(s_at, h[0]);
        tmem_store32(s_at + 32, h[1]);
        l += sum;
        wait_store();
        fence_before();
        mbar_arrive(&sh.p_full[buffer]);
      }
      base += tiles;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      sh.rows[k & 1][tid] = make_float2(m, l);
      mbar_arrive(&sh.l_full[half][k & 1]);
      leave_work(k);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
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
            const int key = tile_key<kFullFirst>(vis, j) + lane * block;
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
          const int st = (base + j) % kStages, round = (base + j) / kStages;
          const int next = slot_of(j + 1);
          if (lane == 0 && j == max(tiles - kDue, 0)) mbar_arrive(&sh.work_due);
          if (round > 0) ok = mbar_wait_inline(&sh.k_empty[st], (round - 1) & 1, &sh.dead, p.wait_limit);
          if (!__all_sync(0xffffffffu, ok)) break;
          if (lane == 0) mbar_expect(&sh.k_full[st], L::kTileBytes);
          __syncwarp();
          ++k_sent;
          load(tiles_at + L::kK + st * L::kTileBytes, &k_map, &sh.k_full[st], slot);
          if (round > 0) ok = mbar_wait_inline(&sh.v_empty[st], (round - 1) & 1, &sh.dead, p.wait_limit);
          if (!__all_sync(0xffffffffu, ok)) break;
          const bool edge = at_edge(vis, tile_key<kFullFirst>(vis, j));
          uint64_t* const full = edge ? &sh.v_edge[st] : &sh.v_full[st];
          if (lane == 0) mbar_expect(full, L::kTileBytes);
          __syncwarp();
          ++v_sent;
          by_edge = (by_edge & ~(1u << st)) | static_cast<uint32_t>(edge) << st;
          if (edge) edges ^= 1u << st;
          load(tiles_at + L::kV + st * L::kTileBytes, &v_map, full, slot);
          slot = next;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        base += tiles;
        leave_work(k);
      }
      if (!ok) {  // a wait ran out: copies may still be on their way into shared memory
        int32_t no = 0;
        for (int n = max(k_sent - kStages, 0); n < k_sent; ++n) mbar_wait_inline(&sh.k_full[n % kStages], (n / kStages) & 1, &no);
        for (int n = max(v_sent - kStages, 0); n < v_sent; ++n) {
          const int st = n % kStages;
          if (by_edge >> st & 1u)
            mbar_wait_inline(&sh.v_edge[st], ~(edges >> st) & 1u, &no);
          else
            mbar_wait_inline(&sh.v_full[st], (n / kStages) & 1, &no);
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
          const int key0 = tile_key<kFullFirst>(vis, j), st = (base + j) % kStages;
          if (!at_edge(vis, key0)) continue;
          ok = mbar_wait_inline(&sh.v_edge[st], edges >> st & 1u, &sh.dead, p.wait_limit);
          if (!__all_sync(0xffffffffu, ok)) break;
          edges ^= 1u << st;
          unsigned char* const tile = dyn + L::kV + st * L::kTileBytes;
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
      // The first is the CTA's number; the others are taken from a counter, each when the one before is nearly loaded.
      Cursor cursor(p);
      if (kParts) cursor.share_out(part_tiles(p, lane));
      Work work;
      int number = blockIdx.x;
      bool taken = false;
      for (int k = 0;; ++k) {
        if (k >= kWorksAhead)
          ok = mbar_wait_inline(&sh.work_empty[k % kWorksAhead], (k / kWorksAhead - 1) & 1, &sh.dead, p.wait_limit);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (k > 0) {
          ok = mbar_wait_inline(&sh.work_due, (k - 1) & 1, &sh.dead, p.wait_limit);
          if (!__all_sync(0xffffffffu, ok)) break;
        }
        bool more = true;
        do {
          if (taken) {
            if (lane == 0) number = static_cast<int>(gridDim.x) + atomicAdd(p.tiles_taken, 1);
            number = __shfl_sync(0xffffffffu, number, 0);
          }
          taken = true;
          more = find_work<kParts>(p, cursor, number, lane, work);
        } while (more && work.tiles == 0);
        if (!more) work.tiles = 0;
        if (lane == 0) {
          sh.work[k % kWorksAhead] = work;
          mbar_arrive(&sh.work_full[k % kWorksAhead]);
          if (kParts && more && work.parts > 1 && work.part == work.first_part)
            joins(p)[atomicAdd(p.tiles_taken + 2, 1)] = {work.rq.q0, work.rows_all, work.head, work.row0, work.parts, work.part};
        }
        if (!more) break;
      }
      // the last CTA to come here leaves the counters as it found them
      if (lane == 0) {
        __threadfence();
        if (atomicAdd(p.tiles_taken + 1, 1) == static_cast<int>(gridDim.x) - 1) {
          p.tiles_taken[0] = 0;
          p.tiles_taken[1] = 0;
        }
      }
      __syncwarp();
    } else if (warp == kProductWarp) {
      // ================================================== products
      // Buffers and stages go round by counting, a half is known where the code is written, and the numbers of tiles
      // come by a shuffle: so all of it stays in uniform registers, and a product's issue takes 11 cycles instead of 33.
      const uint32_t leader = elect_leader();
      const uint32_t at = __shfl_sync(0xffffffffu, tmem, 0), tiles_at = __shfl_sync(0xffffffffu, smem_addr(dyn), 0);
      uint32_t s_tile = 0, p_tile = 0;                          // tiles of keys and of values so far
      uint32_t s_buffer = 0, p_buffer = 0, p_parity = 0;        // of the next scores, of the next probabilities
      // Whether a wait ran out is asked once per tile: products on what is not there yet spoil results only.
      auto wait = [&](uint64_t* b, uint32_t parity) { ok = mbar_wait_inline(b, parity, &sh.dead, p.wait_limit) && ok; };
      auto scores = [&](int i) {  // S_i = Q_i K(j)^T
        const uint32_t st = s_tile % kStages;
        if (i == 0) wait(&sh.k_full[st], (s_tile / kStages) & 1);
        fence_after();
        const uint64_t q = smem_desc(tiles_at + L::kQ + i * L::kTileBytes, 16);
        const uint64_t keys = smem_desc(tiles_at + L::kK + st * L::kTileBytes, 16);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint64_t step = ((s / 4) * kBlockBytes + (s % 4) * 32) >> 4;
          mma_smem(at + s_buffer * 128, q + step, keys + step, instr_desc(kKeys, false, kBf16), s > 0, leader);
        }
        commit(&sh.s_full[s_buffer], leader);
        s_buffer = s_buffer == kBuffers - 1 ? 0 : s_buffer + 1;
        if (i == 1) {
          commit(&sh.k_empty[st], leader);
          ++s_tile;
        }
      };
      // O_i (+)= P_i(j) V(j), for the oldest scores without it.  Scores are up to kBuffers ahead, into the next work.
      int p_left = 0, p_next = 0;             // products left of the work that they are in, and of the next
      uint32_t p_done = 0, p_work = 0, p_fresh = 2;  // products so far; that work's number; its products with a new O
      auto values = [&] {
        const uint32_t i = p_done & 1, st = p_tile % kStages;
        if (i == 0) wait(&sh.v_full[st], (p_tile / kStages) & 1);
        wait(&sh.p_full[p_buffer], p_parity);
        if (p_fresh > 0 && p_work > 0) wait(&sh.o_empty[i], (p_work - 1) & 1);  // the last work's O is read
        fence_after();
        const uint64_t v = smem_desc(tiles_at + L::kV + st * L::kTileBytes, kBlockBytes);
#pragma unroll
        for (int s = 0; s < kKeys / 16; ++s)
          mma_tmem(at + L::kOut + i * D, at + p_buffer * 128 + s * 8, v + s * (2048 >> 4), instr_desc(D, true, kBf16),
                   p_fresh == 0 || s > 0, leader);
        commit(&sh.o_full[i][p_tile & 1], leader);
        if (i == 1) {
          commit(&sh.v_empty[st], leader);
          ++p_tile;
        }
        p_parity ^= p_buffer == kBuffers - 1 ? 1 : 0;
        p_buffer = p_buffer == kBuffers - 1 ? 0 : p_buffer + 1;
        ++p_done;
        if (p_fresh > 0) --p_fresh;
        if (--p_left == 0) {
          p_left = p_next;
          p_next = 0;
          p_fresh = 2;
          ++p_work;
        }
      };
      uint32_t ahead = 0;  // scores whose products are not issued yet
      for (uint32_t k = 0;; ++k) {
        if (!take_work(static_cast<int>(k))) break;
        const int count = 2 * __shfl_sync(0xffffffffu, sh.work[k % kWorksAhead].tiles, 0);  // tiles and halves
        leave_work(static_cast<int>(k));
        if (p_left == 0)
          p_left = count;
        else
          p_next = count;
#pragma unroll 1
        for (int n = 0; n < count; n += 2) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (ahead == kBuffers) {
              values();
              --ahead;
            }
            if (n == 0) wait(&sh.q_full[i], k & 1);
            scores(i);
            ++ahead;
            if (n == count - 2) commit(&sh.q_empty[i], leader);
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        if (!ok) break;
        // the next work is not there before the last one's result is: its products first
        for (; p_work < k; --ahead) values();
      }
      if (ok)
        for (; ahead > 0; --ahead) values();
      ok = __all_sync(0xffffffffu, ok);
      __syncwarp();
    } else {
      // ================================================== queries and results
      // The next work's queries as soon as the last scores of this one are there, two warps a half; then this one's
      // result, 32 rows of each half a warp.
      constexpr int kLanes = D / 8, kRowsAt = 32 / kLanes;  // 16-byte pieces of a row; rows at a time
      const int quarter = warp - kQueryWarp, piece = lane % kLanes;
      auto pack2 = [](float lo, float hi) { return kBf16 ? pack_bf16(lo, hi) : pack_f16(lo, hi); };
      const int q_half = quarter >> 1;
      const uint32_t q_smem = __shfl_sync(0xffffffffu, smem_addr(dyn), 0) + L::kQ + q_half * L::kTileBytes;
      int q_sent = 0;
      auto load_queries = [&](int k) {
        const Work& work = sh.work[k % kWorksAhead];
        const int row0 = work.row0, rows_all = work.rows_all, q0 = work.rq.q0, head = work.head * p.G;
        const int token0 = q0 + static_cast<int>(p.by_group.div(row0 + q_half * kHalf));
        if (k > 0) ok = mbar_wait_inline(&sh.q_empty[q_half], (k - 1) & 1, &sh.dead, p.wait_limit);
        if (!__all_sync(0xffffffffu, ok)) return;
        if (p.q_tma) {  // a half is whole tokens: a box of them by their heads.  Rows of other requests do no harm.
          if (quarter & 1) return;
          if (lane == 0) mbar_expect(&sh.q_full[q_half], L::kTileBytes);
          __syncwarp();
          const uint32_t leader = elect_leader();
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load3(q_smem + c * kBlockBytes, &q_map, &sh.q_full[q_half], c * 64, head, token0, leader);
          q_sent = k + 1;
          return;
        }
        const int row_first = quarter * 64 + lane / kLanes;  // of the 256
#pragma unroll 4
        for (int r = 0; r < 64; r += kRowsAt) {
          const int at = row_first + r, row = row0 + at;
          const bool live = row < rows_all;
          const int i = static_cast<int>(p.by_group.div(live ? row : 0));
          const uint16_t* const from = static_cast<const uint16_t*>(p.q) + static_cast<int64_t>(q0 + i) * p.q_token +
                                       static_cast<int64_t>(head + (live ? row : 0) - i * p.G) * p.q_head + piece * 8;
          cp_async16(q_smem + (piece / 8) * kBlockBytes + (at % kHalf) * 128 + (((piece % 8) ^ (at & 7)) << 4),
                     live ? from : static_cast<const uint16_t*>(p.q), live ? 16 : 0);
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_async();
        mbar_arrive(&sh.q_full[q_half]);
      };
      bool more = take_work(0);
      if (more) load_queries(0);
      for (int k = 0; more && ok; ++k) {
        const Work& work = sh.work[k % kWorksAhead];
        base += work.tiles;
        more = take_work(k + 1);
        if (more) load_queries(k + 1);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int at = half * kHalf + quarter * 32 + lane, row = work.row0 + at;
          const bool live = row < work.rows_all;
          const int token = static_cast<int>(p.by_group.div(live ? row : 0));
          const int64_t t = work.rq.q0 + token, head = work.head * p.G + row - token * p.G;
          uint16_t* const out = static_cast<uint16_t*>(p.out) + t * p.o_token + head * p.o_head;
          ok = mbar_wait_inline(&sh.l_full[half][k & 1], (k >> 1) & 1, &sh.dead, p.wait_limit) && ok;
          ok = mbar_wait_inline(&sh.o_full[half][(base - 1) & 1], ((base - 1) >> 1) & 1, &sh.dead, p.wait_limit) && ok;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          fence_after();
          const float2 ml = sh.rows[k & 1][at];
          const float by = ml.y > 0.f ? 1.f / ml.y : 0.f;
          const bool whole = work.parts == 1, stored = at < p.part_rows;
          float4* const sums = whole ? nullptr : part_sums<D>(p, work.part);
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t x[16], w[8];
            tmem_load16(x, tmem + (static_cast<uint32_t>(quarter) << 21) + L::kOut + half * D + c);
            tmem_wait_load16(x);
            if (!whole) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (stored)
                  __stcg(sums + (c / 4 + i) * p.part_rows + at,
                         make_float4(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1]), __uint_as_float(x[4 * i + 2]),
                                     __uint_as_float(x[4 * i + 3])));
              continue;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = pack2(__uint_as_float(x[2 * i]) * by, __uint_as_float(x[2 * i + 1]) * by);
            if (live && p.out32) {
              store32(out + c, w);
            } else if (live) {
              reinterpret_cast<uint4*>(out + c)[0] = make_uint4(w[0], w[1], w[2], w[3]);
              reinterpret_cast<uint4*>(out + c)[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
          if (!whole && stored) __stcg(reinterpret_cast<float2*>(sums + D / 4 * p.part_rows) + at, ml);
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.o_empty[half]);
          if (whole && p.lse && live)
            p.lse[t * (static_cast<int64_t>(p.H) * p.G) + head] =
                ml.y > 0.f ? (ml.x - Softmax<kBf16>::kTop + log2f(ml.y)) * kLn2 : kNegInf;
        }
        if (ok) leave_work(k);
      }
      if (!ok && q_sent > 0) {  // a wait ran out: the copy may still be on its way
        int32_t no = 0;
        mbar_wait_inline(&sh.q_full[q_half], (q_sent - 1) & 1, &no);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  if (warp == kProductWarp) {
    if (sh.dead) {  // products may still be on their way: wait for them before their memory goes
      if (lane == 0) flag_error(p.err, HC_DEVERR_WAIT);
      int32_t no = 0;
      commit(&sh.drain, elect_leader());
      mbar_wait_inline(&sh.drain, 0, &no);
      __syncwarp();
    }
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
  if (bad) flag_error(p.err, bad);
}

// The parts' sums of a run joined, in their order: 32 rows of a run a CTA, a
// lane for each, several parts' sums on their way together.
constexpr int kJoinThreads = 256;
template <bool kBf16, int D>
__global__ void __launch_bounds__(kJoinThreads, 2) k_join_paged_tiles(const __grid_constant__ AttendPagedParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunks = p.part_rows / 32, run = blockIdx.x / chunks, at = (blockIdx.x - run * chunks) * 32 + lane;
  const bool there = run < __ldcg(p.tiles_taken + 2);
  __syncthreads();
  // the last CTA to come here leaves the counters as they were found
  if (threadIdx.x == 0 && atomicAdd(p.tiles_taken + 3, 1) == static_cast<int>(gridDim.x) - 1) {
    p.tiles_taken[2] = 0;
    p.tiles_taken[3] = 0;
  }
  if (!there) return;
  const Join w = joins(p)[run];
  const int row = w.row0 + at;
  if (row >= w.rows_all) return;
  const int token = static_cast<int>(p.by_group.div(row));
  const int64_t t = w.q0 + token, head = w.head * p.G + row - token * p.G;
  uint16_t* const out = static_cast<uint16_t*>(p.out) + t * p.o_token + head * p.o_head;
  constexpr int kFours = D / 4 / (kJoinThreads / 32);  // of channels, of a thread
  constexpr int kAtOnce = 16 / kFours;
  float top = kNegInf, sum = 0.f;
  float4 acc[kFours];
#pragma unroll
  for (int i = 0; i < kFours; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int k = 0; k < w.parts; k += kAtOnce) {
    float2 ml[kAtOnce];
    float4 v[kAtOnce][kFours];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const float4* const sums = part_sums<D>(p, w.part + min(k + u, w.parts - 1));
      ml[u] = __ldcg(reinterpret_cast<const float2*>(sums + D / 4 * p.part_rows) + at);
#pragma unroll
      for (int i = 0; i < kFours; ++i) v[u][i] = __ldcg(sums + (warp * kFours + i) * p.part_rows + at);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (k + u >= w.parts || ml[u].x == kNegInf) continue;
      const float to = fmaxf(top, ml[u].x), old = ex2(top - to), wt = ex2(ml[u].x - to);  // top -inf: old 0
      top = to;
      sum = sum * old + wt * ml[u].y;
#pragma unroll
      for (int i = 0; i < kFours; ++i) {
        acc[i].x = acc[i].x * old + wt * v[u][i].x, acc[i].y = acc[i].y * old + wt * v[u][i].y;
        acc[i].z = acc[i].z * old + wt * v[u][i].z, acc[i].w = acc[i].w * old + wt * v[u][i].w;
      }
    }
  }
  const float by = sum > 0.f ? 1.f / sum : 0.f;
  auto pack2 = [](float lo, float hi) { return kBf16 ? pack_bf16(lo, hi) : pack_f16(lo, hi); };
#pragma unroll
  for (int i = 0; i < kFours; ++i)
    reinterpret_cast<uint2*>(out)[warp * kFours + i] =
        make_uint2(pack2(acc[i].x * by, acc[i].y * by), pack2(acc[i].z * by, acc[i].w * by));
  if (p.lse && warp == 0)
    p.lse[t * (static_cast<int64_t>(p.H) * p.G) + head] =
        sum > 0.f ? (top - Softmax<kBf16>::kTop + log2f(sum)) * kLn2 : kNegInf;
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

// Queries as [token][head][channel], copied 64 channels of a cache head's query heads for as many tokens as make 128
// rows.  False where that is no box: heads that do not divide 128, or strides that a copy does not take.
template <bool kBf16>
bool queries_map(CUtensorMap* map, const AttendPagedParams& p, int d) {
  const EncodeTiled encode = encode_tiled();
  if (!encode || kHalf % p.G) return false;
  const int64_t heads = static_cast<int64_t>(p.H) * p.G;
  const cuuint64_t sizes[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(p.n_tokens)};
  // of one head or token the stride is not used, and may be anything
  const int64_t head = heads > 1 ? 2 * p.q_head : 2 * d, token = p.n_tokens > 1 ? 2 * p.q_token : 2 * d;
  if (head <= 0 || token <= 0 || head >= int64_t{1} << 40 || token >= int64_t{1} << 40) return false;
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head), static_cast<cuuint64_t>(token)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(kHalf / p.G)}, step[3] = {1, 1, 1};
  return encode(map, kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p.q),
                sizes, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kBf16, int D, Scores kScores, bool kParts>
cudaError_t launch(AttendPagedParams p, const CUtensorMap& k_map, const CUtensorMap& v_map, const CUtensorMap& q_map, int64_t runs,
                   cudaStream_t s) {
  static KernelOnDevice kernel;
  int resident = 0;
  const cudaError_t e = kernel.resident(reinterpret_cast<const void*>(k_attend_paged_tiles<kBf16, D, kScores, kParts>),
                                        kThreadsTiles, Tiles<D>::kAsk, &resident);
  if (e != cudaSuccess) return e;
  // a CTA per work, as far as the host can tell
  const int grid = static_cast<int>(kParts ? resident : std::min<int64_t>(runs, resident));
  k_attend_paged_tiles<kBf16, D, kScores, kParts><<<grid, kThreadsTiles, Tiles<D>::kAsk, s>>>(p, k_map, v_map, q_map);
  return cudaGetLastError();
}

template <bool kBf16, int D, bool kParts>
cudaError_t launch_scores(const AttendPagedParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map, const CUtensorMap& q_map,
                          int64_t runs, cudaStream_t s) {
  if (p.slopes) return launch<kBf16, D, kBiased, kParts>(p, k_map, v_map, q_map, runs, s);
  return p.cap_log2 != 0.f ? launch<kBf16, D, kCapped, kParts>(p, k_map, v_map, q_map, runs, s)
                           : launch<kBf16, D, kPlain, kParts>(p, k_map, v_map, q_map, runs, s);
}

template <bool kBf16, int D>
cudaError_t launch_parts(AttendPagedParams p, cudaStream_t s) {
  CUtensorMap k_map, v_map, q_map = {};
  cudaError_t e = pages_map<kBf16>(&k_map, p.k_pages, p, D);
  if (e == cudaSuccess) e = pages_map<kBf16>(&v_map, p.v_pages, p, D);
  if (e != cudaSuccess) return e;
  p.q_tma = queries_map<kBf16>(&q_map, p, D);
  const int64_t rows = static_cast<int64_t>(p.max_new) * p.G, runs = (rows + kRowsTile - 1) / kRowsTile * p.n_req * p.H;
  p.part_rows = static_cast<int32_t>(std::min<int64_t>((rows + 31) / 32 * 32, kRowsTile));
  const int64_t keys = static_cast<int64_t>(p.table_width) << p.B_log2, places = p.part_bytes / (p.part_rows * (D * 4 + 8));
  // the longest wait is for a whole run, whose tiles take 1 to 2 us each
  p.wait_limit = kWaitLimit + static_cast<uint64_t>(keys / kKeys) * 20000;
  if (!split_rule(p.n_req, runs, keys, p.part_rows, places, device_sm_count(), &p.split))
    return launch_scores<kBf16, D, false>(p, k_map, v_map, q_map, runs, s);
  e = launch_scores<kBf16, D, true>(p, k_map, v_map, q_map, runs, s);
  if (e != cudaSuccess) return e;
  k_join_paged_tiles<kBf16, D><<<static_cast<unsigned>(runs * (p.part_rows / 32)), kJoinThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_tiles(const AttendPagedParams& p, cudaStream_t s) {
  return p.bf16 ? launch_parts<true, D>(p, s) : launch_parts<false, D>(p, s);
}

}  // namespace
}  // namespace hc
