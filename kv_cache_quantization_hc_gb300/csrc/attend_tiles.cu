// Attention of the new tokens over the 4-bit cache, many query rows: tiles of
// 256 rows (new tokens times the query heads of one cache head) against tiles
// of 128 keys on the 5th-generation tensor cores.
//
// One CTA per SM takes runs of 256 rows one after another, the longest first
// (k-th run: number k * CTAs + i, or the mirror of it for odd k, which evens
// the sums out).  Its 14 warps each go through the runs by themselves, so that
// one's codes are converted while the last one's result is still written:
//   warps 0-3, 4-7  the softmax of rows 0-127 and 128-255, a thread per row;
//   warps 8-11      codes and scales into fp16 tiles of keys and values in
//                   shared memory, two of each ahead;
//   warp 12         one thread issues the products: S = Q K^T into tensor
//                   memory, O += P V with P from tensor memory;
//   warp 13         finds the runs, up to four ahead.
// While one half's softmax runs, the other half's products do: per half the
// order is S(j), softmax(j), O += P(j) V(j), S(j + 1).  Tensor memory is full:
// two S of 128 columns, over which P is written, and two O of d.
//
// Mathematics, per row, with a reference m near the running maximum:
//   x_j = f * 2^(ek + 10) * (q . k_j),  p_j = 2^(x_j - m + 11.5),  l = sum p_j,
//   O = sum (p_j * 2^(ev_j - ev)) v_j,  out = O / l * 2^(ev + 10)
// * k_j = code * scale * 2^(-10 - ek) and v_j = code * scale * 2^(-10 - ev_j) in
//   fp16, 2^ek and 2^ev_j the largest scales of the run of 32 keys that j is
//   in, 2^ev the largest so far.  Powers of two, so that scales of any size
//   fit, and each element is rounded once.  A run is one warp's to convert, so
//   its exponents are too: no barrier among those warps.
// * Queries in fp16: each row times a power of two that brings its largest
//   value near 2^14 (f holds the inverse).
// * m moves only when the maximum exceeds it by 3.5, and then to 3 above the
//   maximum, so that O (in tensor memory) is rarely rescaled.  Between, a tile
//   whose probabilities sum up to 60000 (fp16 ends at 65504) moves it too.
//   The largest probability is then 2^8.5: a tile of 128 equal scores sums up to
//   three quarters of what moves m, and a probability keeps fp16's 11 bits down
//   to 2^-22 of the largest and some of them down to 2^-33, which channels need
//   where the larger keys' values are zero.  That takes rows of few keys, mostly,
//   so where a row sees n keys of its first tile m starts 128 / n times lower.
// * The channels of keys, queries and values are permuted within eights
//   (0 4 1 5 2 6 3 7), the order in which a word of codes comes apart; the
//   products over channels do not see it and the output is put back in order.
//
// Bound: the tensor cores (4 d flops per row and key), with the softmax's
// exponentials and the conversion of the codes beside them.  A prompt of 8192
// tokens, 32 query heads of 128 channels: 400 us, 1.37 PFLOP/s, with the same
// inputs again (415 us where they change from call to call); the period of a
// tile is about 2800 cycles, 1040 of them products.  Two halves of 128 rows take
// turns because a row's softmax has to stand between its two products; four
// converting warps, as three are too slow for that (482 us against 387) and
// seven take registers from the softmax (419).
#include <algorithm>
#include <climits>
#include <type_traits>

#include "attend_common.cuh"
#include "mbarrier.cuh"

namespace hc {
namespace {

constexpr int kKeys = 128;       // keys of a tile
constexpr int kHalf = 128;       // rows of a half
constexpr int kRowsTile = 2 * kHalf;
constexpr int kSoftmaxWarps = 8, kConvertWarps = 4;
constexpr int kProductWarp = kSoftmaxWarps + kConvertWarps, kWorkWarp = kProductWarp + 1;
constexpr int kThreadsTiles = (kWorkWarp + 1) * 32;
constexpr int kWorksAhead = 4;   // found before they are begun
constexpr int kBlockBytes = kKeys * 128;  // 128 rows of 64 channels, swizzled in 128-byte rows
constexpr int kNoValues = 1000;  // "exponent" of a run whose values are all zeros: larger than any
constexpr int kExp = -10;        // elements times 2^(kExp - exponent of the run's largest scale)
constexpr float kTop = 11.5f;    // log2 of the probability of a score that equals the reference
constexpr float kMoveAt = 3.5f;  // the reference moves when the maximum is this far above it,
constexpr float kAhead = 3.f;    // to this far above the maximum, or
constexpr float kMostSum = 60000.f;  // when a tile's probabilities sum up to this: fp16 ends at 65504

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
  Request rq;
  int r, head, row0, rows_all, tiles;  // tiles 0: no work, the CTA is done
  Range vis;
};

struct TileShared {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], q_full[2], e_full[4], work_full[kWorksAhead],
      work_empty[kWorksAhead], drain;
  uint32_t tmem;
  int32_t dead;               // some wait ran out
  int4 ek[4], ev[4];          // of tile j at j & 3: the exponents of its 4 runs of 32 keys
  int32_t q_exp[kRowsTile];   // of a row's largest query
  Work work[kWorksAhead];     // work k at k % kWorksAhead
};

// ------------------------------------------------------------ PTX
// The products are issued by one thread (`leader`), but the whole warp goes
// along: what it computes on the way is then the same in all lanes, and stays
// in uniform registers.
__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t leader;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(leader));
  return leader;
}
__device__ __forceinline__ void commit(uint64_t* b, uint32_t leader) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.ne.u32 q, %1, 0;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_addr(b)),
      "r"(leader) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void mma_smem(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add,
                                         uint32_t leader) {
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %4, 0;\nsetp.ne.u32 q, %5, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add),
      "r"(leader) : "memory");
}
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add,
                                         uint32_t leader) {
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %4, 0;\nsetp.ne.u32 q, %5, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(add),
      "r"(leader) : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
            "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
// The loads so far are done; the registers may be used from here on.
__device__ __forceinline__ void tmem_wait_load(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                     "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                       "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :: "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_load16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :: "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11"
      ", %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29"
      ", %30, %31, %32};"
               :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
                   "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
                     "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
                       "r"(r[30]), "r"(r[31])
               : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11"
      ", %12, %13, %14, %15, %16};"
               :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
                   "r"(r[15])
               : "memory");
}

// Shared-memory descriptor of a tile in 128-byte swizzled rows: groups of 8
// rows 1024 bytes apart; for channel-major use (values), blocks of 64
// channels `block_stride` bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t block_stride) {
  return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | (static_cast<uint64_t>(block_stride >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// M = 128, fp16 operands, fp32 sums; `n_major`: B's rows are the reduction
__device__ __forceinline__ constexpr uint32_t instr_desc(int n, bool n_major) {
  return (1u << 4) | (n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// Signed codes of nibbles 0 and 4 (resp. 1 and 5) of w as fp16: 1024 + u in
// the mantissa, u = code + 8, less 1032; or 1024 + 16 u, over 16, less 72.
__device__ __forceinline__ __half2 as_half2(uint32_t u) {
  __half2 h;
  memcpy(&h, &u, 4);
  return h;
}
__device__ __forceinline__ uint32_t as_bits(__half2 h) {
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ __half2 both(uint16_t h) { return __half2half2(__ushort_as_half(h)); }
__device__ __forceinline__ __half2 codes_04(uint32_t w) {
  return __hsub2(as_half2(and_xor(w, 0x000f000fu, 0x64086408u)), both(0x6408));
}
__device__ __forceinline__ __half2 codes_15(uint32_t w) {
  return __hfma2(as_half2(and_xor(w, 0x00f000f0u, 0x64806480u)), both(0x2c00), both(0xd480));
}

// The scale of 32 channels: fp16, with what fp16 leaves of an fp32 scale
// apart, so that the product is rounded once.
template <bool kScaleF16>
struct ScaleH {
  __half2 s, rest;
  __device__ __forceinline__ explicit ScaleH(float v) {
    s = __float2half2_rn(v);
    if (!kScaleF16) rest = __float2half2_rn(v - __low2float(s));
  }
  __device__ __forceinline__ uint32_t times(__half2 codes) const {
    return as_bits(kScaleF16 ? __hmul2(codes, s) : __hfma2(codes, s, __hmul2(codes, rest)));
  }
};

// Number `idx` of the call's works, found by a warp (all lanes get it); false
// past the last.  `c` goes forward only, so idx may not fall.
//
// The order: works whose last rows see the most keys, by powers of two; within
// one, by request and from its last rows.  In the order of the requests alone,
// seven prompts of 129 to 2355 tokens took 131 us instead of 123.  Each class
// goes through the requests again, so many requests, which even out by
// themselves, are one class.
constexpr int kFewestKeys = 256, kMostRequests = 256;
struct Cursor {
  int r0 = 0, before = 0;  // first request of 32, works of those before it
  int upto;                // the works of this class see fewer keys
  __device__ __forceinline__ explicit Cursor(const AttendParams& p) {
    const int64_t keys = static_cast<int64_t>(p.table_width) << p.B_log2;
    upto = p.n_req > kMostRequests || keys >= 1 << 30 ? INT_MAX : 1 << (32 - __clz(static_cast<int>(keys)));
  }
};
// Runs of 256 rows of a request, of `runs` in all, whose last row sees `key` keys or more.
__device__ __forceinline__ int runs_seeing(const AttendParams& p, const Request& q, int runs, int key) {
  if (key <= 0) return runs;
  if (q.kv < key) return 0;
  const int i = key - 1 - q.kv + q.n;  // the first new token to see it: before the last
  return !p.causal || i <= 0 ? runs : runs - i * p.G / kRowsTile;
}
__device__ __forceinline__ bool find_work(const AttendParams& p, Cursor& c, int idx, int lane, Work& w) {
  for (;;) {
    const int from = p.n_req > kMostRequests || c.upto <= kFewestKeys ? 0 : c.upto == INT_MAX ? 1 << 30 : c.upto >> 1;
    for (; c.r0 < p.n_req; c.r0 += 32) {
      Request q{0, 0, 0};
      int bad = 0;  // lengths are reported by k_attend_rows
      if (c.r0 + lane < p.n_req) q = load_request(p, c.r0 + lane, bad);
      const int rows = q.n * p.G > p.rows_above ? q.n * p.G : 0;
      const int runs = (rows + kRowsTile - 1) / kRowsTile;
      const int to_end = runs_seeing(p, q, runs, from);
      const int works = (to_end - runs_seeing(p, q, runs, c.upto)) * p.H;
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
              __shfl_sync(0xffffffffu, q.kv, src)};
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

template <int D, int GROUP, bool kScaleF16>
__global__ void __launch_bounds__(kThreadsTiles, 1) k_attend_tiles(const __grid_constant__ AttendParams p) {
  using Smem = TileSmem<D>;
  extern __shared__ unsigned char dyn_raw[];
  __shared__ TileShared sh;
  unsigned char* const dyn = dyn_raw + (1024 - (smem_addr(dyn_raw) & 1023)) % 1024;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  int bad = 0;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.k_full[i], kConvertWarps * 32);
      mbar_init(&sh.v_full[i], kConvertWarps * 32);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], kHalf);
      mbar_init(&sh.q_full[i], kHalf);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sh.e_full[i], kConvertWarps);
    for (int i = 0; i < kWorksAhead; ++i) {
      mbar_init(&sh.work_full[i], 1);
      mbar_init(&sh.work_empty[i], kWorkWarp);
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
        for (int u = 0; u < 8; ++u) {
          const float2 a = widen(raw[u].x, p.bf16), b = widen(raw[u].y, p.bf16), c = widen(raw[u].z, p.bf16),
                       d = widen(raw[u].w, p.bf16);
          float amax = fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))),
                             fmaxf(fmaxf(fabsf(c.x), fabsf(c.y)), fmaxf(fabsf(d.x), fabsf(d.y))));
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);  // at most 127: finite
          const float up = p.scale_log2 < 0.f ? -pow2(14 - e) : pow2(14 - e);
          uint4 w;  // channels 0 4 1 5 2 6 3 7
          w.x = pack_f16(a.x * up, c.x * up);
          w.y = pack_f16(a.y * up, c.y * up);
          w.z = pack_f16(b.x * up, d.x * up);
          w.w = pack_f16(b.y * up, d.y * up);
          const int at = r0 + u * kRowsAt + lane / kLanes;
          *piece_at(at, piece) = w;
          if (piece == 0) sh.q_exp[warp * 32 + at] = e;
        }
      }
      fence_async();
      mbar_arrive(&sh.q_full[half]);
      int first = 0, last = 0x7fffffff;  // keys that the thread's row sees
      if (row < work.rows_all) {
        const int pos = work.rq.kv - work.rq.n + static_cast<int>(p.by_group.div(row));
        last = p.causal ? min(work.rq.kv, pos + 1) : work.rq.kv;
        if (p.window) first = pos - p.window + 1;
      }
      __syncwarp();
      const float factor = fabsf(p.scale_log2) * pow2(sh.q_exp[tid] - 14);

      float m = kNegInf, l = 0.f;
      int ev = -100;
      for (int j = 0; j < tiles && ok; ++j) {
        const int jj = base + j;
        ok = mbar_wait(&sh.e_full[jj & 3], (jj >> 2) & 1, &sh.dead) && mbar_wait(&sh.s_full[half], (jj + k) & 1, &sh.dead);
        if (!__all_sync(0xffffffffu, ok)) break;
        fence_after();
        const int4 ek4 = sh.ek[jj & 3], ev4 = sh.ev[jj & 3];
        const int ek[4] = {ek4.x, ek4.y, ek4.z, ek4.w};
        int evs[4] = {ev4.x, ev4.y, ev4.z, ev4.w};
        // one above the largest when it moves, so that it moves rarely
        const int ev_tile = max(max(evs[0], evs[1]), max(evs[2], evs[3]));
        int ev_new = ev_tile > ev ? ev_tile + 1 : ev;
        // The scores' factor, of each run of 32 keys: never 0 (queries and keys of zeros, softmax_scale 0), as hidden
        // scores are -inf and go through the same product; 2^-126 times a sum of 2^34 at most is as good as 0.
        float f[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) f[c] = fmaxf(factor * pow2(ek[c] - kExp), 0x1p-126f);
        const int key0 = (work.vis.tile0 + j) * kKeys;
        // A row may see all of this tile and nothing before it (its window starts here): no reference yet, so not
        // for the one pass either.  In the vote that is taken anyway it costs nothing (chunks 133.4 us with and without).
        const bool masked = __any_sync(0xffffffffu, key0 < first || key0 + kKeys > last || (j > 0 && m == kNegInf));
        // Most tiles: all of it seen, by rows that have a reference, and no score far above that.  One pass then, with P kept
        // in registers until the maximum is known, since it goes over the scores.
        float sum = 0.f;
        bool done = false, crowded = false;  // crowded: the sum was too large
        if (!masked && j > 0 && ev_new == ev) {
          uint32_t x[2][16], h[2][32];
          float all = 0.f;
          tmem_load16(x[0], s_at);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int d = max(evs[c] - ev, -126);
            const float off = m == kNegInf ? 0.f : kTop - m + static_cast<float>(d);
            const float2 f2 = make_float2(f[c], f[c]), off2 = make_float2(off, off);
            float2 part = make_float2(0.f, 0.f);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t(&y)[16] = x[u];
              tmem_wait_load16(y);
              if (c < 3 || u < 1) tmem_load16(x[u ^ 1], s_at + c * 32 + (u + 1) * 16);
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                float2 v = __ffma2_rn(make_float2(__uint_as_float(y[k]), __uint_as_float(y[k + 1])), f2, off2);
                v.x = ex2(v.x);
                v.y = ex2(v.y);
                part = __fadd2_rn(part, v);
                h[c / 2][(c % 2) * 16 + u * 8 + k / 2] = pack_f16(v.x, v.y);
              }
            }
            all += part.x + part.y;
            sum = fmaf(part.x + part.y, pow2(-d), sum);
          }
          done = __all_sync(0xffffffffu, all < kMostSum);
          crowded = !done;
          if (done) {
            tmem_store32(s_at, h[0]);
            tmem_store32(s_at + 32, h[1]);
          }
        }
        if (!done) {
          const int lo = first - key0, hi = last - key0;  // columns [lo, hi) count
          // Probabilities are shifted by their run's exponent before they are summed, which would flush the part of a
          // run of zero values beside large ones.  The product does not see such a run: it goes without a shift, and
          // its tile comes here (1.2 us of 417 for a prompt of 8192 tokens; asked in the one pass too: 428).
          if (ev_tile == kNoValues) {
            ev_new = ev;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (evs[c] != kNoValues) ev_new = evs[c] > ev_new ? evs[c] + 1 : ev_new;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (evs[c] == kNoValues) evs[c] = ev_new;
          }
          sum = 0.f;
          uint32_t a[32];
          float top = kNegInf;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_load32(a, s_at + c * 32);
            tmem_wait_load(a);
            float most = kNegInf;
            if (masked) {  // hidden columns become -inf where they are
              const int n = min(max(hi - c * 32, 0), 32), skip = min(max(lo - c * 32, 0), 32);
              const uint32_t seen = (n == 32 ? ~0u : (1u << n) - 1u) & (skip == 32 ? 0u : ~0u << skip);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(seen >> k & 1u)) a[k] = __float_as_uint(kNegInf);
              tmem_store32(s_at + c * 32, a);
            }
#pragma unroll
            for (int k = 0; k < 32; k += 2) most = fmaxf(most, fmaxf(__uint_as_float(a[k]), __uint_as_float(a[k + 1])));
            top = fmaxf(top, most * f[c]);
          }
          if (masked) wait_store();
          // the reference of the row, and O with it
          float ahead = kAhead;
          if (masked) {  // n keys seen: 128 / n times lower, as n of them do not pass kMostSum either
            const int n = min(hi, kKeys) - max(lo, 0);
            if (n < kKeys) ahead -= static_cast<float>(__clz(max(n - 1, 0)) - __clz(kKeys - 1));
          }
          const float m_new =
              top > m + (crowded ? -kAhead : kMoveAt) || (m == kNegInf && top > m) ? top + ahead : m;
          if (__any_sync(0xffffffffu, m_new != m || ev_new != ev)) {
            const float by = m == kNegInf ? 0.f : ex2(m - m_new);
            l *= by;
            if (j > 0) {
              const float by_o = by * pow2(max(ev - ev_new, -126));
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                tmem_load32(a, o_at + c * 32);
                tmem_wait_load(a);
#pragma unroll
                for (int k = 0; k < 32; ++k) a[k] = __float_as_uint(__uint_as_float(a[k]) * by_o);
                tmem_store32(o_at + c * 32, a);
              }
            }
            m = m_new;
            ev = ev_new;
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int d = max(evs[c] - ev, -126);
            const float off = m == kNegInf ? 0.f : kTop - m + static_cast<float>(d);
            const float2 f2 = make_float2(f[c], f[c]), off2 = make_float2(off, off);
            float2 part = make_float2(0.f, 0.f);
            uint32_t h[16];
            tmem_load32(a, s_at + c * 32);
            tmem_wait_load(a);
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float2 v = __ffma2_rn(make_float2(__uint_as_float(a[k]), __uint_as_float(a[k + 1])), f2, off2);
              v.x = ex2(v.x);
              v.y = ex2(v.y);
              part = __fadd2_rn(part, v);
              h[k / 2] = pack_f16(v.x, v.y);
            }
            tmem_store16(s_at + c * 16, h);  // over columns already read
            sum = fmaf(part.x + part.y, pow2(-d), sum);
          }
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
      const float by = l > 0.f ? pow2(ev - kExp) / l : 0.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        tmem_load32(x, o_at + c * 32);
        tmem_wait_load(x);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float v[8];  // channels 0 4 1 5 2 6 3 7 back in order
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(x[u * 8 + 2 * i]) * by;
            v[i + 4] = __uint_as_float(x[u * 8 + 2 * i + 1]) * by;
          }
          uint4 w;
          w.x = p.bf16 ? pack_bf16(v[0], v[1]) : pack_f16(v[0], v[1]);
          w.y = p.bf16 ? pack_bf16(v[2], v[3]) : pack_f16(v[2], v[3]);
          w.z = p.bf16 ? pack_bf16(v[4], v[5]) : pack_f16(v[4], v[5]);
          w.w = p.bf16 ? pack_bf16(v[6], v[7]) : pack_f16(v[6], v[7]);
          *piece_at(lane, c * 4 + u) = w;
        }
      }
      fence_before();
      if (p.lse && row < work.rows_all)
        p.lse[row_offset(row, static_cast<int64_t>(p.H) * p.G, 1)] =
            l > 0.f ? (m - kTop + log2f(l)) * 0.6931471805599453f : kNegInf;
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
  } else if (warp < kSoftmaxWarps + kConvertWarps) {
    // ================================================== codes to fp16 tiles
    constexpr int kParts = D / 32;   // threads of a key, 32 channels each: one group's scale
    constexpr int kIters = kParts;   // a warp has 32 keys of the tile, 32 / kParts at a time
    constexpr int kGroups = D / GROUP;
    const int t = tid - kSoftmaxWarps * 32, w = warp - kSoftmaxWarps;
    const int part = t % kParts;
    auto place = [&](int it) { return w * 32 + it * (32 / kParts) + lane / kParts; };  // a key's, in the tile
    for (int k = 0; take_work(k); ++k) {
      const Work& work = sh.work[k % kWorksAhead];
      const Range vis = work.vis;
      const int r = work.r, head = work.head, tiles = work.tiles;
      const int swap = (part >> 1) & 1;  // block 1 writes its words in the order 2 3 0 1: other banks than block 0's

      // Loads are issued far ahead of their use and without branches: a key that no row sees, or one in a slot
      // that does not exist, is read from a place that does (the nearest seen key's table entry; slot 0) and
      // gets scale 0.  A thread's keys keep their places within their blocks from tile to tile, as a block's
      // size divides a tile's, so an address is the slot times a stride away from one of kIters starts.
      const int32_t* const table = vis.hi > 0 ? p.tables + static_cast<int64_t>(r) * p.table_stride : p.q_starts;
      constexpr int kScaleSize = kScaleF16 ? 2 : 4;
      const uint32_t slab = static_cast<uint32_t>(p.H) << p.B_log2;  // rows of K, or of V, in a slot
      const uint32_t slot_codes = 2 * slab * (D / 2), slot_scales = 2 * slab * kGroups * kScaleSize;
      const uint8_t* code_start[kIters];
      const uint8_t* scale_start[kIters];
#pragma unroll
      for (int it = 0; it < kIters; ++it) {
        const int64_t row = (static_cast<int64_t>(head) << p.B_log2) + (place(it) & ((1 << p.B_log2) - 1));
        code_start[it] = p.codes + row * (D / 2) + part * 16;
        scale_start[it] = static_cast<const uint8_t*>(p.scales) + (row * kGroups + part * 32 / GROUP) * kScaleSize;
      }
      uint4 code[2][kIters];
      // While tile j is converted, the codes and scales of j + 1 and the slots of j + 2 are on their way (L2 answers
      // in 1000 cycles and more under this load; a tile takes 2500).
      uint32_t scale[2][kIters], scale_next[2][kIters];  // of tiles j and j + 1, as stored
      int32_t slots_next[kIters], slots_after[kIters];   // of tiles j + 1 and j + 2
      uint32_t there = 0;                                // bit it: the tile of slots_next has that key
      auto key_of = [&](int j, int it) { return (vis.tile0 + j) * kKeys + place(it); };
      auto load_slots = [&](int j) {
#pragma unroll
        for (int it = 0; it < kIters; ++it)
          slots_after[it] = __ldg(table + (max(min(key_of(j, it), vis.hi - 1), vis.lo) >> p.B_log2));
      };
      auto next_slots = [&](int j) {  // slots_after, of tile j, become slots_next
        there = 0;
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
          const int key = key_of(j, it);
          const bool seen = j < tiles && key >= vis.lo && key < vis.hi;
          const bool in = static_cast<uint32_t>(slots_after[it]) < static_cast<uint32_t>(p.num_slots);
          if (seen && !in) bad |= HC_DEVERR_SLOT;
          if (seen && in) there |= 1u << it;
          slots_next[it] = in ? slots_after[it] : 0;
        }
      };
      auto load_codes = [&](int kv) {
#pragma unroll
        for (int it = 0; it < kIters; ++it)
          code[kv][it] = __ldg(reinterpret_cast<const uint4*>(
              code_start[it] + static_cast<uint64_t>(static_cast<uint32_t>(slots_next[it])) * slot_codes +
              (kv ? slab * (D / 2) : 0u)));
      };
      auto load_scales = [&]() {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
          for (int it = 0; it < kIters; ++it) {
            const uint8_t* at = scale_start[it] + static_cast<uint64_t>(static_cast<uint32_t>(slots_next[it])) * slot_scales +
                                (kv ? slab * (kGroups * kScaleSize) : 0u);
            scale_next[kv][it] = kScaleF16 ? __ldg(reinterpret_cast<const uint16_t*>(at))
                                           : __ldg(reinterpret_cast<const uint32_t*>(at));
          }
      };
      auto take_scales = [&]() {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
          for (int it = 0; it < kIters; ++it) scale[kv][it] = there >> it & 1u ? scale_next[kv][it] : 0u;
      };
      auto scale_value = [&](uint32_t bits) {
        return kScaleF16 ? __half2float(__ushort_as_half(static_cast<uint16_t>(bits))) : __uint_as_float(bits);
      };
      // The nibble u = code + 8 in the low bits of an fp16 is the subnormal u * 2^-24 (u * 2^-20 four bits up), so one
      // fused multiply-add by scale * 2^24 takes off 8 scales and rounds once.  For that the run's scales come to 2^-9
      // at most, and what is below 2^-25 then is lost: 2^-18 of the run's largest element.  An fp32 scale has a rest
      // to an fp16; its products take the codes as whole numbers, 1024 + u less 1032.
      auto convert = [&](unsigned char* tile, auto which, int e) {
        constexpr int kv = decltype(which)::value;
        const float up = pow2(kExp - e);
#pragma unroll
        for (int it = 0; it < kIters; ++it) {
          const int key = place(it);
          const float sc = scale_value(scale[kv][it]) * up;
          const ScaleH<kScaleF16> s(sc);
          const __half2 s24 = __float2half2_rn(sc * 0x1p24f), s20 = __float2half2_rn(sc * 0x1p20f),
                        off = __float2half2_rn(sc * -8.f);
          const uint4 c = code[kv][it];
          const uint32_t words[4] = {swap ? c.z : c.x, swap ? c.w : c.y, swap ? c.x : c.z, swap ? c.y : c.w};
          unsigned char* base = tile + (part >> 1) * kBlockBytes + key * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t lo = words[i], hi = lo >> 8;
            uint4 v;
            if (!kScaleF16) {
              v.x = s.times(codes_04(lo));
              v.y = s.times(codes_15(lo));
              v.z = s.times(codes_04(hi));
              v.w = s.times(codes_15(hi));
            } else {
              v.x = as_bits(__hfma2(as_half2(and_xor(lo, 0x000f000fu, 0x00080008u)), s24, off));
              v.y = as_bits(__hfma2(as_half2(and_xor(lo, 0x00f000f0u, 0x00800080u)), s20, off));
              v.z = as_bits(__hfma2(as_half2(and_xor(hi, 0x000f000fu, 0x00080008u)), s24, off));
              v.w = as_bits(__hfma2(as_half2(and_xor(hi, 0x00f000f0u, 0x00800080u)), s20, off));
            }
            const int chunk = (part & 1) * 4 + (i ^ (swap * 2));
            *reinterpret_cast<uint4*>(base + ((chunk ^ (key & 7)) << 4)) = v;
          }
        }
      };

      load_slots(0);
      next_slots(0);
      load_slots(1);
      load_scales();
      load_codes(0);
      load_codes(1);
      take_scales();
      next_slots(1);
      load_scales();
      load_slots(2);
      for (int j = 0; j < tiles; ++j) {
        const int jj = base + j;
        // the exponents of the run's largest scales
        int e[2];
        bool no_values = false;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          uint32_t top = 0;
#pragma unroll
          for (int it = 0; it < kIters; ++it) top = max(top, scale[kv][it] & (kScaleF16 ? 0x7fffu : 0x7fffffffu));
          top = __float_as_uint(scale_value(__reduce_max_sync(0xffffffffu, top)));
          no_values = top == 0;  // of the values, which come last
          e[kv] = min(max(static_cast<int>(top >> 23) - 127, -100), 110);
        }
        if (lane == 0) {
          reinterpret_cast<int*>(&sh.ek[jj & 3])[w] = e[0];
          reinterpret_cast<int*>(&sh.ev[jj & 3])[w] = no_values ? kNoValues : e[1];
          mbar_arrive(&sh.e_full[jj & 3]);
        }
        ok = __all_sync(0xffffffffu, ok);  // the warp goes on, or not
        if (!ok) break;

        const int st = jj & 1;
        if (jj >= 2) ok = ok && mbar_wait(&sh.k_empty[st], ((jj >> 1) - 1) & 1, &sh.dead);
        convert(dyn + Smem::kK + st * Smem::kTileBytes, std::integral_constant<int, 0>(), e[0]);
        fence_async();
        mbar_arrive(&sh.k_full[st]);
        load_codes(0);  // of j + 1
        if (jj >= 2) ok = ok && mbar_wait(&sh.v_empty[st], ((jj >> 1) - 1) & 1, &sh.dead);
        convert(dyn + Smem::kV + st * Smem::kTileBytes, std::integral_constant<int, 1>(), e[1]);
        fence_async();
        mbar_arrive(&sh.v_full[st]);
        load_codes(1);
        take_scales();
        next_slots(j + 2);
        load_scales();
        load_slots(j + 3);
      }
      // the last tile's waits may have run out for some lanes only: the warp leaves together, or not
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      base += tiles;
      leave_work(k);
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
        mma_smem(at + i * 128, q + step, k + step, instr_desc(kKeys, false), s > 0, leader);
      }
      commit(&sh.s_full[i], leader);
    };
    auto values = [&](int i, int j, bool add) {  // O_i (+)= P_i(j) V(j)
      const uint64_t v = smem_desc(tiles_at + Smem::kV + (j & 1) * Smem::kTileBytes, kBlockBytes);
#pragma unroll
      for (int s = 0; s < kKeys / 16; ++s)
        mma_tmem(at + 256 + i * D, at + i * 128 + s * 8, v + s * (2048 >> 4), instr_desc(D, true), add || s > 0, leader);
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

template <int D, int GROUP, bool kScaleF16>
cudaError_t launch(const AttendParams& p, cudaStream_t s) {
  static KernelOnDevice kernel;
  int resident = 0;
  const cudaError_t e = kernel.resident(reinterpret_cast<const void*>(k_attend_tiles<D, GROUP, kScaleF16>), kThreadsTiles,
                                        TileSmem<D>::kAsk, &resident);
  if (e != cudaSuccess) return e;
  const int64_t runs = (static_cast<int64_t>(p.max_new) * p.G + kRowsTile - 1) / kRowsTile;
  const double works = static_cast<double>(runs) * p.n_req * p.H;
  const int grid = works < resident ? static_cast<int>(works) : resident;
  k_attend_tiles<D, GROUP, kScaleF16><<<grid, kThreadsTiles, TileSmem<D>::kAsk, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_tiles(int d, int group, bool scale_f16, const AttendParams& p, cudaStream_t s) {
  if (d == 64) {
    if (group == 32) return scale_f16 ? launch<64, 32, true>(p, s) : launch<64, 32, false>(p, s);
    return scale_f16 ? launch<64, 64, true>(p, s) : launch<64, 64, false>(p, s);
  }
  if (group == 32) return scale_f16 ? launch<128, 32, true>(p, s) : launch<128, 32, false>(p, s);
  if (group == 64) return scale_f16 ? launch<128, 64, true>(p, s) : launch<128, 64, false>(p, s);
  return scale_f16 ? launch<128, 128, true>(p, s) : launch<128, 128, false>(p, s);
}

}  // namespace hc
