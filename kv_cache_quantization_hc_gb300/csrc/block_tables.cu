// One step's addressing from request lengths: the slots of the new blocks,
// and each new token's request, position and cache row.
//
// With c, n the cached and new tokens of a request and B the block size, it
// holds ceil(c/B) blocks and needs ceil((c+n)/B) - ceil(c/B) more, taken from
// the free list in the order of the requests: two prefix sums (new tokens,
// new blocks), then one write per token and per new block.
//
// Every CTA computes the prefix sums of all requests for itself, 4096 at a
// time in shared memory: the lengths are 8 bytes per request, read from L2
// after the first CTA, which costs less than a second launch or a chain of
// CTAs waiting on one another.  A thread then takes 4 consecutive tokens and
// finds the first one's request by bisection.
//
// Lengths come from the device and may be anything: the sums stop at 2^31 - 1
// (counts.h), more than the arrays hold, and indexes near that are unsigned.
#include <algorithm>

#include "counts.h"
#include "serve.cuh"

namespace hc {
namespace {

constexpr int kTableThreads = 1024;
constexpr int kPerThread = 4;
constexpr int kChunk = kTableThreads * kPerThread;  // requests in shared memory
constexpr int kTokensPerItem = 4;

struct ChunkSmem {
  int32_t tok[kChunk];     // first new token of the request
  int32_t blk[kChunk];     // new blocks of the requests before it
  int32_t cached[kChunk];  // cached tokens; -1: a request with a bad length
  uint64_t warp[kTableThreads / 32];
  uint64_t total;
};

// Last i < n with a[i] <= x (a ascending, a[0] <= x).  Where several entries
// are equal this is the last of them: the one that is not empty.
__device__ __forceinline__ int last_not_above(const int32_t* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTableThreads) k_block_tables(BlockTableParams p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  ChunkSmem& s = *reinterpret_cast<ChunkSmem*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t gthread = blockIdx.x * kTableThreads + tid;
  const uint32_t gthreads = gridDim.x * kTableThreads;
  const int B = 1 << p.block_log2;
  uint64_t carry = 0;  // counts of the requests before this chunk
  int bad = 0;

  for (int r0 = 0; r0 < p.n_req; r0 += kChunk) {
    const int nr = min(kChunk, p.n_req - r0);
    const bool writes_requests = static_cast<int>(blockIdx.x) == (r0 / kChunk) % static_cast<int>(gridDim.x);
    uint64_t v[kPerThread], sum = 0;
    int c[kPerThread], kv[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int r = tid * kPerThread + i;
      v[i] = 0;
      c[i] = kv[i] = 0;
      if (r < nr) {
        const int64_t cr = __ldg(p.cached + r0 + r), n = __ldg(p.fresh + r0 + r);
        const bool ok = cr >= 0 && n >= 0 && cr + n <= (static_cast<int64_t>(p.table_width) << p.block_log2);
        if (!ok) bad |= HC_DEVERR_LENGTH;
        const int need = ok ? static_cast<int>(((cr + n + B - 1) >> p.block_log2) - ((cr + B - 1) >> p.block_log2)) : 0;
        c[i] = ok ? static_cast<int>(cr) : -1;
        kv[i] = ok ? static_cast<int>(cr + n) : 0;
        v[i] = counts(static_cast<uint32_t>(n > 0 ? n : 0), static_cast<uint32_t>(need));
        sum = add_counts(sum, v[i]);
      }
    }
    uint64_t inc = sum;  // inclusive scan over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc = add_counts(inc, t);
    }
    if (lane == 31) s.warp[warp] = inc;
    uint64_t before = __shfl_up_sync(0xffffffffu, inc, 1);  // the lanes before: a sum that stopped has no difference
    if (lane == 0) before = 0;
    __syncthreads();
    if (warp == 0) {
      uint64_t wi = s.warp[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t t = __shfl_up_sync(0xffffffffu, wi, o);
        if (lane >= o) wi = add_counts(wi, t);
      }
      const uint64_t w = __shfl_up_sync(0xffffffffu, wi, 1);
      s.warp[lane] = lane == 0 ? 0 : w;
      if (lane == 31) s.total = wi;
    }
    __syncthreads();
    uint64_t at = add_counts(carry, add_counts(s.warp[warp], before));
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int r = tid * kPerThread + i;
      if (r < nr) {
        s.tok[r] = static_cast<int32_t>(tokens_of(at));
        s.blk[r] = static_cast<int32_t>(blocks_of(at));
        s.cached[r] = c[i];
        if (writes_requests) {
          p.q_starts[r0 + r] = static_cast<int32_t>(tokens_of(at));
          p.kv_lens[r0 + r] = kv[i];
        }
      }
      at = add_counts(at, v[i]);
    }
    const uint64_t next = add_counts(carry, s.total);
    __syncthreads();

    // new blocks: their slots, from the front of the free list
    const uint32_t b_end = blocks_of(next), n_free = static_cast<uint32_t>(p.n_free);
    for (uint32_t b = blocks_of(carry) + gthread; b < b_end; b += gthreads) {
      const int r = last_not_above(s.blk, nr, static_cast<int>(b));
      const int j = ((s.cached[r] + B - 1) >> p.block_log2) + static_cast<int>(b) - s.blk[r];
      int slot = -1;
      if (b < n_free) slot = __ldg(p.free_slots + b); else bad |= HC_DEVERR_FREE;
      p.tables[(r0 + r) * p.table_stride + j] = slot;
    }

    // new tokens, 4 to a thread
    const int t0 = static_cast<int>(tokens_of(carry)), t_end = static_cast<int>(tokens_of(next));
    if (t_end > p.n_tokens) bad |= HC_DEVERR_LENGTH;
    const int t1 = min(t_end, p.n_tokens);
    for (uint32_t item = t0 / kTokensPerItem + gthread; item * kTokensPerItem < static_cast<uint32_t>(t1); item += gthreads) {
      const int t = static_cast<int>(item * kTokensPerItem);
      int req[4], pos[4];
      int64_t row[4];
      int r = last_not_above(s.tok, nr, max(t, t0));
      const bool whole = t >= t0 && t <= t1 - 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        req[i] = pos[i] = 0;
        row[i] = -1;
        if (t < t0 - i || t >= t1 - i) continue;
        const int ti = t + i;
        while (r + 1 < nr && s.tok[r + 1] <= ti) ++r;
        const int cr = s.cached[r];
        req[i] = r0 + r;
        if (cr >= 0) {
          pos[i] = cr + ti - s.tok[r];
          const int j = pos[i] >> p.block_log2, held = (cr + B - 1) >> p.block_log2;
          int slot;
          if (j < held) {
            slot = p.tables[(r0 + r) * p.table_stride + j];
          } else {
            const uint32_t b = static_cast<uint32_t>(s.blk[r]) + static_cast<uint32_t>(j - held);
            slot = b < n_free ? __ldg(p.free_slots + b) : -1;
          }
          if (slot >= 0) row[i] = (static_cast<int64_t>(slot) << p.block_log2) + (pos[i] & (B - 1));
        }
        if (!(whole && p.vec)) {
          p.token_req[ti] = req[i];
          p.token_pos[ti] = pos[i];
          p.token_rows[ti] = row[i];
        }
      }
      if (whole && p.vec) {
        *reinterpret_cast<int4*>(p.token_req + t) = make_int4(req[0], req[1], req[2], req[3]);
        *reinterpret_cast<int4*>(p.token_pos + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<longlong2*>(p.token_rows + t) = make_longlong2(row[0], row[1]);
        *reinterpret_cast<longlong2*>(p.token_rows + t + 2) = make_longlong2(row[2], row[3]);
      }
    }
    carry = next;
    __syncthreads();
  }

  const uint32_t total = tokens_of(carry);
  for (uint32_t t = total + gthread; t < static_cast<uint32_t>(p.n_tokens); t += gthreads) {  // a step padded to n_tokens
    p.token_req[t] = -1;
    p.token_pos[t] = 0;
    p.token_rows[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.q_starts[p.n_req] = static_cast<int32_t>(total);
    *p.n_taken = min(static_cast<int32_t>(blocks_of(carry)), p.n_free);
  }
  flag_error(p.err, bad);
}

}  // namespace

cudaError_t launch_block_tables(const BlockTableParams& p, cudaStream_t s) {
  static KernelOnDevice kernel;
  int resident = 0;
  const cudaError_t e = kernel.resident(reinterpret_cast<const void*>(k_block_tables), kTableThreads,
                                        static_cast<int>(sizeof(ChunkSmem)), &resident);
  if (e != cudaSuccess) return e;
  // one thread per 4 tokens or per new block (at most one per request and block of tokens)
  const int64_t blocks = (static_cast<int64_t>(p.n_tokens) >> p.block_log2) + p.n_req;
  const int64_t items = std::max<int64_t>((static_cast<int64_t>(p.n_tokens) + 3) / 4, blocks);
  const int64_t ctas = (items + kTableThreads - 1) / kTableThreads;
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(ctas, resident)));
  k_block_tables<<<grid, kTableThreads, sizeof(ChunkSmem), s>>>(p);
  return cudaGetLastError();
}

}  // namespace hc
