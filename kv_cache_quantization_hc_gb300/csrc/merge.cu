// Two attention results over different keys joined by their log sums:
//   top = max(lse_a, lse_b),  w = e^(lse - top),  out = (w_a a + w_b b) / (w_a + w_b),
//   lse = top + log(w_a + w_b)
// A side whose lse is -inf counts for nothing, whatever its row holds.
// Memory-bound: a, b read once, out written once, 16 bytes a thread at a time;
// a row's pieces are lanes of one warp, so its log sums may be written over
// those that were read.
#include "paged.cuh"
#include "rope.cuh"

namespace hc {
namespace {

constexpr int kMergeThreads = 256;

template <typename T, int kUnroll>
__global__ void __launch_bounds__(kMergeThreads) k_merge(const __grid_constant__ MergeParams p) {
  constexpr int V = 16 / sizeof(T);
  const int pieces = p.d / V;  // of a row: a power of two, at most 32
  const uint32_t total = static_cast<uint32_t>(p.n_tokens) * p.n_heads * pieces;
  const uint32_t first = blockIdx.x * (kMergeThreads * kUnroll) + threadIdx.x;
  Piece<T, V> a[kUnroll], b[kUnroll];
  float la[kUnroll], lb[kUnroll];
  uint32_t token[kUnroll], head[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t i = first + u * kMergeThreads;
    if (i >= total) continue;
    const uint32_t row = i / pieces, ch = (i & (pieces - 1)) * V;
    p.by_heads.divmod(row, token[u], head[u]);
    a[u] = load_piece<T, V>(static_cast<const T*>(p.a) + token[u] * p.a_token + head[u] * p.a_head + ch);
    b[u] = load_piece<T, V>(static_cast<const T*>(p.b) + token[u] * p.b_token + head[u] * p.b_head + ch);
    la[u] = p.lse_a[row];
    lb[u] = p.lse_b[row];
  }
  __syncwarp();
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t i = first + u * kMergeThreads;
    if (i >= total) continue;
    const uint32_t row = i / pieces, ch = (i & (pieces - 1)) * V;
    const float top = fmaxf(la[u], lb[u]);
    const bool none = top == -INFINITY;
    const float wa = none ? 0.f : __expf(la[u] - top), wb = none ? 0.f : __expf(lb[u] - top);
    const float total_w = wa + wb, inv = none ? 0.f : 1.f / total_w;
    const float fa = wa * inv, fb = wb * inv;
    float x[V], y[V];
    widen_piece(a[u], x);
    widen_piece(b[u], y);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      x[k] = (wa == 0.f ? 0.f : x[k] * fa) + (wb == 0.f ? 0.f : y[k] * fb);
    }
    narrow_piece(x, a[u]);
    store_piece<T, V>(static_cast<T*>(p.out) + token[u] * p.o_token + head[u] * p.o_head + ch, a[u]);
    if (ch == 0 && p.lse) p.lse[row] = none ? -INFINITY : top + logf(total_w);
  }
}

template <typename T>
cudaError_t launch(const MergeParams& p, cudaStream_t s) {
  const int64_t pieces = static_cast<int64_t>(p.n_tokens) * p.n_heads * (p.d * sizeof(T) / 16);
  // few pieces: one a thread, on as many SMs as there are
  if (pieces <= int64_t{device_sm_count()} * kMergeThreads * 4)
    k_merge<T, 1><<<static_cast<unsigned>((pieces + kMergeThreads - 1) / kMergeThreads), kMergeThreads, 0, s>>>(p);
  else
    k_merge<T, 4><<<static_cast<unsigned>((pieces + 4 * kMergeThreads - 1) / (4 * kMergeThreads)), kMergeThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_merge(int dtype, const MergeParams& p, cudaStream_t s) {
  switch (dtype) {
    case HC_F32: return launch<float>(p, s);
    case HC_F16: return launch<__half>(p, s);
    default: return launch<__nv_bfloat16>(p, s);
  }
}

}  // namespace hc
