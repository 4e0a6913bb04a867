// Two attention results over different keys joined by their log sums:
//   top = max(lse_a, lse_b),  w = e^(lse - top),  out = (w_a a + w_b b) / (w_a + w_b),
//   lse = top + log(w_a + w_b)
// A side whose lse is -inf counts for nothing, whatever its row holds.
// Memory-bound: a, b read once, out written once, 16 bytes a thread (four such a
// thread: 38.4 us for 8197 tokens of 28 heads of 128 fp16 channels, one: 33.3);
// a row's pieces are lanes of one warp, so its log sums may be written over
// those that were read.
#include "paged.cuh"
#include "rope.cuh"

namespace hc {
namespace {

constexpr int kMergeThreads = 256;

// Read and written once: nothing of it is worth keeping in the caches (the above 33.3 us so, 31.5 with it).
template <typename T, int V>
__device__ __forceinline__ void load_once(const T* p, float (&x)[V]) {
  const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p));
  Piece<T, V> a;
  memcpy(&a, &w, 16);
  widen_piece(a, x);
}

template <typename T>
__global__ void __launch_bounds__(kMergeThreads) k_merge(const __grid_constant__ MergeParams p) {
  constexpr int V = 16 / sizeof(T);
  const int pieces = p.d / V;  // of a row: a power of two, at most 32
  const uint32_t i = blockIdx.x * kMergeThreads + threadIdx.x, row = i / pieces, ch = (i & (pieces - 1)) * V;
  if (row >= static_cast<uint32_t>(p.n_tokens) * p.n_heads) return;
  uint32_t token, head;
  p.by_heads.divmod(row, token, head);
  float x[V], y[V];
  load_once<T, V>(static_cast<const T*>(p.a) + token * p.a_token + head * p.a_head + ch, x);
  load_once<T, V>(static_cast<const T*>(p.b) + token * p.b_token + head * p.b_head + ch, y);
  const float la = p.lse_a[row], lb = p.lse_b[row], top = fmaxf(la, lb);
  const bool none = top == -INFINITY;
  const float wa = none ? 0.f : __expf(la - top), wb = none ? 0.f : __expf(lb - top);
  const float total = wa + wb, inv = none ? 0.f : 1.f / total;
  const float fa = wa * inv, fb = wb * inv;
#pragma unroll
  for (int k = 0; k < V; ++k) x[k] = (wa == 0.f ? 0.f : x[k] * fa) + (wb == 0.f ? 0.f : y[k] * fb);
  Piece<T, V> out;
  narrow_piece(x, out);
  uint4 w;
  memcpy(&w, &out, 16);
  __stcs(reinterpret_cast<uint4*>(static_cast<T*>(p.out) + token * p.o_token + head * p.o_head + ch), w);
  // the row's lanes have read its log sums; the warp's rows end together or not at all
  __syncwarp((pieces == 32 ? ~0u : (1u << pieces) - 1) << (threadIdx.x & 31 & -pieces));
  if (ch == 0 && p.lse) p.lse[row] = none ? -INFINITY : top + logf(total);
}

template <typename T>
cudaError_t launch(const MergeParams& p, cudaStream_t s) {
  const int64_t pieces = static_cast<int64_t>(p.n_tokens) * p.n_heads * (p.d * sizeof(T) / 16);
  k_merge<T><<<static_cast<unsigned>((pieces + kMergeThreads - 1) / kMergeThreads), kMergeThreads, 0, s>>>(p);
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
