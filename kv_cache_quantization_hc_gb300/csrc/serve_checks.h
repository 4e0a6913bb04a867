// Checks of arguments shared by the serving calls' C entries.
#pragma once

#include <cstring>

#include "serve.cuh"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int elem_size(int dtype) { return dtype == HC_F32 ? 4 : dtype == HC_F16 || dtype == HC_BF16 ? 2 : 0; }

inline int block_log2(int block_size) {
  switch (block_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
  }
  return -1;
}

// A table of n_req rows, and lengths that stay below 2^31.
inline bool table_ok(const int32_t* tables, int64_t stride, int32_t width, int32_t n_req, int log2) {
  if (width < 0 || stride < width || (int64_t{width} << log2) >= (int64_t{1} << 31)) return false;
  return n_req == 0 || width == 0 || (tables && aligned(tables, 4));
}

// Rows moved in 16-byte pieces: base, strides and row length.
inline bool rows16(const hc_rows& r, int es, int64_t n_tokens, int64_t n_heads) {
  return aligned(r.ptr, 16) && (n_tokens <= 1 || (r.token_stride * es) % 16 == 0) &&
         (n_heads <= 1 || (r.head_stride * es) % 16 == 0);
}
// Nothing is behind a pointer to no elements, which may be NULL.
inline bool rows_ok(const hc_rows* r, int es, bool any) {
  return r && (r->ptr || !any) && aligned(r->ptr, es) && r->token_stride >= 0 && r->head_stride >= 0;
}

// Rows that are written: closer together than they are long (a broadcast tensor's), warps would write over each other.
inline bool rows_apart(const hc_rows& r, int64_t n_tokens, int64_t n_heads, int64_t d) {
  return n_tokens == 0 || n_heads == 0 ||
         ((n_tokens == 1 || r.token_stride >= d) && (n_heads == 1 || r.head_stride >= d));
}

inline int check_rope(const hc_rope_axes_desc* r, int d_head, int64_t n_tokens, hc::RopeParams* out) {
  if (!r || (!r->positions && n_tokens > 0) || !r->table) return HC_ERR_INVALID_ARG;
  if (r->n_axes < 1 || r->n_axes > 8 || r->n_positions < 1) return HC_ERR_INVALID_ARG;
  if (r->rot_dim < 2 || r->rot_dim > 256 || (r->rot_dim & 1) || r->rot_dim > d_head) return HC_ERR_INVALID_ARG;
  if (r->pairing != HC_PAIR_INTERLEAVED && r->pairing != HC_PAIR_HALF_SPLIT) return HC_ERR_INVALID_ARG;
  if (r->inverse != 0 && r->inverse != 1) return HC_ERR_INVALID_ARG;
  if (r->position_stride < 0 || (r->n_axes > 1 && r->position_stride < n_tokens)) return HC_ERR_INVALID_ARG;
  if (!aligned(r->positions, 4) || !aligned(r->table, 8)) return HC_ERR_INVALID_ARG;
  for (int i = 0; i < r->rot_dim / 2; ++i)
    if (r->pair_axis[i] >= r->n_axes) return HC_ERR_INVALID_ARG;
  out->positions = r->positions;
  out->position_stride = r->position_stride;
  out->table = reinterpret_cast<const float2*>(r->table);
  out->n_positions = r->n_positions;
  out->half = r->rot_dim / 2;
  out->inverse = r->inverse;
  std::memcpy(out->pair_axis, r->pair_axis, sizeof out->pair_axis);
  out->axes = 0;
  for (int i = 0; i < out->half; ++i) out->axes |= 1u << r->pair_axis[i];
  out->pairs16 = aligned(r->table, 16) && out->half % 2 == 0;
  return HC_OK;
}

}  // namespace
