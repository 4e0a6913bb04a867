// C ABI of the serving operators over a 4-bit cache: host-side validation,
// then the launch on the caller's stream.
#include <algorithm>
#include <cmath>

#include "serve_checks.h"

namespace {

int check_cache(const hc_int4_cache* c, const void* codes, const void* scales) {
  if (!c || !codes || !scales) return HC_ERR_INVALID_ARG;
  if (c->n_kv_heads < 1 || c->num_slots < 1 || c->d_head < 1 || c->block_size < 1) return HC_ERR_INVALID_ARG;
  if (c->scale_dtype != HC_F16 && c->scale_dtype != HC_F32) return HC_ERR_INVALID_ARG;
  if (c->d_head != 64 && c->d_head != 128) return HC_ERR_UNSUPPORTED;
  if (block_log2(c->block_size) < 0) return HC_ERR_UNSUPPORTED;
  if ((c->group != 32 && c->group != 64 && c->group != 128) || c->group > c->d_head) return HC_ERR_UNSUPPORTED;
  if (!aligned(codes, 16) || !aligned(scales, 16)) return HC_ERR_INVALID_ARG;
  return HC_OK;
}

// A request with more query rows (new tokens times query heads per cache
// head) than this is attended in tiles of 256 rows on the 5th-generation
// tensor cores (one CTA walks all keys of a tile), one with fewer in pieces of
// 16 rows whose keys are split over the SMs.  A piece costs the GPU as a whole
// about 1/200 of what a tile costs its SM (64 channels: 1/340), so what counts
// is how many tiles there are: below one per SM the rest of the GPU is idle.
// Even lengths, bf16, groups of 32 and 8 heads of 128 channels, rows against
// tiles: 16 requests of 4000 keys, 28 rows 71 us against 62, 80 rows 146
// against 62, 160 rows 271 against 64; 4 requests, 80 rows 52 against 60, 160
// rows 83 against 62; 1 request, 384 rows 43 against 39 (2000 keys), 164
// against 191 (16000).  2 heads of 64 channels, 16 requests of 4000 keys, 140
// rows 49 against 53, 280 rows 79 against 54.  Pieces share out ragged
// lengths, tiles wait for the longest: the factors lean to the pieces by half.
int rows_for_pieces(int64_t n_req, int64_t heads, int d_head) {
  const int64_t sms = hc::device_sm_count();
  constexpr int kMost = 384;
  const int64_t each = n_req * heads, factor = d_head == 128 ? 300 : 500;
  for (int rows = 16; rows <= kMost; rows += 16) {
    const int64_t tiles = each * ((rows + 255) / 256);
    if (each * (rows / 16) > factor * ((tiles + sms - 1) / sms)) return std::max(16, rows - 16);
  }
  return kMost;
}

int append_int4(const hc_rows* q, const hc_rows* k, const hc_rows* v, int32_t dtype, int32_t n_tokens,
                int32_t n_q_heads, const hc_rope_axes_desc* rope, const int64_t* token_rows,
                const hc_int4_cache* cache, uint8_t* codes, void* scales, const hc_rows* q_out, int32_t* err_flag,
                bool wire_scales, void* stream) {
  const int es = elem_size(dtype);
  if (es == 0 || n_tokens < 0 || n_q_heads < 0) return HC_ERR_INVALID_ARG;
  int st = check_cache(cache, codes, scales);
  if (st != HC_OK) return st;
  const bool any = n_tokens > 0;
  if (!rows_ok(k, es, any) || !rows_ok(v, es, any) || (!token_rows && any) || !err_flag) return HC_ERR_INVALID_ARG;
  if (n_q_heads > 0 && (!rows_ok(q, es, any) || !rows_ok(q_out, es, any))) return HC_ERR_INVALID_ARG;
  if (n_q_heads > 0 && !rows_apart(*q_out, n_tokens, n_q_heads, cache->d_head)) return HC_ERR_INVALID_ARG;
  if (!aligned(token_rows, 8) || !aligned(err_flag, 4)) return HC_ERR_INVALID_ARG;
  hc::AppendParams p;
  std::memset(&p.rope, 0, sizeof p.rope);
  int pairing = HC_PAIR_HALF_SPLIT;
  if (rope) {
    st = check_rope(rope, cache->d_head, n_tokens, &p.rope);
    if (st != HC_OK) return st;
    if (rope->inverse) return HC_ERR_INVALID_ARG;
    if (rope->rot_dim % 16) return HC_ERR_UNSUPPORTED;
    pairing = rope->pairing;
  }
  if (!rows16(*k, es, n_tokens, cache->n_kv_heads) || !rows16(*v, es, n_tokens, cache->n_kv_heads) ||
      (n_q_heads > 0 && (!rows16(*q, es, n_tokens, n_q_heads) || !rows16(*q_out, es, n_tokens, n_q_heads))))
    return HC_ERR_INVALID_ARG;
  if ((int64_t{n_q_heads} + cache->n_kv_heads) * cache->d_head >= (int64_t{1} << 31) ||
      int64_t{n_tokens} * (int64_t{n_q_heads} + cache->n_kv_heads) >= (int64_t{1} << 31) - 8)
    return HC_ERR_INVALID_ARG;
  if (n_tokens == 0) return HC_OK;
  p.q = n_q_heads ? q->ptr : nullptr;
  p.q_out = n_q_heads ? q_out->ptr : nullptr;
  p.q_token = n_q_heads ? q->token_stride : 0;
  p.q_head = n_q_heads ? q->head_stride : 0;
  p.o_token = n_q_heads ? q_out->token_stride : 0;
  p.o_head = n_q_heads ? q_out->head_stride : 0;
  p.k = k->ptr;
  p.k_token = k->token_stride;
  p.k_head = k->head_stride;
  p.v = v->ptr;
  p.v_token = v->token_stride;
  p.v_head = v->head_stride;
  p.n_tokens = n_tokens;
  p.n_q_heads = n_q_heads;
  p.H = cache->n_kv_heads;
  p.B_log2 = block_log2(cache->block_size);
  p.group_log2 = cache->group == 128 ? 7 : cache->group == 64 ? 6 : 5;
  p.scale_f16 = cache->scale_dtype == HC_F16;
  p.wire_scales = wire_scales;
  p.token_rows = token_rows;
  p.n_rows = int64_t{cache->num_slots} * cache->block_size;
  p.codes = codes;
  p.scales = scales;
  p.err = err_flag;
  return hc::record_cuda(
      hc::launch_append_int4(dtype, cache->d_head, pairing, p, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int hc_build_block_tables(const int32_t* cached_lens, const int32_t* new_lens, int32_t n_req,
                          int32_t block_size, const int32_t* free_slots, int32_t n_free,
                          int32_t* block_tables, int64_t table_stride, int32_t table_width,
                          int32_t n_tokens, int32_t* q_starts, int32_t* kv_lens,
                          int32_t* token_req, int32_t* token_pos, int64_t* token_rows,
                          int32_t* n_taken, int32_t* err_flag, void* stream) {
  // a sum that stops at 2^31 - 1 is then more than the call holds, and flagged
  if (n_req < 0 || n_free < 0 || n_tokens < 0 || n_free == INT32_MAX || n_tokens == INT32_MAX || block_size < 1)
    return HC_ERR_INVALID_ARG;
  const int log2 = block_log2(block_size);
  if (log2 < 0) return HC_ERR_UNSUPPORTED;
  if (!q_starts || !n_taken || !err_flag) return HC_ERR_INVALID_ARG;
  if (n_req > 0 && (!cached_lens || !new_lens || !kv_lens)) return HC_ERR_INVALID_ARG;
  if (n_free > 0 && !free_slots) return HC_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!token_req || !token_pos || !token_rows)) return HC_ERR_INVALID_ARG;
  if (!table_ok(block_tables, table_stride, table_width, n_req, log2)) return HC_ERR_INVALID_ARG;
  if (!aligned(cached_lens, 4) || !aligned(new_lens, 4) || !aligned(free_slots, 4) || !aligned(q_starts, 4) ||
      !aligned(kv_lens, 4) || !aligned(token_req, 4) || !aligned(token_pos, 4) || !aligned(token_rows, 8) ||
      !aligned(n_taken, 4) || !aligned(err_flag, 4))
    return HC_ERR_INVALID_ARG;
  hc::BlockTableParams p;
  p.cached = cached_lens;
  p.fresh = new_lens;
  p.free_slots = free_slots;
  p.tables = block_tables;
  p.table_stride = table_stride;
  p.n_req = n_req;
  p.n_free = n_free;
  p.table_width = table_width;
  p.n_tokens = n_tokens;
  p.block_log2 = log2;
  p.q_starts = q_starts;
  p.kv_lens = kv_lens;
  p.token_req = token_req;
  p.token_pos = token_pos;
  p.token_rows = token_rows;
  p.n_taken = n_taken;
  p.err = err_flag;
  p.vec = aligned(token_req, 16) && aligned(token_pos, 16) && aligned(token_rows, 16);
  return hc::record_cuda(hc::launch_block_tables(p, static_cast<cudaStream_t>(stream)));
}

int hc_rope_axes(const hc_rows* x, const hc_rows* y, int32_t dtype, int32_t n_tokens,
                 int32_t n_heads, int32_t d_head, const hc_rope_axes_desc* rope,
                 int32_t* err_flag, void* stream) {
  const int es = elem_size(dtype);
  if (es == 0 || n_tokens < 0 || n_heads < 0 || d_head < 2 || d_head > 256) return HC_ERR_INVALID_ARG;
  const bool any = n_tokens > 0 && n_heads > 0;
  if (!rows_ok(x, es, any) || !rows_ok(y, es, any) || !err_flag || !aligned(err_flag, 4)) return HC_ERR_INVALID_ARG;
  if (!rows_apart(*y, n_tokens, n_heads, d_head)) return HC_ERR_INVALID_ARG;
  hc::RopeAxesParams p;
  const int st = check_rope(rope, d_head, n_tokens, &p.rope);
  if (st != HC_OK) return st;
  // the kernels index a token's pieces, and the grid's warps, in 32 bits
  if (int64_t{n_heads} * d_head >= (int64_t{1} << 31) || int64_t{n_tokens} * n_heads >= (int64_t{1} << 31) - 8)
    return HC_ERR_INVALID_ARG;
  if (n_tokens == 0 || n_heads == 0) return HC_OK;
  const int piece = 16 / es, half = rope->rot_dim / 2;
  const bool whole_pieces = rope->pairing == HC_PAIR_HALF_SPLIT
                                ? half % piece == 0 && (d_head - 2 * half) % piece == 0
                                : 2 * half % piece == 0 && (d_head - 2 * half) % piece == 0;
  const bool pieces16 = whole_pieces && rows16(*x, es, n_tokens, n_heads) && rows16(*y, es, n_tokens, n_heads);
  if (!pieces16 && rope->pairing == HC_PAIR_INTERLEAVED && (d_head & 1)) return HC_ERR_UNSUPPORTED;
  p.x = x->ptr;
  p.y = y->ptr;
  p.x_token = x->token_stride;
  p.x_head = x->head_stride;
  p.y_token = y->token_stride;
  p.y_head = y->head_stride;
  p.n_tokens = n_tokens;
  p.n_heads = n_heads;
  p.d = d_head;
  p.err = err_flag;
  return hc::record_cuda(
      hc::launch_rope_axes(dtype, rope->pairing, pieces16, p, static_cast<cudaStream_t>(stream)));
}

int hc_append_int4(const hc_rows* q, const hc_rows* k, const hc_rows* v, int32_t dtype,
                   int32_t n_tokens, int32_t n_q_heads, const hc_rope_axes_desc* rope,
                   const int64_t* token_rows, const hc_int4_cache* cache, uint8_t* codes,
                   void* scales, const hc_rows* q_out, int32_t* err_flag, void* stream) {
  return append_int4(q, k, v, dtype, n_tokens, n_q_heads, rope, token_rows, cache, codes, scales, q_out, err_flag,
                     false, stream);
}

int hc_append_int4_wire(const hc_rows* q, const hc_rows* k, const hc_rows* v, int32_t dtype,
                        int32_t n_tokens, int32_t n_q_heads, const hc_rope_axes_desc* rope,
                        const int64_t* token_rows, const hc_int4_cache* cache, uint8_t* codes,
                        void* scales, const hc_rows* q_out, int32_t* err_flag, void* stream) {
  return append_int4(q, k, v, dtype, n_tokens, n_q_heads, rope, token_rows, cache, codes, scales, q_out, err_flag,
                     true, stream);
}

int32_t hc_attend_int4_few_rows(int32_t n_req, int32_t n_kv_heads, int32_t d_head) {
  if (n_req < 1 || n_kv_heads < 1 || d_head < 1) return HC_ERR_INVALID_ARG;
  if (d_head != 64 && d_head != 128) return HC_ERR_UNSUPPORTED;
  return rows_for_pieces(n_req, n_kv_heads, d_head);
}

int64_t hc_attend_int4_workspace(void) { return hc::attend_workspace_bytes(); }

int hc_attend_int4(const hc_rows* q, const hc_rows* out, float* lse, int32_t dtype,
                   int32_t n_tokens, int32_t n_q_heads, const hc_int4_cache* cache,
                   const uint8_t* codes, const void* scales, const int32_t* block_tables,
                   int64_t table_stride, int32_t table_width, const int32_t* q_starts,
                   const int32_t* kv_lens, int32_t n_req, int32_t max_new, int32_t causal,
                   int32_t window, float softmax_scale, void* workspace,
                   int64_t workspace_bytes, int32_t* err_flag, void* stream) {
  const int es = elem_size(dtype);
  if (es == 0 || n_tokens < 0 || n_q_heads < 1 || n_req < 0 || max_new < 0) return HC_ERR_INVALID_ARG;
  const int st = check_cache(cache, codes, scales);
  if (st != HC_OK) return st;
  if (dtype == HC_F32) return HC_ERR_UNSUPPORTED;
  if (n_q_heads % cache->n_kv_heads) return HC_ERR_INVALID_ARG;
  if (!rows_ok(q, es, n_tokens > 0) || !rows_ok(out, es, n_tokens > 0) || !err_flag || !aligned(err_flag, 4) || (lse && !aligned(lse, 4)))
    return HC_ERR_INVALID_ARG;
  if (!rows16(*q, es, n_tokens, n_q_heads) || !rows16(*out, es, n_tokens, n_q_heads)) return HC_ERR_INVALID_ARG;
  if (!rows_apart(*out, n_tokens, n_q_heads, cache->d_head)) return HC_ERR_INVALID_ARG;
  if (!q_starts || !aligned(q_starts, 4) || (n_req > 0 && (!kv_lens || !aligned(kv_lens, 4))))
    return HC_ERR_INVALID_ARG;
  const int log2 = block_log2(cache->block_size);
  if (!table_ok(block_tables, table_stride, table_width, n_req, log2)) return HC_ERR_INVALID_ARG;
  if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal)) return HC_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale)) return HC_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < hc::attend_workspace_bytes())
    return HC_ERR_INVALID_ARG;
  const int G = n_q_heads / cache->n_kv_heads;
  // rows of a request, and pieces of 8 rows times tiles of 128 keys of a call, are counted in 32 bits
  if (int64_t{max_new} * G >= (int64_t{1} << 30)) return HC_ERR_INVALID_ARG;
  const int rows_above = n_req > 0 ? rows_for_pieces(n_req, cache->n_kv_heads, cache->d_head) : 0;
  const int64_t pieces = (std::min<int64_t>(int64_t{max_new} * G, rows_above) + 7) / 8;
  const int64_t tiles = ((int64_t{table_width} << log2) + 127) / 128 + 2;
  if (static_cast<double>(n_req) * cache->n_kv_heads * static_cast<double>(pieces * tiles) >= 0x1p31)
    return HC_ERR_INVALID_ARG;
  if (n_tokens == 0 || n_req == 0 || max_new == 0) return HC_OK;
  hc::AttendParams p;
  p.q = q->ptr;
  p.out = out->ptr;
  p.lse = lse;
  p.q_token = q->token_stride;
  p.q_head = q->head_stride;
  p.o_token = out->token_stride;
  p.o_head = out->head_stride;
  p.codes = codes;
  p.scales = scales;
  p.tables = block_tables;
  p.table_stride = table_stride;
  p.q_starts = q_starts;
  p.kv_lens = kv_lens;
  p.n_req = n_req;
  p.n_tokens = n_tokens;
  p.max_new = max_new;
  p.table_width = table_width;
  p.most_keys = static_cast<int32_t>(std::min(int64_t{table_width} << log2, hc::kMostKeys));
  p.num_slots = cache->num_slots;
  p.H = cache->n_kv_heads;
  p.G = G;
  p.B_log2 = log2;
  p.bf16 = dtype == HC_BF16;
  p.causal = causal;
  p.window = window;
  p.by_group = hc::FastDivmod(static_cast<uint32_t>(G));
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.workspace = static_cast<uint8_t*>(workspace);
  p.err = err_flag;
  p.rows_above = rows_above;
  const bool scale_f16 = cache->scale_dtype == HC_F16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (int64_t{max_new} * G > p.rows_above) {
    const int t = hc::record_cuda(hc::launch_attend_tiles(cache->d_head, cache->group, scale_f16, p, s));
    if (t != HC_OK) return t;
  }
  return hc::record_cuda(hc::launch_attend_rows(cache->d_head, cache->group, scale_f16, p, s));
}

}  // extern "C"
