// C ABI of the serving operators over the paged buffer: host-side validation,
// then the launch on the caller's stream.
#include <algorithm>
#include <cmath>

#include "paged.cuh"
#include "serve_checks.h"

namespace {

// One layer's pages.
int check_pages(const hc_paged_desc* d, const void* k, const void* v) {
  if (!d || !k || !v || elem_size(d->dtype) == 0) return HC_ERR_INVALID_ARG;
  if (d->n_layers != 1 || d->n_kv_heads < 1 || d->num_slots < 1 || d->d_head < 1 || d->block_size < 1)
    return HC_ERR_INVALID_ARG;
  if (d->d_head != 64 && d->d_head != 128) return HC_ERR_UNSUPPORTED;
  if (block_log2(d->block_size) < 0) return HC_ERR_UNSUPPORTED;
  // a slot's stride in bytes fits a copy descriptor's 40 bits
  if (d->slot_stride < int64_t{d->block_size} * d->n_kv_heads * d->d_head || d->slot_stride >= int64_t{1} << 37)
    return HC_ERR_INVALID_ARG;
  if ((d->slot_stride * elem_size(d->dtype)) % 16 || !aligned(k, 16) || !aligned(v, 16)) return HC_ERR_INVALID_ARG;
  return HC_OK;
}

// The rows kernel's counters, then partial sums: the tiles kernel's, and once those are joined the rows kernel's; at
// the end the list of the runs to join and the tiles kernel's four counters.
constexpr int64_t kWorkspace = int64_t{32} << 20, kTileCounters = 256, kJoinList = hc::kSplitRuns * 32;
int64_t workspace_bytes_needed() { return std::max(kWorkspace, hc::attend_paged_rows_bytes() + kJoinList + kTileCounters); }

int64_t part_bytes() { return workspace_bytes_needed() - kJoinList - kTileCounters - hc::attend_paged_counter_bytes(); }

// A request with more query rows (new tokens times query heads per cache head)
// than this is attended in tiles of 256 rows on the 5th-generation tensor cores,
// one with fewer in pieces of 16 rows whose keys are split over the SMs.  What
// each takes, in us, fitted to both kernels (1 to 64 requests of 1000 to 30000
// keys, 2 and 8 cache heads, 16 to 512 rows):
//   pieces: 11 + 0.0118 (64 channels: 0.0062) for each piece and 128 keys of a head
//   tiles:  14 + 1.27 (0.88) for each tile of the slowest SM
// The host knows the longest length at most.  Of many requests a piece's keys are
// taken to be a quarter of it and the slowest SM's tiles half, of n the n-th of
// the way back; and where some requests are in pieces and others in tiles, one
// kernel waits for the other: 12.
// Pieces against tiles, of 128 channels and 8 heads: one request of 3000 keys, 256
// rows 41 against 31, of 1000 keys, 64 rows 17 against 25; 16 requests of 4000 keys,
// 16 rows 57 against 60, 32 rows 84 against 60; 16 of 200 to 22000 keys, 64 rows
// 193 against 103; of 64 channels, 2 heads, 37 of 60 to 8400 keys, 14 to 49 rows
// 21 against 50, 112 rows 46 against 49.
int rows_for_pieces(int64_t n_req, int64_t heads, int d_head, int64_t keys) {
  const int sms = hc::device_sm_count();
  constexpr int kMost = 1024;
  const int64_t each = n_req * heads, tiles = std::max<int64_t>(1, (keys + 127) / 128);
  const int64_t places = part_bytes() / (256 * (d_head * 4 + 8));
  const double known = 1.0 / static_cast<double>(n_req);
  const double piece = (0.25 + 0.75 * known) * (d_head == 128 ? 0.0118 : 0.0062) * static_cast<double>(each) * static_cast<double>(tiles);
  for (int block = 1; block * 256 <= kMost; ++block) {
    const double slowest = (0.5 + 0.5 * known) * hc::even_time(n_req, each * block, keys, 256, places, sms);
    const double time = 14 + (d_head == 128 ? 1.27 : 0.88) * slowest + (n_req > 1 ? 12 : 0);
    const double rows = 16 * std::floor((time - 11) / piece);
    if (rows < block * 256) return std::max(16, std::max(static_cast<int>(rows), (block - 1) * 256));
  }
  return kMost;
}

}  // namespace

extern "C" {

int hc_append_paged(const hc_rows* q, const hc_rows* k, const hc_rows* v, int32_t n_tokens, int32_t n_q_heads,
                    const hc_rope_axes_desc* rope, const int64_t* token_rows, const hc_paged_desc* desc, void* k_pages,
                    void* v_pages, const hc_rows* q_out, int32_t* err_flag, void* stream) {
  if (n_tokens < 0 || n_q_heads < 0) return HC_ERR_INVALID_ARG;
  int st = check_pages(desc, k_pages, v_pages);
  if (st != HC_OK) return st;
  if (k_pages == v_pages) return HC_ERR_INVALID_ARG;
  const int es = elem_size(desc->dtype);
  const int64_t H = desc->n_kv_heads, d = desc->d_head;
  const bool any = n_tokens > 0;
  if (!rows_ok(k, es, any) || !rows_ok(v, es, any) || (!token_rows && any) || !err_flag) return HC_ERR_INVALID_ARG;
  if (n_q_heads > 0 && (!rows_ok(q, es, any) || !rows_ok(q_out, es, any))) return HC_ERR_INVALID_ARG;
  if (n_q_heads > 0 && !rows_apart(*q_out, n_tokens, n_q_heads, d)) return HC_ERR_INVALID_ARG;
  if (!aligned(token_rows, 8) || !aligned(err_flag, 4)) return HC_ERR_INVALID_ARG;
  hc::AppendPagedParams p;
  std::memset(&p.rope, 0, sizeof p.rope);
  int pairing = HC_PAIR_HALF_SPLIT;
  if (rope) {
    st = check_rope(rope, desc->d_head, n_tokens, &p.rope);
    if (st != HC_OK) return st;
    if (rope->inverse) return HC_ERR_INVALID_ARG;
    if (rope->rot_dim % 16) return HC_ERR_UNSUPPORTED;
    pairing = rope->pairing;
  }
  if (!rows16(*k, es, n_tokens, H) || !rows16(*v, es, n_tokens, H) ||
      (n_q_heads > 0 && (!rows16(*q, es, n_tokens, n_q_heads) || !rows16(*q_out, es, n_tokens, n_q_heads))))
    return HC_ERR_INVALID_ARG;
  // a token's pieces, and the grid's warps, are counted in 32 bits
  if ((n_q_heads + 2 * H) * d >= (int64_t{1} << 31) || n_tokens * (n_q_heads + 2 * H) >= (int64_t{1} << 31) - 8)
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
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.slot_stride = desc->slot_stride;
  p.n_tokens = n_tokens;
  p.n_q_heads = n_q_heads;
  p.H = desc->n_kv_heads;
  p.d = desc->d_head;
  p.B_log2 = block_log2(desc->block_size);
  p.token_rows = token_rows;
  p.n_rows = int64_t{desc->num_slots} * desc->block_size;
  p.err = err_flag;
  return hc::record_cuda(hc::launch_append_paged(desc->dtype, pairing, p, static_cast<cudaStream_t>(stream)));
}

int32_t hc_attend_paged_few_rows(int32_t n_req, int32_t n_kv_heads, int32_t d_head, int64_t table_keys) {
  if (n_req < 1 || n_kv_heads < 1 || d_head < 1 || table_keys < 0 || table_keys >= int64_t{1} << 31) return HC_ERR_INVALID_ARG;
  if (d_head != 64 && d_head != 128) return HC_ERR_UNSUPPORTED;
  return rows_for_pieces(n_req, n_kv_heads, d_head, table_keys);
}

int64_t hc_attend_paged_workspace(void) { return workspace_bytes_needed(); }

int hc_attend_paged(const hc_rows* q, const hc_rows* out, float* lse, int32_t n_tokens, int32_t n_q_heads,
                    const hc_paged_desc* desc, const void* k_pages, const void* v_pages, const int32_t* block_tables,
                    int64_t table_stride, int32_t table_width, const int32_t* q_starts, const int32_t* kv_lens,
                    int32_t n_req, int32_t max_new, const hc_attend_scores* scores, void* workspace,
                    int64_t workspace_bytes, int32_t* err_flag, void* stream) {
  if (n_tokens < 0 || n_q_heads < 1 || n_req < 0 || max_new < 0 || !scores) return HC_ERR_INVALID_ARG;
  const int st = check_pages(desc, k_pages, v_pages);
  if (st != HC_OK) return st;
  if (desc->dtype == HC_F32) return HC_ERR_UNSUPPORTED;
  const int es = elem_size(desc->dtype), H = desc->n_kv_heads, d = desc->d_head;
  if (n_q_heads % H) return HC_ERR_INVALID_ARG;
  if (!rows_ok(q, es, n_tokens > 0) || !rows_ok(out, es, n_tokens > 0) || !err_flag || !aligned(err_flag, 4) ||
      !aligned(lse, 4))
    return HC_ERR_INVALID_ARG;
  if (!rows16(*q, es, n_tokens, n_q_heads) || !rows16(*out, es, n_tokens, n_q_heads)) return HC_ERR_INVALID_ARG;
  if (!rows_apart(*out, n_tokens, n_q_heads, d)) return HC_ERR_INVALID_ARG;
  if (!q_starts || !aligned(q_starts, 4) || (n_req > 0 && (!kv_lens || !aligned(kv_lens, 4)))) return HC_ERR_INVALID_ARG;
  const int log2 = block_log2(desc->block_size);
  if (!table_ok(block_tables, table_stride, table_width, n_req, log2)) return HC_ERR_INVALID_ARG;
  if ((scores->causal != 0 && scores->causal != 1) || scores->window < 0) return HC_ERR_INVALID_ARG;
  if (!scores->causal && (scores->window > 0 || scores->prefix_lens)) return HC_ERR_INVALID_ARG;
  const float scale_log2 = scores->softmax_scale * 1.4426950408889634f;
  if (!std::isfinite(scale_log2)) return HC_ERR_INVALID_ARG;
  const float cap = scores->softcap, cap_log2 = cap * 1.4426950408889634f;
  const float cap_in = cap > 0.f ? scores->softmax_scale / cap : 0.f;
  if (!(cap >= 0.f) || !std::isfinite(cap_log2) || (cap > 0.f && cap_log2 == 0.f) || !std::isfinite(cap_in))
    return HC_ERR_INVALID_ARG;
  if (!aligned(scores->slopes, 4) || !aligned(scores->positions, 4) || !aligned(scores->prefix_lens, 4))
    return HC_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < workspace_bytes_needed())
    return HC_ERR_INVALID_ARG;
  const int G = n_q_heads / H;
  // rows of a request, pieces of 8 rows times tiles of 64 keys, and tiles of 256 rows are counted in 32 bits
  if (int64_t{max_new} * G >= (int64_t{1} << 30)) return HC_ERR_INVALID_ARG;
  const int rows_above = n_req > 0 ? rows_for_pieces(n_req, H, d, int64_t{table_width} << log2) : 0;
  const int64_t pieces = (std::min<int64_t>(int64_t{max_new} * G, rows_above) + 7) / 8;
  const int64_t tiles = ((int64_t{table_width} << log2) + 63) / 64 + 3;
  const double runs = static_cast<double>((int64_t{max_new} * G + 255) / 256);
  if (static_cast<double>(n_req) * static_cast<double>(pieces * tiles) >= 0x1p31 ||
      static_cast<double>(n_req) * H * runs >= 0x1p30)
    return HC_ERR_INVALID_ARG;
  if (n_tokens == 0 || n_req == 0 || max_new == 0) return HC_OK;
  hc::AttendPagedParams p;
  p.q = q->ptr;
  p.out = out->ptr;
  p.lse = lse;
  p.q_token = q->token_stride;
  p.q_head = q->head_stride;
  p.o_token = out->token_stride;
  p.o_head = out->head_stride;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.slot_stride = desc->slot_stride;
  p.tables = block_tables;
  p.table_stride = table_stride;
  p.q_starts = q_starts;
  p.kv_lens = kv_lens;
  p.positions = scores->positions;
  p.prefix_lens = scores->prefix_lens;
  p.slopes = scores->slopes;
  p.n_req = n_req;
  p.n_tokens = n_tokens;
  p.max_new = max_new;
  p.table_width = table_width;
  p.most_keys = static_cast<int32_t>(std::min(int64_t{table_width} << log2, hc::kMostKeys));
  p.num_slots = desc->num_slots;
  p.H = H;
  p.G = G;
  p.B_log2 = log2;
  p.bf16 = desc->dtype == HC_BF16;
  p.causal = scores->causal;
  p.window = scores->window;
  p.by_group = hc::FastDivmod(static_cast<uint32_t>(G));
  p.by_heads = hc::FastDivmod(static_cast<uint32_t>(H));
  p.scale_log2 = scale_log2;
  p.cap_in = cap_in;
  p.cap_log2 = cap_log2;
  p.out32 = aligned(out->ptr, 32) && out->token_stride % 16 == 0 && out->head_stride % 16 == 0;
  p.workspace = static_cast<uint8_t*>(workspace);
  p.tiles_taken = reinterpret_cast<int32_t*>(p.workspace + workspace_bytes_needed() - kTileCounters);
  p.part_sums = p.workspace + hc::attend_paged_counter_bytes();
  p.part_bytes = part_bytes();
  p.err = err_flag;
  p.rows_above = rows_above;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (int64_t{max_new} * G > p.rows_above) {
    const int t = hc::record_cuda(d == 64 ? hc::launch_attend_paged_tiles_64(p, s) : hc::launch_attend_paged_tiles_128(p, s));
    if (t != HC_OK) return t;
  }
  return hc::record_cuda(hc::launch_attend_paged_rows(d, p, s));
}

int hc_merge_attention(const hc_rows* out_a, const float* lse_a, const hc_rows* out_b, const float* lse_b,
                       const hc_rows* out, float* lse, int32_t dtype, int32_t n_tokens, int32_t n_heads, int32_t d_head,
                       void* stream) {
  const int es = elem_size(dtype);
  if (es == 0 || n_tokens < 0 || n_heads < 0 || d_head < 1) return HC_ERR_INVALID_ARG;
  if (d_head != 64 && d_head != 128) return HC_ERR_UNSUPPORTED;
  const bool any = n_tokens > 0 && n_heads > 0;
  for (const hc_rows* r : {out_a, out_b, out})
    if (!rows_ok(r, es, any) || !rows16(*r, es, n_tokens, n_heads)) return HC_ERR_INVALID_ARG;
  if (!rows_apart(*out, n_tokens, n_heads, d_head)) return HC_ERR_INVALID_ARG;
  if (((!lse_a || !lse_b) && any) || !aligned(lse_a, 4) || !aligned(lse_b, 4) || !aligned(lse, 4))
    return HC_ERR_INVALID_ARG;
  // pieces of 16 bytes are counted in 32 bits
  if (int64_t{n_tokens} * n_heads >= (int64_t{1} << 31) / (d_head * es / 16) - 1024) return HC_ERR_INVALID_ARG;
  if (!any) return HC_OK;
  hc::MergeParams p;
  p.a = out_a->ptr;
  p.b = out_b->ptr;
  p.out = out->ptr;
  p.lse_a = lse_a;
  p.lse_b = lse_b;
  p.lse = lse;
  p.a_token = out_a->token_stride;
  p.a_head = out_a->head_stride;
  p.b_token = out_b->token_stride;
  p.b_head = out_b->head_stride;
  p.o_token = out->token_stride;
  p.o_head = out->head_stride;
  p.n_tokens = n_tokens;
  p.n_heads = n_heads;
  p.d = d_head;
  p.by_heads = hc::FastDivmod(static_cast<uint32_t>(n_heads));
  return hc::record_cuda(hc::launch_merge(dtype, p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
