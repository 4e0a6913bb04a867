// Declarations of the serving operators over the 16-bit paged buffer (append,
// attention, merge), shared by their kernels and the C ABI.
#pragma once

#include <algorithm>

#include "serve.cuh"

namespace hc {

struct AppendPagedParams {
  RopeParams rope;
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_pages;
  void* v_pages;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, o_token, o_head;
  int64_t slot_stride;  // elements
  int32_t n_tokens, n_q_heads, H, d, B_log2;
  int32_t heads_per_warp, q_parts, kv_parts, token_step;
  int32_t items, lanes_per_row;  // pieces of a row, and the lanes that take them
  FastDivmod parts;              // warps of a token
  const int64_t* token_rows;
  int64_t n_rows;  // num_slots * block_size
  int32_t* err;
};

struct AttendPagedParams {
  const void* q;
  void* out;
  float* lse;
  int64_t q_token, q_head, o_token, o_head;
  const void* k_pages;
  const void* v_pages;
  int64_t slot_stride;  // elements
  const int32_t* tables;
  int64_t table_stride;
  const int32_t* q_starts;
  const int32_t* kv_lens;
  const int32_t* positions;    // null: a request's queries are its last positions
  const int32_t* prefix_lens;  // null: none
  const float* slopes;         // null: none
  int32_t n_req, n_tokens, max_new, table_width, num_slots;
  int32_t H, G, B_log2, bf16, causal, window;
  FastDivmod by_group, by_heads;  // division by G, by H
  float scale_log2;     // softmax_scale * log2(e)
  float cap_in, cap_log2;  // softmax_scale / cap and cap * log2(e); cap_log2 0: no cap
  int32_t rows_above;   // requests with more query rows than this go to k_attend_paged_tiles
  int32_t piece_cost;   // of the rows kernel: what a piece's start and end take, in tiles
  int32_t out32;        // rows of out lie on 32-byte boundaries
  int32_t q_tma;        // of the tiles kernel: 128 rows of queries are a box of whole tokens
  uint64_t wait_limit;  // of the tiles kernel: ns
  uint8_t* workspace;
  int32_t* tiles_taken;  // in the workspace: works of the tiles kernel that are taken, CTAs that are done
  uint8_t* part_sums;    // in the workspace, where the rows kernel has its partial sums later
  int64_t part_bytes;
  int32_t split, part_rows;  // of the tiles kernel: parts of a run's tiles, rows of a part's sums
  int32_t* err;
};

struct MergeParams {
  const void* a;
  const void* b;
  void* out;
  const float* lse_a;
  const float* lse_b;
  float* lse;
  int64_t a_token, a_head, b_token, b_head, o_token, o_head;
  int32_t n_tokens, n_heads, d;
  FastDivmod by_heads;
};

// The rows kernel's workspace: bytes of its counters, one per CTA of the largest
// grid, and with the two partial results per CTA that follow.
int64_t attend_paged_counter_bytes();
int64_t attend_paged_rows_bytes();

// Parts that the tiles of a run of 256 rows are shared out in where a call has
// fewer runs than SMs, and the time of the slowest SM in tiles of 128 keys: a
// part's start and end take 3, the join of the parts 6.  At most `places` parts
// of all runs fit the workspace.
constexpr int kLeastPartTiles = 4;
struct Split {
  int parts;
  int64_t time;
};
inline Split split_tiles(int64_t runs, int64_t keys, int64_t places, int sms) {
  const int64_t tiles = std::max<int64_t>(1, (keys + 127) / 128), waves = (runs + sms - 1) / sms;
  Split best{1, waves * (tiles + 3)};
  if (runs >= sms) return best;
  const int64_t most = std::min((tiles + kLeastPartTiles - 1) / kLeastPartTiles, places / runs);
  for (int64_t w = 1; w <= 3; ++w) {  // as many parts as w of them an SM
    const int64_t n = std::min(most, w * sms / runs);
    if (n < 2) continue;
    const int64_t time = w * ((tiles + n - 1) / n + 3) + 6;
    if (time < best.time) best = {static_cast<int>(n), time};
  }
  return best;
}

cudaError_t launch_append_paged(int dtype, int pairing, const AppendPagedParams& p, cudaStream_t s);
// The requests with at most p.rows_above query rows, and those with more.
cudaError_t launch_attend_paged_rows(int d, const AttendPagedParams& p, cudaStream_t s);
cudaError_t launch_attend_paged_tiles(int d, const AttendPagedParams& p, cudaStream_t s);
cudaError_t launch_merge(int dtype, const MergeParams& p, cudaStream_t s);

}  // namespace hc
