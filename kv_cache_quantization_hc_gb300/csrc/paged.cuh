// Declarations of the serving operators over the 16-bit paged buffer (append,
// attention, merge), shared by their kernels and the C ABI.
#pragma once

#include <algorithm>
#include <cmath>

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

// How the tiles of runs of 256 rows are shared out over the SMs where a call has
// few runs: a run of n tiles (of 128 keys) is max(1, n / target) parts.  Decided
// by the kernel, which sees the lengths, and by the host as if they were even.
constexpr int kLeastPartTiles = 4;
struct SplitRule {
  float by_sms = 0.f, by_places = 0.f;  // reciprocals: of the SMs, of the parts that there may be beside one of each run
  // Of three choices, as many parts as 1, 2 or 3 an SM; all parts have a place.
  static constexpr int kChoices = 3;
  HC_HD int target(float total, int c) const {
    const float want = total * by_sms * (c == 0 ? 1.f : c == 1 ? 0.5f : 1.f / 3.f), fits = total * by_places;
    const float t = ceilf(want > fits ? want : fits);
    return t < kLeastPartTiles ? kLeastPartTiles : t > 0x1p30f ? 1 << 30 : static_cast<int>(t);
  }
  // The time of the slowest SM, in tiles, where they take `works` parts of at most `longest` tiles, `total` in all, as
  // they come: a part's start and end take 3.
  HC_HD float time(float works, float longest, float total) const {
    const float waves = ceilf(works * by_sms - 1e-3f) * (longest + 3.f), even = (total + 3.f * works) * by_sms + longest + 3.f;
    return works * by_sms <= 1.001f || waves < even ? waves : even;
  }
  static constexpr float kJoin = 6.f;  // the time of the join
};
// Whether a call's runs may be shared out: a warp goes through the requests
// several times, part sums have places, and the join is one wave of CTAs of 32 rows.
constexpr int kSplitRequests = 160, kSplitRuns = 2000;
inline bool split_rule(int64_t n_req, int64_t runs, int64_t keys, int64_t part_rows, int64_t places, int sms, SplitRule* rule) {
  rule->by_sms = 1.f / static_cast<float>(sms);
  if (n_req > kSplitRequests || keys <= 2 * kLeastPartTiles * 128 || places < runs + sms / 2 ||
      runs * (part_rows / 32) > int64_t{8} * sms || runs > kSplitRuns)
    return false;
  rule->by_places = 1.0001f / static_cast<float>(places - runs);
  return true;
}
// The time of `runs` runs of as many tiles each.
inline float even_time(int64_t n_req, int64_t runs, int64_t keys, int64_t part_rows, int64_t places, int sms) {
  SplitRule rule;
  const float n = static_cast<float>(runs), tiles = static_cast<float>(std::max<int64_t>(1, (keys + 127) / 128));
  const bool may = split_rule(n_req, runs, keys, part_rows, places, sms, &rule);
  float best = rule.time(n, tiles, n * tiles);
  for (int c = 0; may && c < SplitRule::kChoices; ++c) {
    const float parts = std::max(1.f, std::floor(tiles / static_cast<float>(rule.target(n * tiles, c))));
    if (parts > 1.f) best = std::min(best, rule.time(n * parts, std::ceil(tiles / parts), n * tiles) + SplitRule::kJoin);
  }
  return best;
}

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
  // in the workspace: works of the tiles kernel that are taken, CTAs that are done; runs to join, CTAs that are done
  int32_t* tiles_taken;
  uint8_t* part_sums;    // in the workspace, where the rows kernel has its partial sums later
  int64_t part_bytes;    // the list of runs to join is behind them
  int32_t part_rows;    // of the tiles kernel where runs may be shared out: rows of a part's sums
  SplitRule split;
  int32_t most_keys;    // of a request: what its table holds, kMostKeys at most (here it moves no other field: else 0.7% slower)
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

cudaError_t launch_append_paged(int dtype, int pairing, const AppendPagedParams& p, cudaStream_t s);
// The requests with at most p.rows_above query rows, and those with more.
cudaError_t launch_attend_paged_rows(int d, const AttendPagedParams& p, cudaStream_t s);
cudaError_t launch_attend_paged_tiles_64(const AttendPagedParams& p, cudaStream_t s);
cudaError_t launch_attend_paged_tiles_128(const AttendPagedParams& p, cudaStream_t s);
cudaError_t launch_merge(int dtype, const MergeParams& p, cudaStream_t s);

}  // namespace hc
