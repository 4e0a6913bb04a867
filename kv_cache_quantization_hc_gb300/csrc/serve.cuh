// Declarations of the serving operators over a 4-bit cache (block tables,
// rotary positions with several axes, append, attention), shared by their
// kernels and the C ABI.
#pragma once

#include <atomic>

#include "hc_internal.cuh"

namespace hc {

// What a launch needs to know of a kernel and its device, asked once per
// process and device (a query costs about as much host time as a launch).
struct KernelOnDevice {
  static constexpr int kDevices = 32;
  std::atomic<int> grid[kDevices] = {};  // CTAs that are resident at once; 0: not asked yet

  // Lets `f` use `smem` bytes of dynamic shared memory on the current device
  // and gives the number of its CTAs that the device holds at once.
  cudaError_t resident(const void* f, int threads, int smem, int* ctas) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool kept = dev >= 0 && dev < kDevices;
    if (kept && (*ctas = grid[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, f, threads, smem);
    if (e != cudaSuccess) return e;
    *ctas = device_sm_count() * (per_sm > 0 ? per_sm : 1);
    if (kept) grid[dev].store(*ctas, std::memory_order_relaxed);
    return cudaSuccess;
  }
};

// Status of a call from its launch's error, with the text kept for
// hc_last_cuda_error (api.cu).
int record_cuda(cudaError_t e);

struct BlockTableParams {
  const int32_t* cached;
  const int32_t* fresh;
  const int32_t* free_slots;
  int32_t* tables;
  int64_t table_stride;
  int32_t n_req, n_free, table_width, n_tokens, block_log2;
  int32_t* q_starts;
  int32_t* kv_lens;
  int32_t* token_req;
  int32_t* token_pos;
  int64_t* token_rows;
  int32_t* n_taken;
  int32_t* err;
  int32_t vec;  // the token arrays take 16-byte stores
};

// Rotation of rows by positions with several axes; see hc_rope_axes_desc.
struct RopeParams {
  const int32_t* positions;
  int64_t position_stride;
  const float2* table;  // null: no rotation
  int32_t n_positions, half, inverse;
  uint32_t axes;        // bit a: some pair has axis a
  int32_t pairs16;      // two pairs of the table make an aligned 16-byte word
  alignas(16) uint8_t pair_axis[128];
};

struct RopeAxesParams {
  RopeParams rope;
  const void* x;
  void* y;
  int64_t x_token, x_head, y_token, y_head;
  int32_t n_tokens, n_heads, d, heads_per_warp;
  FastDivmod parts, items_per_row;  // warps of a token; pieces of a row
  int32_t* err;
};

struct AppendParams {
  RopeParams rope;
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, o_token, o_head;
  int32_t n_tokens, n_q_heads, H, B_log2, group_log2, scale_f16, wire_scales;
  int32_t q_heads_per_warp, q_parts, kv_parts;
  FastDivmod parts, items_per_row;  // warps of a token; pieces of a row
  const int64_t* token_rows;
  int64_t n_rows;  // num_slots * block_size
  uint8_t* codes;
  void* scales;
  int32_t* err;
};

struct AttendParams {
  const void* q;
  void* out;
  float* lse;
  int64_t q_token, q_head, o_token, o_head;
  const uint8_t* codes;
  const void* scales;
  const int32_t* tables;
  int64_t table_stride;
  const int32_t* q_starts;
  const int32_t* kv_lens;
  int32_t n_req, n_tokens, max_new, table_width, num_slots;
  int32_t H, G, B_log2, bf16, causal, window;
  FastDivmod by_group;  // division by G
  float scale_log2;     // softmax_scale * log2(e)
  int32_t rows_above;   // requests with more query rows than this go to k_attend_tiles
  int32_t piece_cost;  // of the rows kernel: what a piece's start and end take, in tiles
  uint8_t* workspace;
  int32_t* err;
};

// Bytes of the attention's workspace: one counter per CTA of the largest
// grid, then two partial results per CTA.
int64_t attend_workspace_bytes();

cudaError_t launch_block_tables(const BlockTableParams& p, cudaStream_t s);
// `pieces16`: rows move in 16-byte pieces; element by element otherwise.
cudaError_t launch_rope_axes(int dtype, int pairing, bool pieces16, const RopeAxesParams& p,
                             cudaStream_t s);
cudaError_t launch_append_int4(int dtype, int d, int pairing, const AppendParams& p,
                               cudaStream_t s);
// The requests with at most p.rows_above query rows, and those with more.
cudaError_t launch_attend_rows(int d, int group, bool scale_f16, const AttendParams& p,
                               cudaStream_t s);
cudaError_t launch_attend_tiles(int d, int group, bool scale_f16, const AttendParams& p,
                                cudaStream_t s);

}  // namespace hc
