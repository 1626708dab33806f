// Internal host interface of the paged-cache operators (fa_cache_api.cu checks the
// arguments, the launchers below run them).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "fa.h"

namespace fa {

struct PlanArgs {
  int B, rows, max_new, page_shift, num_pages, max_pages, words;
  const int32_t* ctx_len;
  const int32_t* cu_new;
  const int32_t* parent;
  int32_t* block_table;
  int32_t* n_pages;
  int32_t* free_list;
  int32_t* free_count;
  int32_t* seq_len;
  int32_t* slot;
  int32_t* position;
  unsigned long long* tree_mask;
};

// One group of heads a rotary launch moves: `heads` rows of d elements per token.
struct RopePart {
  const uint16_t* src;
  uint16_t* dst;
  long long src_b, src_h, src_n;
  long long dst_b, dst_h, dst_n;  // to_cache: dst_b is the page stride, dst_n that of a row in its page
  int heads;
  int rotate;
  int to_cache;
};

struct RopeArgs {
  RopePart part[3];
  int n_parts;
  int bf16;
  int B, N, d, rot, n_axes, inverse, pairs;
  const int32_t* positions;
  long long pos_axis, pos_b;
  const float* inv_freq;
  const uint8_t* axis;
  const int32_t* slot;  // to_cache parts: cache row of token b * N + n
  int page_shift;
  long long cache_rows;
};

struct CommitArgs {
  uint16_t* k;
  uint16_t* v;
  long long page_stride, head_stride, row_stride;
  int num_pages, page_shift, H_kv, d, B, max_pages, max_accept;
  const int32_t* block_table;
  const int32_t* ctx_len;
  const int32_t* accepted;
  const int32_t* n_accepted;
  int32_t* new_len;
};

struct TreeArgs {
  fa_kv_cache cache;
  fa_rows q, o;
  float* lse;
  int B, rows, max_q, Hq, max_pages, page_shift, words;
  const int32_t* block_table;
  const int32_t* cu_q;
  const int32_t* seq_len;
  const unsigned long long* tree_mask;
  float scale;
  void* workspace;
  int* status;
  uint64_t timeout_ns = 2000000000ull;  // limit of every device-side wait
  int withhold = 0;                     // debug: the producers issue no load
};

// Limits of the ragged batch and of a drafted tree.
constexpr int kCacheMaxB = 4096;

// Return 0 on success, a cudaError_t value otherwise.
int launch_cache_plan(const PlanArgs& a, cudaStream_t stream);
int launch_rope(const RopeArgs& a, cudaStream_t stream);
int launch_cache_commit(const CommitArgs& a, cudaStream_t stream);
int launch_tree_fwd(const TreeArgs& a, cudaStream_t stream);
size_t tree_fwd_workspace(int B, int rows, int max_q, int Hq, int H_kv, int d);

}  // namespace fa
