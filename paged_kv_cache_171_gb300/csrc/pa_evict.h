// pa_evict.h -- host-side interfaces of the operators around eviction by gathered
// attention weight and of tree verification, between their C ABI (pa_evict_api.cu)
// and their kernels.
#pragma once

#include "pa_internal.h"

namespace pa {

inline int sms_or_default() { return sm_count() > 0 ? sm_count() : 152; }

// Decode that also gathers attention weight (pa_weighted.cu).
struct WeightedLaunch {
  const void *q, *k_cache, *v_cache;
  float *weights;
  const int32_t *block_table, *ctx_lens;
  float *out;
  void *workspace;
  int *status;
  float scale;
  int n_q_heads, n_kv_heads, head_dim, batch, max_blocks, num_pages, fresh;
  bool bf16;
};
size_t weighted_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int head_dim,
                                int max_blocks, int sms);
int launch_weighted(const WeightedLaunch &a, cudaStream_t stream);

// Gathered weight of a chunk's queries (pa_weights_tc.cu).  Strides in elements.
struct WeightsLaunch {
  const void *q, *k_cache;
  float *weights;
  const int32_t *block_table, *ctx_lens;
  void *workspace;
  int *status;
  float scale;
  int64_t q_batch_stride, q_token_stride;
  int n_new, n_q_heads, n_kv_heads, head_dim, batch, max_blocks, num_pages, fresh;
  bool bf16;
};
size_t weights_workspace_bytes(int batch, int n_new, int n_q_heads, int n_kv_heads,
                               int max_blocks, int sms);
int launch_weights(const WeightsLaunch &a, cudaStream_t stream);

// Eviction and compaction (pa_evict.cu).  A move takes, for every sequence and kv head,
// row first + src[j] to position first + j of dst_table, j < n; src ascending.
struct EvictLaunch {
  void *k_cache, *v_cache;
  float *weights;  // null: none to move (compaction only)
  const int32_t *block_table, *ctx_lens, *dst_table;
  int32_t *new_lens;
  void *workspace;
  int *status;
  int n_kv_heads, head_dim, batch, max_blocks, dst_blocks, num_pages;
  // eviction
  int budget, sink, recent;
  // compaction: [batch][max_keep] and [batch]
  const int32_t *keep, *n_keep;
  int max_keep;
};
size_t evict_workspace_bytes(int batch, int n_kv_heads, int max_blocks, int budget);
int launch_evict(const EvictLaunch &a, cudaStream_t stream);
int launch_compact(const EvictLaunch &a, cudaStream_t stream);

// Attention of a tree of drafted tokens (pa_tree.cu).
struct TreeLaunch {
  const void *q, *k_cache, *v_cache;
  const int32_t *block_table, *ctx_lens;
  const uint32_t *mask;
  void *out, *workspace;
  int *status;
  float scale;
  int n_new, n_q_heads, n_kv_heads, head_dim, batch, max_blocks, num_pages;
  bool bf16;
};
size_t tree_workspace_bytes(int batch, int n_new, int n_q_heads, int n_kv_heads, int head_dim,
                            int max_blocks, int sms);
int launch_tree(const TreeLaunch &a, cudaStream_t stream);
int launch_tree_mask(const int32_t *parents, uint32_t *mask, int32_t *depth, int *status, int batch,
                     int n_new, cudaStream_t stream);

}  // namespace pa
