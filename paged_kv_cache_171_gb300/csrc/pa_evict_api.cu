// pa_evict_api.cu -- the C ABI of eviction by gathered attention weight and of tree
// verification: argument validation and dispatch.
#include "pa_evict.h"

using namespace pa;

namespace {

// check_common, and grids that take a CTA or more a (sequence, kv head) in 32 bits.
int check_lists(int n_q_heads, int n_kv_heads, int head_dim, int page_size, int batch,
                int max_blocks, int num_pages, int dtype) {
  const int rc = check_common(n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks,
                              num_pages, dtype);
  if (rc) return rc;
  if (n_q_heads > 65535) return PA_ERR_HEADS;
  return static_cast<int64_t>(batch) * n_kv_heads >= (int64_t(1) << 24) ? PA_ERR_SHAPE : PA_OK;
}

// Whether two device arrays of n and m 32-bit words have one in common.
bool overlap(const void *a, int64_t n, const void *b, int64_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return n > 0 && m > 0 && x < y + 4 * m && y < x + 4 * n;
}

constexpr int kMaxGroup = 1024;  // rows whose (m, 1 / l) shared memory holds

int check_weighted(int n_q_heads, int n_kv_heads, int head_dim, int page_size, int batch,
                   int max_blocks, int num_pages, int dtype) {
  const int rc = check_lists(n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks,
                             num_pages, dtype);
  if (rc) return rc;
  if (n_q_heads / n_kv_heads > kMaxGroup) return PA_ERR_HEADS;
  // CTAs of the second kernel, and items, in 32 bits
  return static_cast<int64_t>(batch) * n_q_heads >= (int64_t(1) << 30) ? PA_ERR_SHAPE : PA_OK;
}

// A chunk's rows a kv head and its CTAs in 32 bits.
int check_chunk(int n_new, int n_q_heads, int n_kv_heads, int batch, int max_blocks,
                int page_size) {
  const int64_t tokens = static_cast<int64_t>(max_blocks) * page_size;
  if (n_new < 0 || n_new > tokens) return PA_ERR_SHAPE;
  const int64_t rows = static_cast<int64_t>(n_new) * (n_q_heads / n_kv_heads);
  const int64_t lists = static_cast<int64_t>(batch) * n_kv_heads;
  return rows >= (int64_t(1) << 30) || lists * (rows / 128 + 1) >= (int64_t(1) << 30) ||
                 lists * (tokens / 128 + 1) >= (int64_t(1) << 31)
             ? PA_ERR_SHAPE : PA_OK;
}

}  // namespace

extern "C" {

size_t pa_decode_weighted_workspace_size(int batch, int n_q_heads, int n_kv_heads, int head_dim,
                                         int page_size, int max_blocks_per_seq) {
  if (check_weighted(n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq, 1,
                     PA_BF16))
    return 0;
  return weighted_workspace_bytes(batch, n_q_heads, n_kv_heads, head_dim, max_blocks_per_seq,
                                  sms_or_default());
}

int pa_decode_weighted(const void *q, const void *k_cache, const void *v_cache, float *weights,
                       const int32_t *block_table, const int32_t *ctx_lens, float *out,
                       float scale, int fresh, int n_q_heads, int n_kv_heads, int head_dim,
                       int page_size, int batch, int max_blocks_per_seq, int num_pages,
                       pa_dtype dtype, void *workspace, size_t workspace_bytes,
                       pa_stream_t stream) {
  if (!q || !k_cache || !v_cache || !weights || !block_table || !ctx_lens || !out)
    return PA_ERR_NULL;
  int rc = check_weighted(n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
                          num_pages, dtype);
  if (rc) return rc;
  if (fresh < 0) return PA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(weights) ||
      !aligned16(out))
    return PA_ERR_ALIGN;
  if (!workspace ||
      workspace_bytes < weighted_workspace_bytes(batch, n_q_heads, n_kv_heads, head_dim,
                                                 max_blocks_per_seq, sms_or_default()))
    return PA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return PA_ERR_ALIGN;
  WeightedLaunch a;
  if ((rc = current_status_ptr(&a.status))) return rc;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.weights = weights;
  a.block_table = block_table;
  a.ctx_lens = ctx_lens;
  a.out = out;
  a.workspace = workspace;
  a.scale = scale;
  a.n_q_heads = n_q_heads;
  a.n_kv_heads = n_kv_heads;
  a.head_dim = head_dim;
  a.batch = batch;
  a.max_blocks = max_blocks_per_seq;
  a.num_pages = num_pages;
  a.fresh = fresh;
  a.bf16 = dtype == PA_BF16;
  return launch_weighted(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t pa_evict_kv_workspace_size(int batch, int n_kv_heads, int head_dim, int page_size,
                                  int max_blocks_per_seq, int budget) {
  if (check_lists(n_kv_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq, 1,
                  PA_BF16) ||
      budget < 0)
    return 0;
  return evict_workspace_bytes(batch, n_kv_heads, max_blocks_per_seq, budget);
}

int pa_evict_kv(void *k_cache, void *v_cache, float *weights, const int32_t *block_table,
                const int32_t *ctx_lens, const int32_t *dst_table, int32_t *new_lens, int budget,
                int sink_tokens, int recent_tokens, int n_kv_heads, int head_dim, int page_size,
                int batch, int max_blocks_per_seq, int dst_blocks_per_seq, int num_pages,
                pa_dtype dtype, void *workspace, size_t workspace_bytes, pa_stream_t stream) {
  if (!k_cache || !v_cache || !weights || !block_table || !ctx_lens || !dst_table || !new_lens)
    return PA_ERR_NULL;
  int rc = check_lists(n_kv_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
                       num_pages, dtype);
  if (rc) return rc;
  if (budget < 0 || sink_tokens < 0 || recent_tokens < 0 ||
      static_cast<int64_t>(sink_tokens) + recent_tokens > budget)
    return PA_ERR_SHAPE;
  if (dst_blocks_per_seq <= 0 ||
      static_cast<int64_t>(dst_blocks_per_seq) * page_size > (int64_t(1) << 30))
    return PA_ERR_SHAPE;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(weights)) return PA_ERR_ALIGN;
  // read by some CTAs while another writes the new lengths
  if (overlap(new_lens, batch, ctx_lens, batch) ||
      overlap(new_lens, batch, block_table, int64_t(batch) * max_blocks_per_seq) ||
      overlap(new_lens, batch, dst_table, int64_t(batch) * dst_blocks_per_seq))
    return PA_ERR_SHAPE;
  if (!workspace ||
      workspace_bytes < evict_workspace_bytes(batch, n_kv_heads, max_blocks_per_seq, budget))
    return PA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return PA_ERR_ALIGN;
  EvictLaunch a = {};
  if ((rc = current_status_ptr(&a.status))) return rc;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.weights = weights;
  a.block_table = block_table;
  a.ctx_lens = ctx_lens;
  a.dst_table = dst_table;
  a.new_lens = new_lens;
  a.workspace = workspace;
  a.n_kv_heads = n_kv_heads;
  a.head_dim = head_dim;
  a.batch = batch;
  a.max_blocks = max_blocks_per_seq;
  a.dst_blocks = dst_blocks_per_seq;
  a.num_pages = num_pages;
  a.budget = budget;
  a.sink = sink_tokens;
  a.recent = recent_tokens;
  return launch_evict(a, reinterpret_cast<cudaStream_t>(stream));
}

int pa_compact_kv(void *k_cache, void *v_cache, float *weights, const int32_t *block_table,
                  const int32_t *ctx_lens, const int32_t *keep, const int32_t *n_keep,
                  int max_keep, int32_t *new_lens, int n_kv_heads, int head_dim, int page_size,
                  int batch, int max_blocks_per_seq, int num_pages, pa_dtype dtype,
                  pa_stream_t stream) {
  if (!k_cache || !v_cache || !block_table || !ctx_lens || !keep || !n_keep || !new_lens)
    return PA_ERR_NULL;
  int rc = check_lists(n_kv_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
                       num_pages, dtype);
  if (rc) return rc;
  if (max_keep < 0 || max_keep > max_blocks_per_seq * page_size) return PA_ERR_SHAPE;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(weights)) return PA_ERR_ALIGN;
  if (overlap(new_lens, batch, ctx_lens, batch) || overlap(new_lens, batch, n_keep, batch) ||
      overlap(new_lens, batch, keep, int64_t(batch) * max_keep) ||
      overlap(new_lens, batch, block_table, int64_t(batch) * max_blocks_per_seq))
    return PA_ERR_SHAPE;
  EvictLaunch a = {};
  if ((rc = current_status_ptr(&a.status))) return rc;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.weights = weights;
  a.block_table = a.dst_table = block_table;
  a.ctx_lens = ctx_lens;
  a.new_lens = new_lens;
  a.n_kv_heads = n_kv_heads;
  a.head_dim = head_dim;
  a.batch = batch;
  a.max_blocks = a.dst_blocks = max_blocks_per_seq;
  a.num_pages = num_pages;
  a.keep = keep;
  a.n_keep = n_keep;
  a.max_keep = max_keep;
  return launch_compact(a, reinterpret_cast<cudaStream_t>(stream));
}

size_t pa_prefill_weights_workspace_size(int batch, int n_new, int n_q_heads, int n_kv_heads,
                                         int head_dim, int page_size, int max_blocks_per_seq) {
  if (check_lists(n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq, 1,
                  PA_BF16) ||
      check_chunk(n_new, n_q_heads, n_kv_heads, batch, max_blocks_per_seq, page_size) ||
      n_new == 0)
    return 0;
  return weights_workspace_bytes(batch, n_new, n_q_heads, n_kv_heads, max_blocks_per_seq,
                                 sms_or_default());
}

int pa_prefill_weights(const void *q, const void *k_cache, float *weights,
                       const int32_t *block_table, const int32_t *ctx_lens, int n_new,
                       float scale, int fresh, int64_t q_batch_stride, int64_t q_token_stride,
                       int n_q_heads, int n_kv_heads, int head_dim, int page_size, int batch,
                       int max_blocks_per_seq, int num_pages, pa_dtype dtype, void *workspace,
                       size_t workspace_bytes, pa_stream_t stream) {
  if (!q || !k_cache || !weights || !block_table || !ctx_lens) return PA_ERR_NULL;
  int rc = check_lists(n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
                       num_pages, dtype);
  if (!rc)
    rc = check_chunk(n_new, n_q_heads, n_kv_heads, batch, max_blocks_per_seq, page_size);
  if (rc) return rc;
  if (fresh < 0) return PA_ERR_SHAPE;
  const int64_t row = static_cast<int64_t>(n_q_heads) * head_dim;
  if (q_token_stride < row || q_batch_stride < row || q_token_stride >= (int64_t(1) << 38) ||
      q_batch_stride >= (int64_t(1) << 38))
    return PA_ERR_SHAPE;
  if (q_token_stride % 8 || q_batch_stride % 8) return PA_ERR_ALIGN;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(weights)) return PA_ERR_ALIGN;
  if (n_new == 0) return PA_OK;
  if (!workspace ||
      workspace_bytes < weights_workspace_bytes(batch, n_new, n_q_heads, n_kv_heads,
                                                max_blocks_per_seq, sms_or_default()))
    return PA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return PA_ERR_ALIGN;
  WeightsLaunch a;
  if ((rc = current_status_ptr(&a.status))) return rc;
  a.q = q;
  a.k_cache = k_cache;
  a.weights = weights;
  a.block_table = block_table;
  a.ctx_lens = ctx_lens;
  a.workspace = workspace;
  a.scale = scale;
  a.q_batch_stride = q_batch_stride;
  a.q_token_stride = q_token_stride;
  a.n_new = n_new;
  a.n_q_heads = n_q_heads;
  a.n_kv_heads = n_kv_heads;
  a.head_dim = head_dim;
  a.batch = batch;
  a.max_blocks = max_blocks_per_seq;
  a.num_pages = num_pages;
  a.fresh = fresh;
  a.bf16 = dtype == PA_BF16;
  return launch_weights(a, reinterpret_cast<cudaStream_t>(stream));
}

int pa_tree_mask(const int32_t *parents, int32_t *mask, int32_t *depth, int batch, int n_new,
                 pa_stream_t stream) {
  if (!parents || !mask) return PA_ERR_NULL;
  if (batch <= 0 || batch > 65535 || n_new < 0 || n_new > (1 << 20)) return PA_ERR_SHAPE;
  if (n_new == 0) return PA_OK;
  int *status = nullptr;
  const int rc = current_status_ptr(&status);
  if (rc) return rc;
  return launch_tree_mask(parents, reinterpret_cast<uint32_t *>(mask), depth, status, batch,
                          n_new, reinterpret_cast<cudaStream_t>(stream));
}

size_t pa_prefill_tree_workspace_size(int batch, int n_new, int n_q_heads, int n_kv_heads,
                                      int head_dim, int page_size, int max_blocks_per_seq) {
  if (check_lists(n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq, 1,
                  PA_BF16) ||
      check_chunk(n_new, n_q_heads, n_kv_heads, batch, max_blocks_per_seq, page_size) ||
      n_new == 0)
    return 0;
  return tree_workspace_bytes(batch, n_new, n_q_heads, n_kv_heads, head_dim, max_blocks_per_seq,
                              sms_or_default());
}

int pa_prefill_tree(const void *q, const void *k_cache, const void *v_cache,
                    const int32_t *block_table, const int32_t *ctx_lens, const int32_t *mask,
                    int n_new, void *out, float scale, int n_q_heads, int n_kv_heads,
                    int head_dim, int page_size, int batch, int max_blocks_per_seq,
                    int num_pages, pa_dtype dtype, void *workspace, size_t workspace_bytes,
                    pa_stream_t stream) {
  if (!q || !k_cache || !v_cache || !block_table || !ctx_lens || !mask || !out)
    return PA_ERR_NULL;
  int rc = check_lists(n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
                       num_pages, dtype);
  if (!rc)
    rc = check_chunk(n_new, n_q_heads, n_kv_heads, batch, max_blocks_per_seq, page_size);
  if (rc) return rc;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
    return PA_ERR_ALIGN;
  if (n_new == 0) return PA_OK;
  const size_t need = tree_workspace_bytes(batch, n_new, n_q_heads, n_kv_heads, head_dim,
                                           max_blocks_per_seq, sms_or_default());
  if (need && (!workspace || workspace_bytes < need)) return PA_ERR_WORKSPACE;
  if (need && !aligned16(workspace)) return PA_ERR_ALIGN;
  TreeLaunch a;
  if ((rc = current_status_ptr(&a.status))) return rc;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.ctx_lens = ctx_lens;
  a.mask = reinterpret_cast<const uint32_t *>(mask);
  a.out = out;
  a.workspace = workspace;
  a.scale = scale;
  a.n_new = n_new;
  a.n_q_heads = n_q_heads;
  a.n_kv_heads = n_kv_heads;
  a.head_dim = head_dim;
  a.batch = batch;
  a.max_blocks = max_blocks_per_seq;
  a.num_pages = num_pages;
  a.bf16 = dtype == PA_BF16;
  return launch_tree(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
