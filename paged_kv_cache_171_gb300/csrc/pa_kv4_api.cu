// pa_kv4_api.cu -- the C ABI of the rotated appends and of the 4-bit cache:
// argument validation and dispatch.
#include "pa_kv4.cuh"

using namespace pa;

namespace {

// check_common, and heads whose blocks and rows keep within 32 bits.
int check_heads(int n_q_heads, int n_kv_heads, int head_dim, int page_size, int batch,
                int max_blocks, int num_pages, int dtype) {
  const int rc = check_common(n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks,
                              num_pages, dtype);
  return rc ? rc : n_q_heads > 65535 ? PA_ERR_HEADS : PA_OK;
}

// A chunk's rows a kv head, and the (256 rows, 128 keys) tiles of one, in 32 bits.
int check_chunk(int n_new, int n_q_heads, int n_kv_heads, int max_blocks, int page_size) {
  const int64_t tokens = static_cast<int64_t>(max_blocks) * page_size;
  if (n_new > tokens) return PA_ERR_SHAPE;
  const int64_t rows = static_cast<int64_t>(n_new) * (n_q_heads / n_kv_heads);
  return rows >= (int64_t(1) << 30) || (rows / 256 + 1) * (tokens / 128 + 16) >= (int64_t(1) << 31)
             ? PA_ERR_SHAPE
             : PA_OK;
}

int check_append(const AppendRopeLaunch &a, int page_size, int dtype) {
  const int rc = check_heads(a.q ? a.n_q_heads : a.n_kv_heads, a.n_kv_heads, a.head_dim,
                             page_size, a.batch, a.max_blocks, a.num_pages, dtype);
  if (rc) return rc;
  if (a.n_tok < 0) return PA_ERR_SHAPE;
  if (a.cos_sin && (a.rot_dim < 16 || a.rot_dim > a.head_dim || a.rot_dim % 16 || a.max_pos <= 0))
    return PA_ERR_ROPE;
  const int64_t kv = static_cast<int64_t>(a.n_kv_heads) * a.head_dim;
  if (a.k_stride < kv || a.v_stride < kv ||
      (a.q && a.q_stride < static_cast<int64_t>(a.n_q_heads) * a.head_dim))
    return PA_ERR_SHAPE;
  if (a.k_stride % 8 || a.v_stride % 8 || (a.q && a.q_stride % 8)) return PA_ERR_ALIGN;
  if (!aligned16(a.k_new) || !aligned16(a.v_new) || !aligned16(a.q) || !aligned16(a.q_out) ||
      !aligned16(a.k_cache) || !aligned16(a.v_cache) || !aligned16(a.kv4_cache) ||
      !aligned16(a.cos_sin))
    return PA_ERR_ALIGN;
  return PA_OK;
}

int append(AppendRopeLaunch &a, int page_size, int dtype, pa_stream_t stream) {
  int rc = check_append(a, page_size, dtype);
  if (rc || a.n_tok == 0) return rc;
  if ((rc = current_status_ptr(&a.status))) return rc;
  a.bf16 = dtype == PA_BF16;
  return launch_append_rope(a, reinterpret_cast<cudaStream_t>(stream));
}

// Whether a chunk goes to the tile kernel: by its rows (queries x group) a kv head.
// The row kernel turns the codes once for 8 of them, the tile kernel once for 256, at
// the price of whole operand tiles; fp16's tile form is the slower one.  Rows against
// tiles in us, 8 kv heads, rows a kv head across:
//                                 8        16        24        32        64
//   bf16  4 x 32768, 128    52 /  84  85 /  85  119 /  85  153 /  85  290 /  86
//         4 x 32768, 64     35 /  67  56 /  68   77 /  68   98 /  68  184 /  68
//         16 x 2000, 128    21 /  33  32 /  35   40 /  35   49 /  35   86 /  38
//         16 x 2000, 64     15 /  27  22 /  28   28 /  28   33 /  28   56 /  29
//         8 x 700, 128      12 /  17  15 /  17   18 /  18   18 /  18   30 /  18
//         1 x 300, 128      10 /  12  11 /  12   11 /  12   11 /  13   11 /  14
//   fp16  4 x 32768, 128    51 / 124  85 / 125  118 / 126  152 / 126  288 / 127
//         4 x 32768, 64     35 /  98  56 /  98   76 /  99   98 /  99  184 /  99
//         16 x 2000, 128    21 /  44  32 /  45   40 /  45   49 /  45   86 /  46
//         16 x 2000, 64     15 /  35  22 /  35   28 /  35   33 /  36   56 /  36
//         8 x 700, 128      12 /  21  15 /  21   18 /  22   18 /  22   30 /  22
//         1 x 300, 128      10 /  12  10 /  13   11 /  13   10 /  14   11 /  15
// (Lengths are not known to the host: a short context may take 4 us more than it need.)
bool wants_tiles(int n_new, int n_q_heads, int n_kv_heads, bool bf16) {
  return n_new > 0 &&
         static_cast<int64_t>(n_new) * (n_q_heads / n_kv_heads) > (bf16 ? 16 : 24);
}

// The larger of the two kernels' workspaces where the type decides between them.
size_t chunk_workspace(int n_new, int n_q_heads, int n_kv_heads, int head_dim, int sms) {
  return wants_tiles(n_new, n_q_heads, n_kv_heads, true)
             ? kv4_tiles_workspace_bytes(head_dim, sms)
             : kv4_rows_workspace_bytes(head_dim, sms);
}

int sms_or_default() { return sm_count() > 0 ? sm_count() : 152; }

int attention(Kv4AttentionLaunch &a, int page_size, int dtype, size_t workspace_bytes,
              pa_stream_t stream) {
  if (!a.q || !a.cache || !a.block_table || !a.ctx_lens || !a.out) return PA_ERR_NULL;
  int rc = check_heads(a.n_q_heads, a.n_kv_heads, a.head_dim, page_size, a.batch, a.max_blocks,
                       a.num_pages, dtype);
  if (!rc) rc = check_chunk(a.n_new, a.n_q_heads, a.n_kv_heads, a.max_blocks, page_size);
  if (rc) return rc;
  if (!aligned16(a.q) || !aligned16(a.cache) || !aligned16(a.out)) return PA_ERR_ALIGN;
  const bool tiles = wants_tiles(a.n_new, a.n_q_heads, a.n_kv_heads, dtype == PA_BF16);
  const size_t need = chunk_workspace(a.n_new, a.n_q_heads, a.n_kv_heads, a.head_dim,
                                      sms_or_default());
  if (!a.workspace || workspace_bytes < need) return PA_ERR_WORKSPACE;
  if (!aligned16(a.workspace)) return PA_ERR_ALIGN;
  if ((rc = current_status_ptr(&a.status))) return rc;
  a.bf16 = dtype == PA_BF16;
  return tiles ? launch_kv4_tiles(a, reinterpret_cast<cudaStream_t>(stream))
               : launch_kv4_rows(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int pa_append_kv_rope(const void *k_new, const void *v_new, const void *q, void *k_cache,
                      void *v_cache, void *q_out, const int32_t *block_table,
                      const int32_t *seq_idx, const int32_t *pos, const float *cos_sin,
                      int n_tok, int64_t k_stride, int64_t v_stride, int64_t q_stride,
                      int n_q_heads, int n_kv_heads, int head_dim, int page_size, int batch,
                      int max_blocks_per_seq, int num_pages, int max_pos, int rot_dim,
                      int interleaved, pa_dtype dtype, pa_stream_t stream) {
  if (!k_new || !v_new || !k_cache || !v_cache || !block_table || !seq_idx || !pos || !cos_sin ||
      !q != !q_out)
    return PA_ERR_NULL;
  AppendRopeLaunch a = {k_new, v_new, q, q_out, k_cache, v_cache, nullptr, block_table, seq_idx,
                        pos, cos_sin, nullptr, k_stride, v_stride, q_stride, n_tok, n_q_heads,
                        n_kv_heads, head_dim, batch, max_blocks_per_seq, num_pages, max_pos,
                        rot_dim, interleaved != 0, false};
  return append(a, page_size, dtype, stream);
}

int pa_append_kv_rope_at(const void *k_new, const void *v_new, const void *q, void *k_cache,
                         void *v_cache, void *q_out, const int32_t *block_table,
                         const int32_t *seq_idx, const int32_t *pos, const int32_t *rope_pos,
                         const float *cos_sin, int n_tok, int64_t k_stride, int64_t v_stride,
                         int64_t q_stride, int n_q_heads, int n_kv_heads, int head_dim,
                         int page_size, int batch, int max_blocks_per_seq, int num_pages,
                         int max_pos, int rot_dim, int interleaved, pa_dtype dtype,
                         pa_stream_t stream) {
  if (!k_new || !v_new || !k_cache || !v_cache || !block_table || !seq_idx || !pos ||
      !rope_pos || !cos_sin || !q != !q_out)
    return PA_ERR_NULL;
  AppendRopeLaunch a = {k_new, v_new, q, q_out, k_cache, v_cache, nullptr, block_table, seq_idx,
                        pos, cos_sin, nullptr, k_stride, v_stride, q_stride, n_tok, n_q_heads,
                        n_kv_heads, head_dim, batch, max_blocks_per_seq, num_pages, max_pos,
                        rot_dim, interleaved != 0, false, rope_pos};
  return append(a, page_size, dtype, stream);
}

size_t pa_kv4_block_bytes(int head_dim) {
  return head_dim == 64 || head_dim == 128 ? kv4::block_bytes(head_dim) : 0;
}

int pa_append_kv4(const void *k_new, const void *v_new, const void *q, void *kv_cache,
                  void *q_out, const int32_t *block_table, const int32_t *seq_idx,
                  const int32_t *pos, const float *cos_sin, int n_tok, int64_t k_stride,
                  int64_t v_stride, int64_t q_stride, int n_q_heads, int n_kv_heads,
                  int head_dim, int page_size, int batch, int max_blocks_per_seq,
                  int num_pages, int max_pos, int rot_dim, int interleaved, pa_dtype dtype,
                  pa_stream_t stream) {
  if (!k_new || !v_new || !kv_cache || !block_table || !seq_idx || !pos || !q != !q_out)
    return PA_ERR_NULL;
  AppendRopeLaunch a = {k_new, v_new, q, q_out, nullptr, nullptr,
                        static_cast<uint8_t *>(kv_cache), block_table, seq_idx, pos, cos_sin,
                        nullptr, k_stride, v_stride, q_stride, n_tok, n_q_heads, n_kv_heads,
                        head_dim, batch, max_blocks_per_seq, num_pages, max_pos,
                        cos_sin ? rot_dim : 0, interleaved != 0, false};
  return append(a, page_size, dtype, stream);
}

int pa_read_kv4(const void *kv_cache, const int32_t *block_table, const int32_t *seq_idx,
                const int32_t *pos, void *k_out, void *v_out, int n_tok, int n_kv_heads,
                int head_dim, int page_size, int batch, int max_blocks_per_seq, int num_pages,
                pa_dtype dtype, pa_stream_t stream) {
  if (!kv_cache || !block_table || !seq_idx || !pos || !k_out || !v_out) return PA_ERR_NULL;
  int rc = check_heads(n_kv_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
                       num_pages, dtype);
  if (rc) return rc;
  if (n_tok < 0) return PA_ERR_SHAPE;
  if (!aligned16(kv_cache) || !aligned16(k_out) || !aligned16(v_out)) return PA_ERR_ALIGN;
  if (n_tok == 0) return PA_OK;
  ReadKv4Launch a = {static_cast<const uint8_t *>(kv_cache), block_table, seq_idx, pos, k_out,
                     v_out, nullptr, n_tok, n_kv_heads, head_dim, batch, max_blocks_per_seq,
                     num_pages, dtype == PA_BF16};
  if ((rc = current_status_ptr(&a.status))) return rc;
  return launch_read_kv4(a, reinterpret_cast<cudaStream_t>(stream));
}

int pa_copy_pages_kv4(void *kv_cache, const int32_t *src, const int32_t *dst, int n,
                      int n_kv_heads, int head_dim, int page_size, int num_pages,
                      pa_stream_t stream) {
  if (!kv_cache || !src || !dst) return PA_ERR_NULL;
  int rc = check_heads(n_kv_heads, n_kv_heads, head_dim, page_size, 1, 1, num_pages, PA_BF16);
  if (rc) return rc;
  if (n < 0) return PA_ERR_SHAPE;
  if (!aligned16(kv_cache)) return PA_ERR_ALIGN;
  if (n == 0) return PA_OK;
  int *status = nullptr;
  if ((rc = current_status_ptr(&status))) return rc;
  return launch_copy_pages_kv4(static_cast<uint8_t *>(kv_cache), src, dst, status, n, n_kv_heads,
                               head_dim, num_pages, reinterpret_cast<cudaStream_t>(stream));
}

size_t pa_decode_kv4_workspace_size(int head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return kv4_rows_workspace_bytes(head_dim, sms_or_default());
}

int pa_decode_kv4(const void *q, const void *kv_cache, const int32_t *block_table,
                  const int32_t *ctx_lens, float *out, float scale, int n_q_heads,
                  int n_kv_heads, int head_dim, int page_size, int batch,
                  int max_blocks_per_seq, int num_pages, pa_dtype dtype, void *workspace,
                  size_t workspace_bytes, pa_stream_t stream) {
  Kv4AttentionLaunch a = {q, static_cast<const uint8_t *>(kv_cache), block_table, ctx_lens, out,
                          workspace, nullptr, scale, 0, n_q_heads, n_kv_heads, head_dim, batch,
                          max_blocks_per_seq, num_pages, false};
  return attention(a, page_size, dtype, workspace_bytes, stream);
}

size_t pa_prefill_kv4_workspace_size(int batch, int n_new, int n_q_heads, int n_kv_heads,
                                     int head_dim, int page_size, int max_blocks_per_seq) {
  if (check_heads(n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq, 1,
                  PA_BF16) ||
      n_new <= 0 || check_chunk(n_new, n_q_heads, n_kv_heads, max_blocks_per_seq, page_size))
    return 0;
  return chunk_workspace(n_new, n_q_heads, n_kv_heads, head_dim, sms_or_default());
}

int pa_prefill_kv4(const void *q, const void *kv_cache, const int32_t *block_table,
                   const int32_t *ctx_lens, int n_new, void *out, float scale, int n_q_heads,
                   int n_kv_heads, int head_dim, int page_size, int batch,
                   int max_blocks_per_seq, int num_pages, pa_dtype dtype, void *workspace,
                   size_t workspace_bytes, pa_stream_t stream) {
  if (!q || !kv_cache || !block_table || !ctx_lens || !out) return PA_ERR_NULL;
  if (n_new < 0) return PA_ERR_SHAPE;
  Kv4AttentionLaunch a = {q, static_cast<const uint8_t *>(kv_cache), block_table, ctx_lens, out,
                          workspace, nullptr, scale, n_new, n_q_heads, n_kv_heads, head_dim,
                          batch, max_blocks_per_seq, num_pages, false};
  if (n_new == 0)  // nothing to compute; the other arguments are still checked
    return check_heads(n_q_heads, n_kv_heads, head_dim, page_size, batch, max_blocks_per_seq,
                       num_pages, dtype);
  return attention(a, page_size, dtype, workspace_bytes, stream);
}

}  // extern "C"
