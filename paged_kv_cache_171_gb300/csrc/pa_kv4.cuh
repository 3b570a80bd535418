// pa_kv4.cuh -- the 4-bit cache block: its layout, and the interfaces of the
// kernels that write and read it.
//
// A block holds one (page, kv head): the K and V rows of 16 tokens, each row
// as head_dim 4-bit codes with one 16-bit (scale, zero) pair,
//   x = zero + scale * (code - 8),            code = 0 .. 15,
// laid out as
//   [K, V][16 tokens][head_dim / 2] bytes of codes: dimension 2 i in the low
//       four bits of byte i, 2 i + 1 in the high four
//   [K, V][16 tokens][scale, zero] 16-bit floats of the cache's dtype.
// K and V of a page sit side by side, so a decode step fetches both with one
// bulk copy; at head_dim 128 a block is 2176 bytes (17 lines of 128), at 64
// 1152 (9 lines), 3.76 / 3.56 times less than in 16 bits.
//
// These kernels start while the kernel before them in the stream still runs, and wait for
// it before they read.  What a kernel before may write (the blocks, tables, lengths,
// angles) is therefore read by ordinary or L2 loads, never by ld.global.nc, which wants
// memory that stays as it is for the kernel's whole life.
#pragma once

#include "pa_internal.h"

namespace pa {
namespace kv4 {

// Bytes of one block, and of the codes of one row.
__host__ __device__ constexpr int block_bytes(int head_dim) { return 16 * head_dim + 128; }
__host__ __device__ constexpr int row_bytes(int head_dim) { return head_dim / 2; }
// Byte offsets inside a block: the codes of row `slot` of K (which = 0) or V
// (1), and its (scale, zero) pair.
__host__ __device__ constexpr int code_offset(int head_dim, int which, int slot) {
  return (which * kPageSize + slot) * row_bytes(head_dim);
}
__host__ __device__ constexpr int meta_offset(int head_dim, int which, int slot) {
  return 16 * head_dim + (which * kPageSize + slot) * 4;
}

// a / b of numbers that are not negative; 64-bit division only where 32 bits do not hold them.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

}  // namespace kv4

// The rows of an append: token j's K row of head g is k_new[j * k_stride + g *
// head_dim ..], likewise V and q.
struct AppendRopeLaunch {
  const void *k_new, *v_new, *q;  // q may be null
  void *q_out;
  void *k_cache, *v_cache;        // 16-bit cache, or null
  uint8_t *kv4_cache;             // 4-bit cache, or null
  const int32_t *block_table, *seq_idx, *pos;
  const float *cos_sin;           // [max_pos][rot_dim]; null: no rotation
  int *status;
  int64_t k_stride, v_stride, q_stride;
  int n_tok, n_q_heads, n_kv_heads, head_dim, batch, max_blocks, num_pages;
  int max_pos, rot_dim;
  bool interleaved, bf16;
};
int launch_append_rope(const AppendRopeLaunch &a, cudaStream_t stream);

struct ReadKv4Launch {
  const uint8_t *cache;
  const int32_t *block_table, *seq_idx, *pos;
  void *k_out, *v_out;
  int *status;
  int n_tok, n_kv_heads, head_dim, batch, max_blocks, num_pages;
  bool bf16;
};
int launch_read_kv4(const ReadKv4Launch &a, cudaStream_t stream);

int launch_copy_pages_kv4(uint8_t *cache, const int32_t *src, const int32_t *dst, int *status,
                          int n, int n_kv_heads, int head_dim, int num_pages,
                          cudaStream_t stream);

// Attention over the 4-bit cache.  n_new = 0: decode, one query a sequence
// that sees its ctx_lens[b] tokens, fp32 out.  n_new > 0: a chunk, query i
// sees ctx_lens[b] + i + 1 tokens, 16-bit out.
struct Kv4AttentionLaunch {
  const void *q;
  const uint8_t *cache;
  const int32_t *block_table, *ctx_lens;
  void *out;
  void *workspace;
  int *status;
  float scale;
  int n_new, n_q_heads, n_kv_heads, head_dim, batch, max_blocks, num_pages;
  bool bf16;
};
// Workspace of the row kernel on a device of `sms` SMs.
size_t kv4_rows_workspace_bytes(int head_dim, int sms);
int launch_kv4_rows(const Kv4AttentionLaunch &a, cudaStream_t stream);
// The tile kernel (tcgen05): chunks of many rows.
size_t kv4_tiles_workspace_bytes(int head_dim, int sms);
int launch_kv4_tiles(const Kv4AttentionLaunch &a, cudaStream_t stream);

}  // namespace pa
