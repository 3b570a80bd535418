// pa_tree.cu -- attention of a tree of drafted tokens over the paged cache, and the masks of
// a tree.
//
// Drafted token i of sequence b lies in the cache at position ctx + i.  Its query sees the ctx
// cached tokens and the drafted ones whose bit its mask has (its ancestors and itself):
//   out_i = softmax over those of (q_i K^T scale) V
// The kernel is the chunked prefill's (pa_prefill_tc.cuh) with the rows of a kv head's group
// laid end to end and the mask's bits in place of the causal limit.  Few rows over long
// contexts: each sequence's keys are cut into equal ranges, whose states a second kernel
// merges.
//
// Bound: the MMAs, 4 D a row and key; two CTAs never share an SM, so the ranges fill one wave
// and no more (two or three waves of shorter ranges: 205 -> 216 us and up, for a start and
// a merge each).  4 x 64 drafted tokens of 64 heads over 32768: 217 us with new inputs each
// call, 1.27 PFLOP/s (203 with the same ones), the tensor pipe busy 65% of the cycles that a CTA
// runs and waiting for the softmax in the others.  16 x 60 of 32 heads over 500 to 8000: 100 us; equal parts of every sequence
// leave the CTAs of the longest one the last to end.
#include "pa_evict.h"
#include "pa_prefill_tc.cuh"

namespace pa {
namespace {

struct Plan {
  int rows, pairs, parts;
};
// One CTA an SM holds two row tiles (256 rows).  Fewer CTAs than SMs: as many key ranges as
// fit one wave.
Plan plan_of(int batch, int n_new, int n_q_heads, int n_kv_heads, int max_blocks, int sms) {
  Plan y;
  y.rows = n_new * (n_q_heads / n_kv_heads);
  y.pairs = (y.rows + 2 * kRows - 1) / (2 * kRows);
  const int64_t ctas = static_cast<int64_t>(batch) * n_kv_heads * y.pairs;
  const int64_t most = (static_cast<int64_t>(max_blocks) * kPageSize + 4 * kKeys - 1) /
                       (4 * kKeys);  // ranges of 4 tiles
  int64_t parts = sms / ctas;
  if (parts > most) parts = most;
  y.parts = static_cast<int>(parts < 1 ? 1 : parts);
  return y;
}

// One warp a row: its ranges' states folded, O / l written in 16 bits.
template <int D, bool BF16>
__global__ void __launch_bounds__(256)
    tree_merge_kernel(const float *states, const int32_t *ctx_lens, uint16_t *out, int64_t n_rows,
                      int rows_per_seq, int n_new, int max_tokens, int n_parts) {
  constexpr int E = D / 32;  // dimensions a lane
  griddep_release();
  griddep_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= n_rows) return;
  const int ctx = max(0, min(ctx_lens[row / rows_per_seq], max_tokens - n_new));
  const int tiles = (ctx + n_new + kKeys - 1) / kKeys;
  const int per = tree_part_tiles(ctx + n_new, n_parts);
  const int n = (tiles + per - 1) / per;  // ranges that hold keys
  const float *s = states + row * n_parts * (D + 4);
  float m = -INFINITY, l = 0.f;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, s[i * (D + 4) + D]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, x));
  const float ref = m == -INFINITY ? 0.f : m;  // a row that sees nothing
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float2 ml = *reinterpret_cast<const float2 *>(s + i * (D + 4) + D);
    const float f = ex2((ml.x - ref) * kLog2e);
    l = fmaf(f, ml.y, l);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(f, s[i * (D + 4) + lane * E + e], acc[e]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t h[E / 2];
#pragma unroll
  for (int e = 0; e < E; e += 2) h[e / 2] = pack2<BF16>(acc[e] * inv, acc[e + 1] * inv);
  uint32_t *dst = reinterpret_cast<uint32_t *>(out + row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = h[e];
}

// A thread a drafted token climbs to its root.  Ancestors come in falling order, so a word
// is written once, and those passed over are zero.
__global__ void __launch_bounds__(128)
    tree_mask_kernel(const int32_t *parents, uint32_t *mask, int32_t *depth, int *status,
                     int64_t total, int n_new, int words) {
  griddep_release();
  griddep_wait();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (at >= total) return;
  const int i = static_cast<int>(at % n_new);
  const int32_t *row = parents + (at - i);
  uint32_t *out = mask + at * words;
  for (int w = words - 1; w > i >> 5; --w) out[w] = 0;
  int j = i, w = i >> 5, up = -1;
  uint32_t bits = 0;
  while (j >= 0) {
    for (; w > j >> 5; --w) {
      out[w] = bits;
      bits = 0;
    }
    bits |= 1u << (j & 31);
    ++up;
    const int parent = row[j];
    if (parent >= j || parent < -1) {
      record_error(status, PA_ERR_BAD_INDEX);
      break;
    }
    j = parent;
  }
  for (; w >= 0; --w) {
    out[w] = bits;
    bits = 0;
  }
  if (depth) depth[at] = up;
}

// Whether `kern` is launched with the registers that its setmaxnreg split adds up to; of fewer
// its softmax warps would wait for ever.
template <class K>
bool launched_with(K *kern, int registers, ContextCache<bool> &known) {
  bool fits = false;
  if (known.get(current_context_id(), &fits)) return fits;
  cudaFuncAttributes attr;
  if (cudaFuncGetAttributes(&attr, kern) != cudaSuccess) return false;
  fits = attr.numRegs >= registers;
  known.put(current_context_id(), fits);
  return fits;
}

template <int D, bool BF16>
int launch_t(const TreeLaunch &a, cudaStream_t stream) {
  using L = TcSmem<D>;
  auto kern = prefill_tc_kernel<D, 1, BF16, true>;
  static ContextCache<bool> smem_set, regs_known;
  if (set_smem_limit(kern, L::kAlloc, smem_set) != PA_OK) return PA_ERR_CUDA;
  if (!launched_with(kern, kTreeRegs, regs_known)) return PA_ERR_CUDA;
  const int sms = sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  const Plan y = plan_of(a.batch, a.n_new, a.n_q_heads, a.n_kv_heads, a.max_blocks, sms);
  CUtensorMap kmap, vmap;
  const uint64_t rows = static_cast<uint64_t>(a.num_pages) * a.n_kv_heads * kPageSize;
  if (make_rows_map(&kmap, a.k_cache, rows, D, kPageSize) != PA_OK) return PA_ERR_CUDA;
  if (make_rows_map(&vmap, a.v_cache, rows, D, kPageSize) != PA_OK) return PA_ERR_CUDA;
  TcParams p = {};
  p.q = static_cast<const uint16_t *>(a.q);
  p.v_cache = static_cast<const uint16_t *>(a.v_cache);
  p.block_table = a.block_table;
  p.ctx_lens = a.ctx_lens;
  p.status = a.status;
  // a positive factor, as for a chunk (pa_prefill_tc.cu)
  p.qscale = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
  p.qsign = a.scale < 0.f ? 0x80008000u : 0u;
  p.n_new = y.rows;
  p.n_q_heads = a.n_q_heads;
  p.n_kv_heads = a.n_kv_heads;
  p.group = 1;
  p.batch = a.batch;
  p.max_blocks = a.max_blocks;
  p.num_pages = a.num_pages;
  p.ws = y.parts > 1 ? static_cast<float *>(a.workspace) : nullptr;
  p.n_parts = p.ws_slots = y.parts;
  p.shared_ctx = -1;
  p.mask = a.mask;
  p.out16 = static_cast<uint16_t *>(a.out);
  p.tree_n = a.n_new;
  p.tree_group = a.n_q_heads / a.n_kv_heads;
  p.mask_words = (a.n_new + 31) / 32;
  if (launch_pdl(kern, dim3(y.pairs * y.parts, a.n_kv_heads, a.batch), dim3(kThreads), L::kAlloc,
                 stream, kmap, vmap, p) != cudaSuccess)
    return PA_ERR_CUDA;
  if (y.parts == 1) return PA_OK;
  const int64_t n_rows = static_cast<int64_t>(a.batch) * a.n_new * a.n_q_heads;
  return launch_pdl(tree_merge_kernel<D, BF16>, dim3(static_cast<unsigned>((n_rows + 7) / 8)),
                    dim3(256), 0, stream, static_cast<const float *>(a.workspace), a.ctx_lens,
                    p.out16, n_rows, a.n_new * a.n_q_heads, a.n_new, a.max_blocks * kPageSize,
                    y.parts) == cudaSuccess
             ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

// Partial states [batch][n_new][query heads][ranges][D + 4].
size_t tree_workspace_bytes(int batch, int n_new, int n_q_heads, int n_kv_heads, int head_dim,
                            int max_blocks, int sms) {
  const Plan y = plan_of(batch, n_new, n_q_heads, n_kv_heads, max_blocks, sms);
  return y.parts > 1 ? static_cast<size_t>(batch) * n_new * n_q_heads * y.parts *
                           (head_dim + 4) * sizeof(float)
                     : 0;
}

int launch_tree(const TreeLaunch &a, cudaStream_t stream) {
  if (a.head_dim == 128)
    return a.bf16 ? launch_t<128, true>(a, stream) : launch_t<128, false>(a, stream);
  return a.bf16 ? launch_t<64, true>(a, stream) : launch_t<64, false>(a, stream);
}

int launch_tree_mask(const int32_t *parents, uint32_t *mask, int32_t *depth, int *status, int batch,
                     int n_new, cudaStream_t stream) {
  const int64_t total = static_cast<int64_t>(batch) * n_new;
  return launch_pdl(tree_mask_kernel, dim3(static_cast<unsigned>((total + 127) / 128)), dim3(128),
                    0, stream, parents, mask, depth, status, total, n_new,
                    (n_new + 31) / 32) == cudaSuccess
             ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
