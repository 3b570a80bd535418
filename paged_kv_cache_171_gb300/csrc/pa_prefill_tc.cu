// pa_prefill_tc.cu -- launches of the chunked-prefill kernel (pa_prefill_tc.cuh): causal
// chunks, key ranges with their merge, and shared keys.
#include "pa_prefill_tc.cuh"

namespace pa {
namespace {

template <int D, int GT, bool BF16>
int launch_tc_t(const PrefillLaunch &a, cudaStream_t stream) {
  using L = TcSmem<D>;
  auto kern = prefill_tc_kernel<D, GT, BF16, false>;
  static ContextCache<bool> smem_set;  // contexts where the limit is set
  if (set_smem_limit(kern, L::kAlloc, smem_set) != PA_OK) return PA_ERR_CUDA;
  CUtensorMap kmap, vmap;
  const uint64_t rows = static_cast<uint64_t>(a.num_pages) * a.n_kv_heads * 16;
  if (make_rows_map(&kmap, a.k_cache, rows, D, 16) != PA_OK) return PA_ERR_CUDA;
  if (make_rows_map(&vmap, a.v_cache, rows, D, 16) != PA_OK) return PA_ERR_CUDA;
  TcParams p = {};
  p.q = static_cast<const uint16_t *>(a.q);
  p.block_table = a.block_table;
  p.ctx_lens = a.ctx_lens;
  p.out = a.out;
  p.status = a.status;
  // The kernel takes the maximum of the raw scores, so it needs a positive
  // factor: a negative scale flips the sign of Q instead (exact in 16 bits),
  // and a zero scale becomes a factor small enough that every weight is 1.
  p.qscale = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
  p.qsign = a.scale < 0.f ? 0x80008000u : 0u;
  p.n_new = a.n_new;
  p.n_q_heads = a.n_q_heads;
  p.n_kv_heads = a.n_kv_heads;
  p.group = a.n_q_heads / a.n_kv_heads;
  p.batch = a.batch;
  p.max_blocks = a.max_blocks;
  p.num_pages = a.num_pages;
  p.ws = a.workspace;
  p.n_parts = a.n_parts > 1 ? a.n_parts : 1;
  p.part_tiles = a.n_parts > 1 ? a.part_tokens / kKeys : (a.max_blocks * 16 + kKeys - 1) / kKeys;
  p.ws_slots = a.ws_slots > 0 ? a.ws_slots : p.n_parts;
  p.shared_ctx = a.shared_ctx;
  constexpr int BQ = kRows / GT;
  const dim3 grid(((a.n_new + 2 * BQ - 1) / (2 * BQ)) * p.n_parts,
                  a.n_kv_heads * (p.group / GT), a.batch);
  if (launch_pdl(kern, grid, dim3(kThreads), L::kAlloc, stream, kmap, vmap, p) != cudaSuccess)
    return PA_ERR_CUDA;
  if (p.n_parts > 1 && a.merge)
    return launch_merge_rows(a.workspace, a.ctx_lens, a.out, a.status, a.batch, a.n_q_heads,
                             D, p.n_parts, a.part_tokens, a.n_new, stream);
  return PA_OK;
}

template <int D, bool BF16>
int launch_tc_d(const PrefillLaunch &a, cudaStream_t stream) {
  switch (group_tile(a.n_q_heads / a.n_kv_heads)) {
    case 8: return launch_tc_t<D, 8, BF16>(a, stream);
    case 4: return launch_tc_t<D, 4, BF16>(a, stream);
    case 2: return launch_tc_t<D, 2, BF16>(a, stream);
    default: return launch_tc_t<D, 1, BF16>(a, stream);
  }
}

}  // namespace

int launch_prefill(const PrefillLaunch &a, cudaStream_t stream) {
  if (a.head_dim == 128)
    return a.bf16 ? launch_tc_d<128, true>(a, stream) : launch_tc_d<128, false>(a, stream);
  return a.bf16 ? launch_tc_d<64, true>(a, stream) : launch_tc_d<64, false>(a, stream);
}

}  // namespace pa
