// pa_evict.cu -- eviction by gathered attention weight, and the move of kept rows.
//
// Eviction.  Of a sequence of T > budget tokens every kv head keeps its first `sink`, its
// last `recent` and, of the others, the budget - sink - recent with the largest weight (ties
// to the lowest position; a NaN weight behind every number).  The kept rows of K, V and
// weights move to positions 0, 1, .. in their order.
//
// select_kernel: one CTA a (sequence, kv head).  The weights become 32-bit keys of the same
// order; a radix select over digits of 11, 11 and 10 bits finds the least key kept and how
// many of its ties are; then each warp numbers the kept ones of a span of tokens by ballots
// and writes their positions.
//
// move_kernel: row src[j] to position j, where src is ascending, so src[j] >= j: the list
// may be worked off in place from its start, if a row is stored only when every row of the
// list up to it has been loaded.  A CTA therefore takes one (sequence, kv head) and a strip
// of the rows (of K or V, 32 bytes or more; or of the weights) through the whole list, a
// chunk of rows at a time: a thread loads chunk c + 1 into registers, a barrier, then
// chunk c is stored.  Strips are independent of each other: no CTA waits for another,
// however few lists there are.
//
// Bound: memory, 8 D bytes a kept token and kv head (K and V read and written).
#include "pa_device.cuh"
#include "pa_evict.h"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSelThreads = 1024;
constexpr int kSelKeys = 49152;  // keys of a row that shared memory holds
constexpr int kSelSmem = kSelKeys * 4;
constexpr int kBins = 2048;

struct SelectParams {
  const float *weights;
  const int32_t *block_table, *ctx_lens;
  int32_t *kept;   // [batch][kv heads][budget]
  int32_t *n_kept; // [batch]; -1: every token stays where it is in the list
  int32_t *new_lens;
  int *status;
  int n_kv_heads, batch, max_blocks, num_pages, budget, sink, recent;
};

// Ascending with the weight; NaN below every number, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0u : u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

// Inclusive sum over the CTA's threads.
__device__ __forceinline__ int block_scan(int v, int *warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += x;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += x;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  if (warp > 0) v += warp_sums[warp - 1];
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ int hist[kBins];
  __shared__ int sums[32], sums2[32];
  __shared__ int pick[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.n_kv_heads, h = blockIdx.x - b * p.n_kv_heads;
  griddep_release();
  griddep_wait();
  const int most = p.max_blocks * kPageSize;
  int T = p.ctx_lens[b];
  if (T < 0 || T > most) {
    if (tid == 0) record_error(p.status, PA_ERR_BAD_CTX);
    T = T < 0 ? 0 : most;
  }
  if (tid == 0 && h == 0) {
    p.n_kept[b] = T > p.budget ? p.budget : -1 - T;
    p.new_lens[b] = min(T, p.budget);
  }
  if (T <= p.budget) return;
  const int32_t *row = p.block_table + static_cast<size_t>(b) * p.max_blocks;
  const int lo = p.sink, hi = T - p.recent;  // the candidates
  auto load_key = [&](int t) {
    const int page = row[t / kPageSize];
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {
      record_error(p.status, PA_ERR_BAD_BLOCK);
      return 0u;
    }
    return key_of(p.weights[(static_cast<size_t>(page) * p.n_kv_heads + h) * kPageSize +
                            t % kPageSize]);
  };
  const bool held = hi - lo <= kSelKeys;
  if (held) {
#pragma unroll 4
    for (int t = lo + tid; t < hi; t += kSelThreads) keys[t - lo] = load_key(t);
    __syncthreads();
  }
  auto key_at = [&](int t) { return held ? keys[t - lo] : load_key(t); };

  // ---- the least key kept, and how many of its ties
  int need = p.budget - p.sink - p.recent;
  uint32_t least = 0xffffffffu;  // none of the candidates
  if (need > 0) {
    uint32_t prefix = 0, known = 0;
    int shift = 21, bits = 11;
    for (int pass = 0; pass < 3; ++pass) {
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      const uint32_t mask = (1u << bits) - 1;
      for (int t = lo + tid; t < hi; t += kSelThreads) {
        const uint32_t k = key_at(t);
        if ((k & known) == prefix) atomicAdd(&hist[(k >> shift) & mask], 1);
      }
      __syncthreads();
      // thread i looks after bins kBins - 1 - 2 i and the one below: from the top
      const int b0 = kBins - 1 - 2 * tid;
      const int c0 = hist[b0], c1 = hist[b0 - 1];
      const int incl = block_scan(c0 + c1, sums);
      const int before = incl - c0 - c1;
      if (before < need && need <= incl) {
        const bool first = need <= before + c0;
        pick[0] = first ? b0 : b0 - 1;
        pick[1] = need - before - (first ? 0 : c0);
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(pick[0]) << shift;
      known |= mask << shift;
      need = pick[1];
      __syncthreads();
      shift = pass == 0 ? 10 : 0;
      bits = pass == 0 ? 11 : 10;
    }
    least = prefix;
  }
  const int ties = need;  // of key `least` that are kept

  // ---- positions of the kept: warp w numbers those of its span of tokens
  const int span = ((T + 31) / 32 + 31) / 32 * 32;
  const int t0 = warp * span, t1 = min(T, t0 + span);
  auto look = [&](int t, uint32_t *more, uint32_t *tie) {
    bool m = false, e = false;
    if (t < t1) {
      m = t < lo || t >= hi;
      if (!m && p.budget > p.sink + p.recent) {
        const uint32_t k = key_at(t);
        m = k > least;
        e = k == least;
      }
    }
    *more = __ballot_sync(kFull, m);
    *tie = __ballot_sync(kFull, e);
  };
  int n_more = 0, n_tie = 0;
  uint32_t more, tie;
  for (int t = t0; t < t1; t += 32) {
    look(t + lane, &more, &tie);
    n_more += __popc(more);
    n_tie += __popc(tie);
  }
  if (lane == 0) {
    sums[warp] = n_more;
    sums2[warp] = n_tie;
  }
  __syncthreads();
  int at_more = 0, at_tie = 0;  // before the warp's span
  for (int w = 0; w < warp; ++w) {
    at_more += sums[w];
    at_tie += sums2[w];
  }
  int32_t *kept = p.kept + static_cast<size_t>(blockIdx.x) * p.budget;
  const uint32_t below = (1u << lane) - 1;
  for (int t = t0; t < t1; t += 32) {
    look(t + lane, &more, &tie);
    const int my_tie = at_tie + __popc(tie & below);
    const bool stays = (more >> lane & 1) || ((tie >> lane & 1) && my_tie < ties);
    if (stays) kept[at_more + __popc(more & below) + min(my_tie, ties)] = t + lane;
    at_more += __popc(more);
    at_tie += __popc(tie);
  }
}

// ---- the move
constexpr int kMoveThreads = 256, kMoveUnroll = 4;

struct MoveParams {
  char *k_cache, *v_cache;
  float *weights;
  const int32_t *block_table, *dst_table;
  const int32_t *list;     // kept positions, or null: every token
  const int32_t *n_kept;   // [batch] (select_kernel), or null for a compaction
  const int32_t *ctx_lens, *n_keep;  // of a compaction
  int32_t *new_lens;       // of a compaction
  int *status;
  int64_t list_stride_b, list_stride_h;
  int n_kv_heads, row_bytes, strips, max_blocks, dst_blocks, num_pages, max_keep;
};

// V: what a thread moves of a row; LPR threads a row.
template <typename V>
__device__ __forceinline__ void move_rows(const MoveParams &p, char *base, size_t head_bytes,
                                          int row_bytes, int offset, int lpr, int b, int h,
                                          const int32_t *list, int n, int first) {
  const int tid = threadIdx.x;
  const int per = kMoveThreads / lpr;  // rows a step
  const int r = tid / lpr, c = offset + (tid % lpr) * static_cast<int>(sizeof(V));
  const int32_t *src_row = p.block_table + static_cast<size_t>(b) * p.max_blocks;
  const int32_t *dst_row = p.dst_table + static_cast<size_t>(b) * p.dst_blocks;
  const size_t page_bytes = head_bytes * p.n_kv_heads;
  const size_t head = h * head_bytes;
  auto place = [&](const int32_t *table, int blocks, int pos, size_t *off) {
    const int page = pos / kPageSize < blocks ? table[pos / kPageSize] : -1;
    *off = page * page_bytes + head + static_cast<size_t>(pos % kPageSize) * row_bytes + c;
    return static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
  };
  struct Step {
    size_t src[kMoveUnroll], dst[kMoveUnroll];
    unsigned real;  // bit u: row u is to be moved
  };
  auto plan = [&](int j0, Step &s) {
    s.real = 0;
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int j = j0 + u * per + r;
      s.src[u] = s.dst[u] = 0;
      if (j < n) {
        const int from = first + (list ? list[j] : j);
        const bool ok = place(src_row, p.max_blocks, from, &s.src[u]) &
                        place(dst_row, p.dst_blocks, first + j, &s.dst[u]);
        if (!ok)
          record_error(p.status, PA_ERR_BAD_BLOCK);
        else if (s.src[u] != s.dst[u])
          s.real |= 1u << u;
      }
    }
  };
  const int rows = per * kMoveUnroll;
  Step now, then;
  V v[kMoveUnroll], w[kMoveUnroll];
  auto load = [&](const Step &s, V (&x)[kMoveUnroll]) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (s.real >> u & 1) x[u] = __ldcg(reinterpret_cast<const V *>(base + s.src[u]));
  };
  plan(0, now);
  load(now, v);
  plan(rows, then);
  for (int j0 = 0; j0 < n; j0 += rows) {
    load(then, w);
    __syncthreads();  // every row up to this chunk's last has been loaded
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (now.real >> u & 1) *reinterpret_cast<V *>(base + now.dst[u]) = v[u];
    now = then;
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) v[u] = w[u];
    plan(j0 + 2 * rows, then);
  }
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveParams p) {
  __shared__ int bad;
  const int tid = threadIdx.x;
  const int bh = blockIdx.x, b = bh / p.n_kv_heads, h = bh - b * p.n_kv_heads;
  const int plane = blockIdx.y;  // strips of K, strips of V, the weights
  griddep_release();
  griddep_wait();  // the lists
  int n, first = 0;
  const int32_t *list = p.list + b * p.list_stride_b + h * p.list_stride_h;
  if (p.n_kept) {
    n = p.n_kept[b];
    if (n < 0) {  // every token
      n = -1 - n;
      list = nullptr;
      if (p.dst_table == p.block_table) return;
    }
  } else {
    first = p.ctx_lens[b];
    n = p.n_keep[b];
    const int most = p.max_blocks * kPageSize;
    if (tid == 0) bad = first < 0 || first > most || n < 0 || n > p.max_keep;
    __syncthreads();
    if (!bad) {  // ascending, and within the table
      bool wrong = false;
      for (int j = tid; j < n; j += kMoveThreads) {
        const int at = list[j], before = j > 0 ? list[j - 1] : -1;
        wrong |= at <= before || at >= most - first;
      }
      if (wrong) bad = 1;
    }
    __syncthreads();
    if (bad) {  // nothing is kept
      if (tid == 0) {
        record_error(p.status, first < 0 || first > most ? PA_ERR_BAD_CTX : PA_ERR_BAD_INDEX);
        if (h == 0 && plane == 0) p.new_lens[b] = min(max(first, 0), most);
      }
      return;
    }
    if (tid == 0 && h == 0 && plane == 0) p.new_lens[b] = first + n;
  }
  if (plane == 2 * p.strips) {
    move_rows<float>(p, reinterpret_cast<char *>(p.weights), kPageSize * sizeof(float),
                     sizeof(float), 0, 1, b, h, list, n, first);
  } else {
    const int strip = plane % p.strips, bytes = p.row_bytes / p.strips;
    move_rows<uint4>(p, plane < p.strips ? p.k_cache : p.v_cache,
                     static_cast<size_t>(kPageSize) * p.row_bytes, p.row_bytes, strip * bytes,
                     bytes / 16, b, h, list, n, first);
  }
}

int launch_move(const EvictLaunch &a, MoveParams &p, cudaStream_t stream) {
  p.k_cache = static_cast<char *>(a.k_cache);
  p.v_cache = static_cast<char *>(a.v_cache);
  p.weights = a.weights;
  p.block_table = a.block_table;
  p.dst_table = a.dst_table;
  p.new_lens = a.new_lens;
  p.status = a.status;
  p.n_kv_heads = a.n_kv_heads;
  p.row_bytes = a.head_dim * 2;
  p.max_blocks = a.max_blocks;
  p.dst_blocks = a.dst_blocks;
  p.num_pages = a.num_pages;
  // as many strips as give every SM four CTAs, of 32 bytes or more
  const int64_t lists = static_cast<int64_t>(a.batch) * a.n_kv_heads;
  p.strips = 1;
  while (p.strips < p.row_bytes / 32 && lists * p.strips * 2 < 4 * sms_or_default())
    p.strips *= 2;
  const dim3 grid(static_cast<unsigned>(lists), 2 * p.strips + (a.weights ? 1 : 0));
  return launch_pdl(move_kernel, grid, dim3(kMoveThreads), 0, stream, p) == cudaSuccess
             ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

// The kept positions, then the number of each sequence.
size_t evict_workspace_bytes(int batch, int n_kv_heads, int max_blocks, int budget) {
  const int64_t most = static_cast<int64_t>(max_blocks) * kPageSize;
  const int64_t per = budget < most ? budget : 0;  // else every token stays
  return (static_cast<size_t>(batch) * n_kv_heads * per + batch) * sizeof(int32_t);
}

int launch_evict(const EvictLaunch &a, cudaStream_t stream) {
  SelectParams s;
  s.weights = a.weights;
  s.block_table = a.block_table;
  s.ctx_lens = a.ctx_lens;
  s.n_kept = static_cast<int32_t *>(a.workspace);
  s.kept = s.n_kept + a.batch;
  s.new_lens = a.new_lens;
  s.status = a.status;
  s.n_kv_heads = a.n_kv_heads;
  s.batch = a.batch;
  s.max_blocks = a.max_blocks;
  s.num_pages = a.num_pages;
  s.budget = a.budget;
  s.sink = a.sink;
  s.recent = a.recent;
  static ContextCache<bool> smem_set;
  if (set_smem_limit(select_kernel, kSelSmem, smem_set) != PA_OK) return PA_ERR_CUDA;
  const int64_t most = static_cast<int64_t>(a.max_blocks) * kPageSize;
  const int64_t keys = most - a.sink - a.recent;
  const size_t smem = keys <= 0 ? 0 : (keys < kSelKeys ? keys : kSelKeys) * 4;
  if (launch_pdl(select_kernel, dim3(static_cast<unsigned>(a.batch) * a.n_kv_heads),
                 dim3(kSelThreads), smem, stream, s) != cudaSuccess)
    return PA_ERR_CUDA;
  MoveParams p = {};
  p.list = s.kept;
  p.n_kept = s.n_kept;
  p.list_stride_b = static_cast<int64_t>(a.n_kv_heads) * a.budget;
  p.list_stride_h = a.budget;
  return launch_move(a, p, stream);
}

int launch_compact(const EvictLaunch &a, cudaStream_t stream) {
  MoveParams p = {};
  p.list = a.keep;
  p.list_stride_b = a.max_keep;
  p.ctx_lens = a.ctx_lens;
  p.n_keep = a.n_keep;
  p.max_keep = a.max_keep;
  return launch_move(a, p, stream);
}

}  // namespace pa
