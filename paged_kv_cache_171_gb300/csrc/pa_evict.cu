// pa_evict.cu -- eviction by gathered attention weight, and the move of kept rows.
//
// Eviction.  Of a sequence of T > budget tokens every kv head keeps its first `sink`, its
// last `recent` and, of the others, the budget - sink - recent with the largest weight (ties
// to the lowest position; a NaN weight behind every number).  The kept rows of K, V and
// weights move to positions 0, 1, .. in their order.
//
// select_kernel: a cluster of up to 8 CTAs a (sequence, kv head), each with a part of the
// candidates in its shared memory as 32-bit keys of the weights' order.  A radix select over
// digits of 11, 11 and 10 bits finds the least key kept and how many of its ties are: a CTA's
// histogram each, and its sums over 32 bins; one warp of every CTA adds the sums of all CTAs up
// through distributed shared memory, then the 32 bins of the one that matters, and picks the
// same bin as the others (with all 2048 bins read by every CTA 1 x 32768 to 4096 took 36 us).
// Then each warp numbers the kept ones of a span of tokens by ballots and writes their positions.
//
// move_kernel: row src[j] to position j, where src is ascending, so src[j] >= j: the list
// may be worked off in place from its start, if a row is stored only when every row of the
// list up to it has been loaded.  A CTA therefore takes one (sequence, kv head) and a strip
// of the rows (of K or V, 32 bytes or more; or of the weights) through the whole list, a
// chunk of rows at a time: a thread loads chunk c + 1 into registers, a barrier, then
// chunk c is stored.  Strips are independent of each other: no CTA waits for another,
// however few lists there are.
//
// Bound: memory, 8 D bytes a kept token and kv head (K and V read and written).  32 sequences
// of 2000 to 4096 tokens to 2048: 108 us, of which 16 select and 90 move 0.5 GB.  Few
// long lists: the chain of passes and barriers (1 x 32768 to 4096, 8 lists: 30 us, 17 select).
#include "pa_device.cuh"
#include "pa_evict.h"

namespace pa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 49152;  // keys of a row that shared memory holds
constexpr int kSelSmem = kSelKeys * 4;
constexpr int kBins = 2048, kCoarse = kBins / 32, kMaxRanks = 8;
constexpr int kLoadAhead = 4;    // tokens a thread fetches at a time

struct SelectParams {
  const float *weights;
  const int32_t *block_table, *ctx_lens;
  int32_t *kept;   // [batch][kv heads][budget]
  int32_t *n_kept; // [batch]; -1: every token stays where it is in the list
  int32_t *new_lens;
  int *status;
  int n_kv_heads, batch, max_blocks, num_pages, budget, sink, recent;
  int held_keys;   // keys that a CTA's shared memory has room for
};

// Ascending with the weight; NaN below every number, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0u : u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

// Inclusive sum over the warp.
__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ int cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return static_cast<int>(r);
}
// Every thread of the cluster: shared memory written before it is seen behind it.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();  // the aligned forms want whole warps
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Two words (or one) at the place in rank `rank`'s shared memory that p has in this CTA's.
__device__ __forceinline__ uint32_t place_in(const int *p, int rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ int2 load2_of(const int *p, int rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y) : "r"(place_in(p, rank)));
  return v;
}
__device__ __forceinline__ int load_of(const int *p, int rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(place_in(p, rank)));
  return v;
}

__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) int hist[3][kBins];
  __shared__ __align__(16) int coarse[3][kCoarse];  // sums of 32 bins
  __shared__ int sums[kSelWarps], sums2[kSelWarps];
  __shared__ int pick[2];
  __shared__ __align__(16) int counts[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_rank(), ranks = cluster_size();
  const int bh = blockIdx.x / ranks, b = bh / p.n_kv_heads, h = bh - b * p.n_kv_heads;
  for (int i = tid; i < 3 * kBins; i += kSelThreads) hist[0][i] = 0;
  griddep_release();
  griddep_wait();
  const int most = p.max_blocks * kPageSize;
  int T = p.ctx_lens[b];
  if (T < 0 || T > most) {
    if (tid == 0) record_error(p.status, PA_ERR_BAD_CTX);
    T = T < 0 ? 0 : most;
  }
  if (tid == 0 && h == 0 && rank == 0) {
    p.n_kept[b] = T > p.budget ? p.budget : -1 - T;
    p.new_lens[b] = min(T, p.budget);
  }
  if (T <= p.budget) return;  // the whole cluster
  const int32_t *row = p.block_table + static_cast<size_t>(b) * p.max_blocks;
  int32_t *kept = p.kept + static_cast<size_t>(bh) * p.budget;
  const int c0 = p.sink, c1 = T - p.recent;  // the candidates
  // what stays anyway
  for (int t = rank * kSelThreads + tid; t < c0; t += ranks * kSelThreads) kept[t] = t;
  for (int t = c1 + rank * kSelThreads + tid; t < T; t += ranks * kSelThreads)
    kept[p.budget - (T - t)] = t;
  int need = p.budget - p.sink - p.recent;
  if (need == 0) return;  // the whole cluster

  // ---- this CTA's candidates [lo, hi), as keys
  const int part = (c1 - c0 + ranks - 1) / ranks;
  const int lo = min(c1, c0 + rank * part), hi = min(c1, lo + part);
  auto page_at = [&](int t) { return row[t / kPageSize]; };
  auto key_in = [&](int page, int t) {
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {
      record_error(p.status, PA_ERR_BAD_BLOCK);
      return 0u;
    }
    return key_of(p.weights[(static_cast<size_t>(page) * p.n_kv_heads + h) * kPageSize +
                            t % kPageSize]);
  };
  const bool held = part <= p.held_keys;
  __syncthreads();  // the histograms are clear
  if (held) {  // with the first digit's histogram
    for (int t0 = lo + tid; t0 < hi; t0 += kLoadAhead * kSelThreads) {
      int page[kLoadAhead];
      uint32_t k[kLoadAhead];
#pragma unroll
      for (int u = 0; u < kLoadAhead; ++u)
        page[u] = t0 + u * kSelThreads < hi ? page_at(t0 + u * kSelThreads) : 0;
#pragma unroll
      for (int u = 0; u < kLoadAhead; ++u)
        if (t0 + u * kSelThreads < hi) k[u] = key_in(page[u], t0 + u * kSelThreads);
#pragma unroll
      for (int u = 0; u < kLoadAhead; ++u)
        if (t0 + u * kSelThreads < hi) {
          keys[t0 + u * kSelThreads - lo] = k[u];
          atomicAdd(&hist[0][k[u] >> 21], 1);
        }
    }
  }
  auto key_at = [&](int t) { return held ? keys[t - lo] : key_in(page_at(t), t); };

  // ---- the least key kept, and how many of its ties
  uint32_t prefix = 0, known = 0;
  int shift = 21, bits = 11;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const uint32_t mask = (1u << bits) - 1;
    if (pass > 0 || !held)
      for (int t = lo + tid; t < hi; t += kSelThreads) {
        const uint32_t k = key_at(t);
        if ((k & known) == prefix) atomicAdd(&hist[pass][(k >> shift) & mask], 1);
      }
    __syncthreads();
    {
      static_assert(kBins == 4 * kSelThreads, "four bins a thread");
      const int4 v = *reinterpret_cast<const int4 *>(&hist[pass][4 * tid]);
      int n = v.x + v.y + v.z + v.w;
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) n += __shfl_xor_sync(kFull, n, x);
      if (tid % 8 == 0) coarse[pass][tid / 8] = n;
    }
    cluster_sync();
    if (warp == 0) {
      // From the top: which 32 bins, then which of them.  Lane i looks after two sums, the
      // (2 i + 1)-th and (2 i + 2)-th, then after a bin.
      int2 v[kMaxRanks];
#pragma unroll
      for (int k = 0; k < kMaxRanks; ++k)  // all on their way at once
        v[k] = k < ranks ? load2_of(&coarse[pass][kCoarse - 2 - 2 * lane], k) : make_int2(0, 0);
      int first = 0, second = 0;
#pragma unroll
      for (int k = 0; k < kMaxRanks; ++k) first += v[k].y, second += v[k].x;
      int before = warp_scan(first + second, lane) - first - second;
      const bool here = before < need && need <= before + first + second;
      const int src = __ffs(__ballot_sync(kFull, here)) - 1;
      const bool low = need > before + first;
      if (low) before += first;
      const int bin = 32 * (__shfl_sync(kFull, kCoarse - 1 - 2 * lane - low, src) + 1) - 1 - lane;
      const int rest = need - __shfl_sync(kFull, before, src);
      int n[kMaxRanks], total = 0;
#pragma unroll
      for (int k = 0; k < kMaxRanks; ++k) n[k] = k < ranks ? load_of(&hist[pass][bin], k) : 0;
#pragma unroll
      for (int k = 0; k < kMaxRanks; ++k) total += n[k];
      before = warp_scan(total, lane) - total;
      if (before < rest && rest <= before + total) {
        pick[0] = bin;
        pick[1] = rest - before;
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(pick[0]) << shift;
    known |= mask << shift;
    need = pick[1];
    __syncthreads();  // (the next pass writes them behind a barrier of its own)
    shift = pass == 0 ? 10 : 0;
    bits = pass == 0 ? 11 : 10;
  }
  const uint32_t least = prefix;
  const int ties = need;  // of key `least` that are kept

  // ---- positions of the kept: warp w numbers those of its span of tokens
  const int span = ((hi - lo + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int t0 = lo + warp * span, t1 = min(hi, t0 + span);
  auto look = [&](int t, uint32_t *more, uint32_t *tie) {
    const uint32_t k = t < t1 ? key_at(t) : 0u;
    *more = __ballot_sync(kFull, t < t1 && k > least);
    *tie = __ballot_sync(kFull, t < t1 && k == least);
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
  if (warp == kSelWarps - 1 && lane == 0) {
    counts[0] = at_more + n_more;
    counts[1] = at_tie + n_tie;
  }
  cluster_sync();
  for (int k = 0; k < rank; ++k) {
    const int2 v = load2_of(counts, k);
    at_more += v.x;
    at_tie += v.y;
  }
  const uint32_t below = (1u << lane) - 1;
  for (int t = t0; t < t1; t += 32) {
    look(t + lane, &more, &tie);
    const int my_tie = at_tie + __popc(tie & below);
    const bool stays = (more >> lane & 1) || ((tie >> lane & 1) && my_tie < ties);
    if (stays) kept[c0 + at_more + __popc(more & below) + min(my_tie, ties)] = t + lane;
    at_more += __popc(more);
    at_tie += __popc(tie);
  }
  cluster_sync();  // the others have read this CTA's shared memory
}

// ---- the move
constexpr int kMoveMaxThreads = 1024, kMoveUnroll = 4, kMovePart = 2048;

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

// V: what a thread moves of a row; lpr threads a row.  The rows' places are looked up a part
// of the list at a time, so that nothing but the rows is waited for in the loop.
template <typename V>
__device__ __forceinline__ void move_rows(const MoveParams &p, char *base, int row_bytes,
                                          int offset, int lpr, int b, int h, const int32_t *list,
                                          int n, int first, int *from, int *to) {
  const int tid = threadIdx.x;
  const int threads = blockDim.x;
  const int per = threads / lpr;  // rows a step
  const int r = tid / lpr;
  base += offset + (tid % lpr) * static_cast<int>(sizeof(V));
  const int32_t *src_row = p.block_table + static_cast<size_t>(b) * p.max_blocks;
  const int32_t *dst_row = p.dst_table + static_cast<size_t>(b) * p.dst_blocks;
  auto place = [&](const int32_t *table, int blocks, int pos) {  // row of the pool, or -1
    const int page = pos / kPageSize < blocks ? table[pos / kPageSize] : -1;
    return static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)
               ? (page * p.n_kv_heads + h) * kPageSize + pos % kPageSize : -1;
  };
  const int rows = per * kMoveUnroll;
  V v[kMoveUnroll], w[kMoveUnroll];
  for (int part = 0; part < n; part += kMovePart) {
    const int m = min(kMovePart, n - part);
    if (part > 0) __syncthreads();  // the places before have been used
#pragma unroll 4
    for (int i = tid; i < m; i += threads) {
      const int j = part + i;
      const int src = place(src_row, p.max_blocks, first + (list ? list[j] : j));
      const int dst = place(dst_row, p.dst_blocks, first + j);
      if (src < 0 || dst < 0) record_error(p.status, PA_ERR_BAD_BLOCK);
      from[i] = src;
      to[i] = src < 0 || src == dst ? -1 : dst;  // -1: not moved
    }
    __syncthreads();
    auto load = [&](int i0, V (&x)[kMoveUnroll]) {
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const int i = i0 + u * per + r;
        if (i < m && to[i] >= 0)
          x[u] = __ldcg(
              reinterpret_cast<const V *>(base + static_cast<size_t>(from[i]) * row_bytes));
      }
    };
    load(0, v);
    for (int i0 = 0; i0 < m; i0 += rows) {
      load(i0 + rows, w);
      __syncthreads();  // every row up to this chunk's last has been loaded
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const int i = i0 + u * per + r;
        if (i < m && to[i] >= 0)
          *reinterpret_cast<V *>(base + static_cast<size_t>(to[i]) * row_bytes) = v[u];
        v[u] = w[u];
      }
    }
  }
}

__global__ void __launch_bounds__(kMoveMaxThreads) move_kernel(const MoveParams p) {
  __shared__ int bad;
  __shared__ int from[kMovePart], to[kMovePart];
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
      for (int j = tid; j < n; j += blockDim.x) {
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
    move_rows<float>(p, reinterpret_cast<char *>(p.weights), sizeof(float), 0, 1, b, h, list, n,
                     first, from, to);
  } else {
    const int strip = plane % p.strips, bytes = p.row_bytes / p.strips;
    move_rows<uint4>(p, plane < p.strips ? p.k_cache : p.v_cache, p.row_bytes, strip * bytes,
                     bytes / 16, b, h, list, n, first, from, to);
  }
}

// longest: rows of a list at most.
int launch_move(const EvictLaunch &a, MoveParams &p, int longest, cudaStream_t stream) {
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
  // As many strips, of 32 bytes or more, as make one wave of K's and V's CTAs, one an SM (4 x 4096
  // of 8192 tokens: 128 CTAs 26 us, 256 32; with the weights' plane 160 CTAs, 29), and CTAs of 1024 threads, so that one has 64 KB in flight:
  // with four CTAs of 256 an SM instead, 1 x 4096 of 32768 took 52 us for 37, 4 x 4096 of 8192
  // 42 for 32, 32 x 2048 110 for 109.  Short lists: one chunk of 256 threads.
  const int64_t lists = static_cast<int64_t>(a.batch) * a.n_kv_heads;
  p.strips = 1;
  while (p.strips < p.row_bytes / 32 && lists * p.strips * 4 <= sms_or_default()) p.strips *= 2;
  const int threads = static_cast<int64_t>(longest) * (p.row_bytes / p.strips / 16) <=
                              256 * kMoveUnroll ? 256 : kMoveMaxThreads;
  const dim3 grid(static_cast<unsigned>(lists), 2 * p.strips + (a.weights ? 1 : 0));
  return launch_pdl(move_kernel, grid, dim3(threads), 0, stream, p) == cudaSuccess
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
  const int64_t keys = most - a.sink - a.recent > 0 ? most - a.sink - a.recent : 0;
  // Few lists of many tokens: a cluster each, of 2048 keys or more a CTA (8 lists of 32768:
  // 68 us with 1 CTA, 21 with 8, and 17 since the sums are taken in two steps).
  const int64_t lists = static_cast<int64_t>(a.batch) * a.n_kv_heads;
  int ranks = 1;
  while (ranks < kMaxRanks && lists * ranks * 2 <= sms_or_default() && keys >= 2 * 2048 * ranks)
    ranks *= 2;
  const int64_t part = (keys + ranks - 1) / ranks;
  s.held_keys = static_cast<int>(part < kSelKeys ? part : kSelKeys);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(lists * ranks));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = s.held_keys * sizeof(uint32_t);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, select_kernel, s) != cudaSuccess) return PA_ERR_CUDA;
  MoveParams p = {};
  p.list = s.kept;
  p.n_kept = s.n_kept;
  p.list_stride_b = static_cast<int64_t>(a.n_kv_heads) * a.budget;
  p.list_stride_h = a.budget;
  return launch_move(a, p, static_cast<int>(a.budget < most ? a.budget : most), stream);
}

int launch_compact(const EvictLaunch &a, cudaStream_t stream) {
  MoveParams p = {};
  p.list = a.keep;
  p.list_stride_b = a.max_keep;
  p.ctx_lens = a.ctx_lens;
  p.n_keep = a.n_keep;
  p.max_keep = a.max_keep;
  return launch_move(a, p, a.max_keep, stream);
}

}  // namespace pa
