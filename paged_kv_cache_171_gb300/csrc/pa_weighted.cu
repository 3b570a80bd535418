// pa_weighted.cu -- decode attention that also gathers, for every cached token and kv
// head, the attention weight the step's queries gave it.
//
//   s_t = scale q_h . k_t,  p_h[t] = e^(s_t - m) / l,  out_h = sum_t p_h[t] v_t
//   weights[t] = (t < T - fresh ? weights[t] : 0) + sum_{h in the kv head's group} p_h[t]
//
// A weight needs the row's final m and l, which no CTA has before the last key.  So the
// pass over K and V stores each score (4 bytes a query head and token beside the 4 D
// bytes a kv head and token of K and V) and a second, short kernel folds the rows'
// partial states into (m, l) and out, reads the scores back, mostly from L2, and adds
// e^(s - m) / l over the group.  Reading K again instead would cost 2 D bytes a token
// and kv head: 32 to 256 bytes against 8 a query head.
//
// Operand form.  mma.sync m16n8k16 with the tokens (then the head dimensions) as the 16
// rows and up to 8 query rows as the columns: S = K Q^T straight from the page's tile by
// ldmatrix, O = V^T P by its transposing form, P from the accumulators by movmatrix.  The
// weights p enter as bf16 in three terms (24 bits) or as fp16 in two (22 bits, of 2^7 p,
// so down to 2^-32 of the row's largest): one term would leave 2^-9 or 2^-12 of every
// weight in an fp32 result.  A page's sum has an accumulator of its own that a rounding
// add joins to the state, because the tensor cores' sums round toward zero.
//
// Work split.  The pages of all (sequence, kv head, tile of 8 query rows) items, laid end
// to end, are cut into equal runs, one a warp: eight warps an SM, each with a ring of
// pages (K and V, 2-D TMA, 128-byte swizzle) that it feeds itself across item borders.
// An item cut between warps leaves a partial state a warp; states are numbered item +
// warp, which grows along the list, so that the second kernel finds an item's in order
// and results do not depend on timing.
#include "pa_device.cuh"
#include "pa_evict.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleSlack = 8.0f;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kNoKey = -3.402823466e38f;  // running max of a row before its first key
constexpr int kWarps = 8;                   // a CTA, one CTA an SM
constexpr int kTile = 8;                    // query rows a tile
constexpr int kMinPages = 2;                // least pages a run has
constexpr int kFoldThreads = 256;

struct WeightedParams {
  const uint16_t *q;
  const int32_t *block_table, *ctx_lens;
  float *out, *weights;
  float *states;  // [item + warp][kTile][D + 4]: O, m (log2), l
  int2 *span;     // [item]: first and last warp that holds a part of it
  float *scores;  // per tile [T][rows], tiles at (first row) * max_tokens
  int *status;
  float qscale;   // scale * log2 e
  int n_q_heads, n_kv_heads, group, n_sub, tile_rows, batch, max_blocks, num_pages, fresh;
  int seg_tokens, segs;  // tokens a CTA of the second kernel looks after, CTAs an item
};

template <int D>
struct WeightedSmem {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kTileBytes = kPageSize * D * 2;  // K or V of a page and kv head
  static constexpr int kStage = 2 * kTileBytes;
  static constexpr int kBars = kWarps * kStages * kStage;
  static constexpr int kBytes = kBars + kWarps * kStages * 8;
  static constexpr int kAlloc = kBytes + 1024;  // the swizzle wants 1024-byte tiles
  static_assert(kAlloc <= 232448, "shared memory of an SM");
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Tokens of sequence b; a length outside the table is clamped (and reported).
__device__ __forceinline__ int tokens_of(const WeightedParams &p, int b, bool report) {
  const int most = p.max_blocks * kPageSize;
  int t = p.ctx_lens[b];
  if (t < 0 || t > most) {
    if (report) record_error(p.status, PA_ERR_BAD_CTX);
    t = t < 0 ? 0 : most;
  }
  return t;
}
// An empty sequence counts one page, so that someone writes its state.
__device__ __forceinline__ int pages_of(int tokens) {
  return max(1, (tokens + kPageSize - 1) / kPageSize);
}

// A place in the list of pages of all items.
struct Cursor {
  int b, g, sub, page, n_pages, tokens;
  __device__ void enter_sequence(const WeightedParams &p) {
    tokens = tokens_of(p, b, false);
    n_pages = pages_of(tokens);
  }
  __device__ void next_item(const WeightedParams &p) {
    page = 0;
    if (++sub < p.n_sub) return;
    sub = 0;
    if (++g < p.n_kv_heads) return;
    g = 0;
    ++b;
    enter_sequence(p);
  }
  __device__ int item(const WeightedParams &p) const {
    return (b * p.n_kv_heads + g) * p.n_sub + sub;
  }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kWarps * 32, 1)
    weighted_kernel(const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const WeightedParams p) {
  using L = WeightedSmem<D>;
  constexpr int KS = D / 16, kTerms = BF16 ? 3 : 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ln = lane >> 2, lc = lane & 3;
  const int n_workers = gridDim.x * kWarps, worker = warp * gridDim.x + blockIdx.x;
  const uint32_t ring = smem_u32(smem) + warp * L::kStages * L::kStage;
  const uint32_t bars = smem_u32(smem) + L::kBars + warp * L::kStages * 8;
  if (lane == 0) {
    for (int s = 0; s < L::kStages; ++s) mbar_init(bars + 8 * s, 1);
    fence_mbar_init();
  }
  __syncwarp();
  griddep_release();
  griddep_wait();  // inputs may come from the previous kernel in the stream

  // ---- the run: lane l sums the pages of sequences [l per, (l + 1) per), a scan finds
  // the sequence in which the run starts
  const int heads = p.n_kv_heads * p.n_sub;
  Cursor at;
  int64_t run, w0;
  int left;  // pages of the run not yet done
  {
    const int per = (p.batch + 31) / 32;
    const int b0 = min(p.batch, lane * per), b1 = min(p.batch, b0 + per);
    int64_t sum = 0;
#pragma unroll 4
    for (int i = b0; i < b1; ++i) sum += pages_of(tokens_of(p, i, worker == 0));
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    const int64_t total = __shfl_sync(kFull, incl, 31) * heads;
    run = max((total + n_workers - 1) / n_workers, static_cast<int64_t>(kMinPages));
    w0 = worker * run;
    if (w0 >= total) return;
    left = static_cast<int>(min(total - w0, run));
    const int src = __ffs(__ballot_sync(kFull, incl * heads > w0)) - 1;
    at.b = __shfl_sync(kFull, b0, src);
    int64_t base = __shfl_sync(kFull, incl - sum, src) * heads;
    at.enter_sequence(p);
    while (base + static_cast<int64_t>(at.n_pages) * heads <= w0) {
      base += static_cast<int64_t>(at.n_pages) * heads;
      ++at.b;
      at.enter_sequence(p);
    }
    const int64_t rel = w0 - base;
    const int hs = static_cast<int>(rel / at.n_pages);
    at.page = static_cast<int>(rel - static_cast<int64_t>(hs) * at.n_pages);
    at.g = hs / p.n_sub;
    at.sub = hs - at.g * p.n_sub;
  }

  // ---- the feed: copies pages up to kStages ahead, across item borders
  Cursor fc = at;
  int feed_left = left, ids = 0;
  uint32_t issued = 0, waited = 0;
  auto load_ids = [&]() {  // ids of pages 32 k .. 32 k + 31 that hold fc.page, one a lane
    const int pg = (fc.page & ~31) + lane;
    ids = pg < fc.n_pages && fc.tokens > 0
              ? p.block_table[static_cast<size_t>(fc.b) * p.max_blocks + pg] : 0;
  };
  load_ids();
  auto issue = [&]() {  // the next page that has keys, if the run has one
    while (feed_left > 0) {
      const bool real = fc.tokens > 0;
      if (real) {
        int id = __shfl_sync(kFull, ids, fc.page & 31);
        if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) {
          if (lane == 0) record_error(p.status, PA_ERR_BAD_BLOCK);
          id = 0;  // read a page that exists; the result is flagged as invalid
        }
        if (lane == 0) {
          const uint32_t s = issued % L::kStages, bar = bars + 8 * s;
          const uint32_t dst = ring + s * L::kStage;
          const int y = (id * p.n_kv_heads + fc.g) * kPageSize;
          fence_proxy_async_smem();
          mbar_arrive_expect_tx(bar, L::kStage);
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            tma_load_2d(dst + x * 2048, &kmap, 64 * x, y, bar);
            tma_load_2d(dst + L::kTileBytes + x * 2048, &vmap, 64 * x, y, bar);
          }
        }
        ++issued;
      }
      --feed_left;
      if (++fc.page == fc.n_pages && feed_left > 0) {
        fc.next_item(p);
        load_ids();
      } else if ((fc.page & 31) == 0 && feed_left > 0) {
        load_ids();
      }
      if (real) return;
    }
  };
#pragma unroll 1
  for (int s = 0; s < L::kStages; ++s) issue();

  int64_t unit = w0;
  while (left > 0) {  // part by part
    const int pg0 = at.page, n = min(left, at.n_pages - pg0);
    const int r0 = at.sub * p.tile_rows, n_r = min(p.tile_rows, p.group - r0);
    const int row0 = at.b * p.n_q_heads + at.g * p.group + r0;  // first query row of the tile
    const int item = at.item(p);
    if (pg0 == 0 && lane == 0)
      p.span[item] = make_int2(worker, static_cast<int>((unit + at.n_pages - 1) / run));

    // q as the first product's second operand: column ln, dimensions 2 lc + {0, 1} (+ 8)
    uint32_t qb[KS][2];
#pragma unroll
    for (int k = 0; k < KS; ++k) qb[k][0] = qb[k][1] = 0;
    if (ln < n_r) {
      const uint32_t *src =
          reinterpret_cast<const uint32_t *>(p.q + static_cast<size_t>(row0 + ln) * D) + lc;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qb[k][0] = src[8 * k];
        qb[k][1] = src[8 * k + 4];
      }
    }
    float2 o[KS][2];  // dimensions 16 k + ln (+ 8), columns 2 lc + {0, 1}
#pragma unroll
    for (int k = 0; k < KS; ++k) o[k][0] = o[k][1] = make_float2(0.f, 0.f);
    float2 m = make_float2(kNoKey, kNoKey), l = make_float2(0.f, 0.f);
    float *score = p.scores + static_cast<size_t>(row0) * p.max_blocks * kPageSize;

    for (int i = 0; i < n && at.tokens > 0; ++i) {
      const uint32_t st = waited % L::kStages;
      if (!__all_sync(kFull, mbar_wait(bars + 8 * st, (waited / L::kStages) & 1))) {
        if (lane == 0) record_error(p.status, PA_ERR_TIMEOUT);
        for (uint32_t k = waited + 1; k < issued; ++k)  // copies in flight still land
          mbar_wait(bars + 8 * (k % L::kStages), (k / L::kStages) & 1);
        return;
      }
      ++waited;
      const uint32_t kt = ring + st * L::kStage, vt = kt + L::kTileBytes;
      const int key0 = (pg0 + i) * kPageSize;
      const int seen = at.tokens - key0;  // keys of this page
      if (seen < kPageSize) {  // rows past the end may hold anything: 0 * NaN is NaN
        for (int e = lane; e < (kPageSize - seen) * (D / 8); e += 32) {
          const int r = seen + e / (D / 8), c = e % (D / 8);
          st_shared_v4(vt + (c >> 3) * 2048 + swz128(r, c), 0u, 0u, 0u, 0u);
        }
        __syncwarp();
      }

      // ---- scores of tokens ln and ln + 8, rows 2 lc and 2 lc + 1
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a[4];
        ldsm_x4(kt + (k >> 2) * 2048 + swz128(lane & 15, 2 * (k & 3) + (lane >> 4)), a[0], a[1],
                a[2], a[3]);
        mma16816<BF16>(s, a, qb[k][0], qb[k][1]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] *= p.qscale;
      if (seen < kPageSize) {
        if (ln >= seen) s[0] = s[1] = -INFINITY;
        if (ln + 8 >= seen) s[2] = s[3] = -INFINITY;
      }
      // kept for the second kernel, [token][row]
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (ln + 8 * u < seen && 2 * lc < n_r) {
          float *dst = score + static_cast<size_t>(key0 + ln + 8 * u) * n_r + 2 * lc;
          if ((n_r & 1) == 0) {
            *reinterpret_cast<float2 *>(dst) = make_float2(s[2 * u], s[2 * u + 1]);
          } else {
            dst[0] = s[2 * u];
            if (2 * lc + 1 < n_r) dst[1] = s[2 * u + 1];
          }
        }
      }

      // ---- move the references when a score outgrows them
      const float grow = fmaxf(fmaxf(s[0], s[2]) - m.x, fmaxf(s[1], s[3]) - m.y);
      if (__any_sync(kFull, grow > kRescaleSlack)) {
        float a = fmaxf(s[0], s[2]), b = fmaxf(s[1], s[3]);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          a = fmaxf(a, __shfl_xor_sync(kFull, a, x));
          b = fmaxf(b, __shfl_xor_sync(kFull, b, x));
        }
        a = fmaxf(m.x, a);
        b = fmaxf(m.y, b);
        const float2 c = make_float2(ex2(m.x - a), ex2(m.y - b));
        m = make_float2(a, b);
        l = __fmul2_rn(l, c);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          o[k][0] = __fmul2_rn(o[k][0], c);
          o[k][1] = __fmul2_rn(o[k][1], c);
        }
      }

      // ---- weights, in terms, as the second product's operand (row ln, tokens 2 lc ..)
      uint32_t pb[kTerms][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float2 w = make_float2(ex2(s[2 * u] - m.x), ex2(s[2 * u + 1] - m.y));
        l = __fadd2_rn(l, w);
        if (!BF16) w = make_float2(w.x * 128.f, w.y * 128.f);
#pragma unroll
        for (int t = 0; t < kTerms; ++t) {
          const uint32_t head = pack2<BF16>(w.x, w.y);
          pb[t][u] = transpose8x8(head);
          w = __ffma2_rn(unpack2<BF16>(head), make_float2(-1.f, -1.f), w);
        }
      }

      // ---- O[dimension][row] += V^T P
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a[4];
        ldsm_x4_t(vt + (k >> 2) * 2048 +
                      swz128((lane & 7) + 8 * (lane >> 4), 2 * (k & 3) + ((lane >> 3) & 1)),
                  a[0], a[1], a[2], a[3]);
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = kTerms - 1; x >= 0; --x) mma16816<BF16>(t, a, pb[x][0], pb[x][1]);
        o[k][0] = __fadd2_rn(o[k][0], make_float2(t[0], t[1]));
        o[k][1] = __fadd2_rn(o[k][1], make_float2(t[2], t[3]));
      }
      __syncwarp();  // the stage has been read by every lane
      issue();
    }

    // ---- the part's state
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l.x += __shfl_xor_sync(kFull, l.x, x);
      l.y += __shfl_xor_sync(kFull, l.y, x);
    }
    float *state = p.states + (static_cast<size_t>(item) + worker) * (kTile * (D + 4));
    const float down = BF16 ? 1.f : 1.f / 128.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (2 * lc + u >= n_r) continue;
      float *row = state + (2 * lc + u) * (D + 4);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        row[16 * k + ln] = (u ? o[k][0].y : o[k][0].x) * down;
        row[16 * k + 8 + ln] = (u ? o[k][1].y : o[k][1].x) * down;
      }
      if (ln == 0)
        *reinterpret_cast<float2 *>(row + D) = u ? make_float2(m.y, l.y) : make_float2(m.x, l.x);
    }
    left -= n;
    unit += n;
    if (left > 0) at.next_item(p);
  }
}

// The second kernel: CTA (sequence x kv head, segment).  The rows' states are folded into
// (m, 1 / l), one warp a row; out's elements are shared out among the segments' CTAs; then
// a thread a token adds the group's weights to the pool.
template <int D>
__global__ void __launch_bounds__(kFoldThreads) weighted_fold_kernel(const WeightedParams p) {
  extern __shared__ float2 rows[];  // [group]: m, 1 / l
  const int bg = blockIdx.x / p.segs, seg = blockIdx.x - bg * p.segs;
  const int b = bg / p.n_kv_heads, g = bg - b * p.n_kv_heads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_release();
  griddep_wait();  // the states and scores
  const int tokens = tokens_of(p, b, false);
  const int seg0 = seg * p.seg_tokens;
  if (seg0 > 0 && seg0 >= tokens) return;
  const int segs = max(1, (tokens + p.seg_tokens - 1) / p.seg_tokens);

  for (int r = warp; r < p.group; r += kFoldThreads / 32) {
    const int sub = r / p.tile_rows, rr = r - sub * p.tile_rows;
    const int item = bg * p.n_sub + sub;
    const int2 span = p.span[item];
    float m = kNoKey, l = 0.f;
    for (int c = span.x + lane; c <= span.y; c += 32) {
      const float2 ml = *reinterpret_cast<const float2 *>(
          p.states + ((static_cast<size_t>(item) + c) * kTile + rr) * (D + 4) + D);
      const float mn = fmaxf(m, ml.x);
      l = l * ex2(m - mn) + ml.y * ex2(ml.x - mn);
      m = mn;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
      const float mo = __shfl_xor_sync(kFull, m, x), lo = __shfl_xor_sync(kFull, l, x);
      const float mn = fmaxf(m, mo);
      l = l * ex2(m - mn) + lo * ex2(mo - mn);
      m = mn;
    }
    if (lane == 0) rows[r] = make_float2(m, l == 0.f ? 0.f : 1.f / l);
  }
  __syncthreads();

  // ---- out: four dimensions of a row at a time, a warp each, lanes over the states
  const int n_el = p.group * (D / 4);
  const int e0 = static_cast<int>(static_cast<int64_t>(n_el) * seg / segs);
  const int e1 = static_cast<int>(static_cast<int64_t>(n_el) * (seg + 1) / segs);
  for (int e = e0 + warp; e < e1; e += kFoldThreads / 32) {
    const int r = e / (D / 4), d = 4 * (e % (D / 4));
    const int sub = r / p.tile_rows, rr = r - sub * p.tile_rows;
    const int item = bg * p.n_sub + sub;
    const int2 span = p.span[item];
    const float2 row = rows[r];
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = span.x + lane; c <= span.y; c += 32) {
      const float *s = p.states + ((static_cast<size_t>(item) + c) * kTile + rr) * (D + 4);
      const float f = ex2(s[D] - row.x);
      const float4 v = *reinterpret_cast<const float4 *>(s + d);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
      acc.x += __shfl_xor_sync(kFull, acc.x, x);
      acc.y += __shfl_xor_sync(kFull, acc.y, x);
      acc.z += __shfl_xor_sync(kFull, acc.z, x);
      acc.w += __shfl_xor_sync(kFull, acc.w, x);
    }
    if (lane == 0)
      *reinterpret_cast<float4 *>(
          p.out + (static_cast<size_t>(b) * p.n_q_heads + g * p.group + r) * D + d) =
          make_float4(acc.x * row.y, acc.y * row.y, acc.z * row.y, acc.w * row.y);
  }

  // ---- weights: a thread a token
  const int t1 = min(tokens, seg0 + p.seg_tokens);
  const size_t row0 = static_cast<size_t>(b) * p.n_q_heads + g * p.group;
  const size_t max_tokens = static_cast<size_t>(p.max_blocks) * kPageSize;
  for (int t = seg0 + tid; t < t1; t += kFoldThreads) {
    const int page = p.block_table[static_cast<size_t>(b) * p.max_blocks + t / kPageSize];
    float sum = 0.f;
    for (int r0 = 0; r0 < p.group; r0 += p.tile_rows) {
      const int n_r = min(p.tile_rows, p.group - r0);
      const float *s = p.scores + (row0 + r0) * max_tokens + static_cast<size_t>(t) * n_r;
      if (n_r % 4 == 0) {
        for (int r = 0; r < n_r; r += 4) {
          const float4 v = *reinterpret_cast<const float4 *>(s + r);
          sum += ex2(v.x - rows[r0 + r].x) * rows[r0 + r].y;
          sum += ex2(v.y - rows[r0 + r + 1].x) * rows[r0 + r + 1].y;
          sum += ex2(v.z - rows[r0 + r + 2].x) * rows[r0 + r + 2].y;
          sum += ex2(v.w - rows[r0 + r + 3].x) * rows[r0 + r + 3].y;
        }
      } else {
        for (int r = 0; r < n_r; ++r) sum += ex2(s[r] - rows[r0 + r].x) * rows[r0 + r].y;
      }
    }
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) continue;  // reported
    float *w = p.weights + (static_cast<size_t>(page) * p.n_kv_heads + g) * kPageSize +
               t % kPageSize;
    *w = (t < tokens - p.fresh ? *w : 0.f) + sum;
  }
}

// Row tiles of a group: as few as there can be, of nearly equal size.
void tiles_of(int group, int *n_sub, int *rows) {
  *n_sub = (group + kTile - 1) / kTile;
  *rows = (group + *n_sub - 1) / *n_sub;
  *n_sub = (group + *rows - 1) / *rows;
}

struct Layout {
  size_t span, scores, bytes;
};
Layout layout_of(int batch, int n_q_heads, int n_kv_heads, int head_dim, int max_blocks,
                 int sms) {
  int n_sub, rows;
  tiles_of(n_q_heads / n_kv_heads, &n_sub, &rows);
  const size_t items = static_cast<size_t>(batch) * n_kv_heads * n_sub;
  Layout y;
  y.span = (items + static_cast<size_t>(sms) * kWarps) * kTile * (head_dim + 4) * sizeof(float);
  y.scores = (y.span + items * sizeof(int2) + 15) & ~size_t(15);
  y.bytes = y.scores + static_cast<size_t>(batch) * n_q_heads * max_blocks * kPageSize *
                           sizeof(float);
  return y;
}

template <int D, bool BF16>
int launch_t(const WeightedLaunch &a, cudaStream_t stream) {
  auto kern = weighted_kernel<D, BF16>;
  static ContextCache<bool> smem_set;
  if (set_smem_limit(kern, WeightedSmem<D>::kAlloc, smem_set) != PA_OK) return PA_ERR_CUDA;
  const int sms = sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  CUtensorMap kmap, vmap;
  const uint64_t rows = static_cast<uint64_t>(a.num_pages) * a.n_kv_heads * kPageSize;
  if (make_rows_map(&kmap, a.k_cache, rows, D, kPageSize) != PA_OK) return PA_ERR_CUDA;
  if (make_rows_map(&vmap, a.v_cache, rows, D, kPageSize) != PA_OK) return PA_ERR_CUDA;
  const Layout y = layout_of(a.batch, a.n_q_heads, a.n_kv_heads, D, a.max_blocks, sms);
  char *ws = static_cast<char *>(a.workspace);
  WeightedParams p;
  p.q = static_cast<const uint16_t *>(a.q);
  p.block_table = a.block_table;
  p.ctx_lens = a.ctx_lens;
  p.out = a.out;
  p.weights = a.weights;
  p.states = reinterpret_cast<float *>(ws);
  p.span = reinterpret_cast<int2 *>(ws + y.span);
  p.scores = reinterpret_cast<float *>(ws + y.scores);
  p.status = a.status;
  p.qscale = a.scale * kLog2e;
  p.n_q_heads = a.n_q_heads;
  p.n_kv_heads = a.n_kv_heads;
  p.group = a.n_q_heads / a.n_kv_heads;
  tiles_of(p.group, &p.n_sub, &p.tile_rows);
  p.batch = a.batch;
  p.max_blocks = a.max_blocks;
  p.num_pages = a.num_pages;
  p.fresh = a.fresh;
  // about 16 CTAs an SM if every sequence filled its table, of 256 tokens or more
  const int64_t all = static_cast<int64_t>(a.max_blocks) * kPageSize * a.batch * a.n_kv_heads;
  const int64_t seg = (all / (16 * sms) + 255) / 256 * 256;
  p.seg_tokens = static_cast<int>(seg < 256 ? 256 : seg);
  if (launch_pdl(kern, dim3(sms), dim3(kWarps * 32), WeightedSmem<D>::kAlloc, stream, kmap, vmap,
                 p) != cudaSuccess)
    return PA_ERR_CUDA;
  p.segs = (a.max_blocks * kPageSize + p.seg_tokens - 1) / p.seg_tokens;
  const dim3 grid(static_cast<unsigned>(a.batch) * a.n_kv_heads * p.segs);
  return launch_pdl(weighted_fold_kernel<D>, grid, dim3(kFoldThreads),
                    p.group * sizeof(float2), stream, p) == cudaSuccess
             ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

size_t weighted_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int head_dim,
                                int max_blocks, int sms) {
  return layout_of(batch, n_q_heads, n_kv_heads, head_dim, max_blocks, sms).bytes;
}

int launch_weighted(const WeightedLaunch &a, cudaStream_t stream) {
  if (a.head_dim == 128)
    return a.bf16 ? launch_t<128, true>(a, stream) : launch_t<128, false>(a, stream);
  return a.bf16 ? launch_t<64, true>(a, stream) : launch_t<64, false>(a, stream);
}

}  // namespace pa
