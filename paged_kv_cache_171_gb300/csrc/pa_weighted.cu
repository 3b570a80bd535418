// pa_weighted.cu -- decode attention that also gathers, for every cached token and kv
// head, the attention weight the step's queries gave it.
//
//   s_t = scale q_h . k_t,  p_h[t] = e^(s_t - m) / l,  out_h = sum_t p_h[t] v_t
//   weights[t] = (t < T - fresh ? weights[t] : 0) + sum_{h in the kv head's group} p_h[t]
//
// A weight needs the row's final m and l, which no CTA has before the last key.  So the
// pass over K and V stores each score (4 bytes a query head and token beside the 4 D
// bytes a kv head and token of K and V), a second, short kernel folds the rows' partial
// states into (m, l) and out, and a third reads the scores back, mostly from L2, and adds
// e^(s - m) / l over the group.  Reading K again instead would cost 2 D bytes a token
// and kv head: 32 to 256 bytes against 8 a query head.
//
// Operand form.  mma.sync m16n8k16 with the tokens (then the head dimensions) as the 16
// rows and up to 8 query rows as the columns: S = K Q^T straight from the page's tile by
// ldmatrix, O = V^T P by its transposing form, P from the accumulators by movmatrix.  The
// weights p enter as bf16 in three terms (24 bits) or as fp16 in two (22 bits, of 2^13 p,
// so down to 2^-38 of the row's largest; p is at most 2^2 there, 2^8 in bf16): one term would
// leave up to 2^-8 or 2^-11 of every weight in an fp32 result.  The normaliser takes the
// weights of 16 pages at a time: added one by one to a sum that holds an attention sink's,
// weights 14 to 17 nats below it round to whole last places of that sum (2e-4 of the result
// over 32768 keys, now 4e-6).  A page's sum has an accumulator of its own that a rounding add
// joins to the state, because the tensor cores' sums round toward zero.
//
// Work split.  The pages of all (sequence, kv head, tile of 8 query rows) items, laid end
// to end, are cut into equal runs, one a warp: eight warps an SM, each with a ring of
// pages (K and V, 2-D TMA, 128-byte swizzle) that it feeds itself across item borders.
// An item cut between warps leaves a partial state a warp; states are numbered item +
// warp, which grows along the list, so that the second kernel finds an item's in order
// and results do not depend on timing.
//
// Bound: memory.  64 sequences of 128 to 8192 tokens, 32/8 heads of 128: 201 us, of which
// 179 are the pass over K and V (6.1 TB/s with the scores it writes), 9 the fold and 13 the
// weights.  4 x 32768, 64/8 heads: 110 us (92, 6 and 11).
#include "pa_device.cuh"
#include "pa_evict.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kNoKey = -3.402823466e38f;  // running max of a row before its first key
constexpr int kWarps = 8;                   // a CTA, one CTA an SM
constexpr int kTile = 8;                    // query rows a tile
constexpr int kMinPages = 2;                // least pages a run has
constexpr int kSumPages = 16;               // whose weights are summed before they join l
constexpr int kFoldThreads = 256;           // of the second and third kernel
constexpr int kFoldTokens = 512;            // of the third, a round
constexpr int kFoldElements = 32;           // of the second, a CTA

struct WeightedParams {
  const uint16_t *q;
  const int32_t *block_table, *ctx_lens;
  float *out, *weights;
  float *states;  // [item + warp][kTile][D + 4]: O, m (log2), l
  int2 *span;     // [item]: first and last warp that holds a part of it
  float2 *rows;   // [sequence][query head]: m, 1 / l
  float *scores;  // per tile [T][rows], tiles at (first row) * max_tokens
  int *status;
  float qscale;   // scale * log2 e
  int n_q_heads, n_kv_heads, group, n_sub, tile_rows, batch, max_blocks, num_pages, fresh;
  int workers;           // warps of the first kernel
  int parts;             // CTAs a list of the second kernel
  int seg_tokens, segs;  // tokens a CTA of the third looks after, CTAs a list
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
  // How far (log2) scores may pass the reference; fp16's weights fill its range above that.
  // (Slack 0 to 8 in fp16: the same time.  2^7 p left 1e-4 behind a sink 17 nats above 32768 keys.)
  constexpr int kSlack = BF16 ? 8 : 2;
  constexpr float kLift = BF16 ? 1.f : static_cast<float>(1 << (15 - kSlack));
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ln = lane >> 2, lc = lane & 3;
  const int n_workers = p.workers, worker = warp * gridDim.x + blockIdx.x;
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
    float2 some = make_float2(0.f, 0.f);  // of up to kSumPages pages, then part of l
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
      if (__any_sync(kFull, grow > kSlack)) {
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
        some = __fmul2_rn(some, c);
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
        some = __fadd2_rn(some, w);
        if (!BF16) w = make_float2(w.x * kLift, w.y * kLift);
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
      if (i % kSumPages == kSumPages - 1) {
        l = __fadd2_rn(l, some);
        some = make_float2(0.f, 0.f);
      }
      __syncwarp();  // the stage has been read by every lane
      issue();
    }
    l = __fadd2_rn(l, some);

    // ---- the part's state
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l.x += __shfl_xor_sync(kFull, l.x, x);
      l.y += __shfl_xor_sync(kFull, l.y, x);
    }
    float *state = p.states + (static_cast<size_t>(item) + worker) * (kTile * (D + 4));
    constexpr float down = 1.f / kLift;
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

// Folds the states of a list's (sequence x kv head's) elements [e0, e1): an element is four
// dimensions of a row.  Eight neighbouring threads go over its states, eight loads ahead of
// the arithmetic, and join theirs by shuffles; no barrier.  out gets O / l, `rows` the (m, 1 / l)
// of rows whose first element is among these.
template <int D>
__device__ __forceinline__ void fold_elements(const WeightedParams &p, int bg, int e0, int e1,
                                              float2 *rows) {
  constexpr int kOver = 8, kAhead = 4;
  // The warps that hold an item.  Where one gave up, the place was not written: whatever it
  // holds stays within the states.
  auto span_of = [&](int item) {
    const int2 s = p.span[item];
    return make_int2(max(s.x, 0), min(s.y, p.workers - 1));
  };
  const int2 first_span = span_of(bg * p.n_sub);
  for (int eb = e0; eb < e1; eb += kFoldThreads / kOver) {
    const int e = eb + threadIdx.x / kOver;
    const bool real = e < e1;
    const int r = real ? e / (D / 4) : e0 / (D / 4), d = 4 * (e % (D / 4));
    const int sub = p.n_sub == 1 ? 0 : r / p.tile_rows, rr = r - sub * p.tile_rows;
    const int item = bg * p.n_sub + sub;
    const int2 span = p.n_sub == 1 ? first_span : span_of(item);
    const float *states = p.states + (static_cast<size_t>(item) * kTile + rr) * (D + 4);
    float m = kNoKey, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto join = [&](float mo, float lo, float4 v) {
      const float mn = fmaxf(m, mo), a = ex2(m - mn), f = ex2(mo - mn);
      l = fmaf(lo, f, l * a);
      acc.x = fmaf(v.x, f, acc.x * a);
      acc.y = fmaf(v.y, f, acc.y * a);
      acc.z = fmaf(v.z, f, acc.z * a);
      acc.w = fmaf(v.w, f, acc.w * a);
      m = mn;
    };
    for (int c = span.x + threadIdx.x % kOver; c <= span.y; c += kOver * kAhead) {
      float2 ml[kAhead];
      float4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {  // past the last state, it again
        const float *s =
            states + static_cast<size_t>(min(c + u * kOver, span.y)) * kTile * (D + 4);
        ml[u] = *reinterpret_cast<const float2 *>(s + D);
        v[u] = *reinterpret_cast<const float4 *>(s + d);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (c + u * kOver <= span.y) join(ml[u].x, ml[u].y, v[u]);
    }
#pragma unroll
    for (int x = kOver / 2; x > 0; x >>= 1) {
      float4 v;
      const float mo = __shfl_xor_sync(kFull, m, x), lo = __shfl_xor_sync(kFull, l, x);
      v.x = __shfl_xor_sync(kFull, acc.x, x);
      v.y = __shfl_xor_sync(kFull, acc.y, x);
      v.z = __shfl_xor_sync(kFull, acc.z, x);
      v.w = __shfl_xor_sync(kFull, acc.w, x);
      join(mo, lo, v);
    }
    if (!real || threadIdx.x % kOver != 0) continue;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (d == 0) rows[r] = make_float2(m, inv);
    *reinterpret_cast<float4 *>(p.out + (static_cast<size_t>(bg) * p.group + r) * D + d) =
        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  }
}

// Adds the group's weights for the tokens of a list's segment, two tokens a thread, so that
// the two rounds of loads (page and scores; old weight) are covered by many threads.
// NR: rows of a kv head where all of them are one tile of 1, 2, 4 or 8, else 0.
template <int NR>
__device__ __forceinline__ void add_tokens(const WeightedParams &p, int bg, int seg,
                                           const float2 *rows) {
  constexpr int U = kFoldTokens / kFoldThreads;  // tokens a thread
  const int b = bg / p.n_kv_heads, g = bg - b * p.n_kv_heads;
  const int32_t *table = p.block_table + static_cast<size_t>(b) * p.max_blocks;
  const size_t max_tokens = static_cast<size_t>(p.max_blocks) * kPageSize;
  const size_t row0 = static_cast<size_t>(bg) * p.group;
  const int tokens = tokens_of(p, b, false);
  const int t1 = min(tokens, (seg + 1) * p.seg_tokens);
  for (int t0 = seg * p.seg_tokens; t0 < t1; t0 += kFoldTokens) {
    int page[U];
    float sc[U][NR > 0 ? NR : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + threadIdx.x + kFoldThreads * u;
      page[u] = t < t1 ? table[t / kPageSize] : -1;
      if constexpr (NR > 0) {
        if (t >= t1) continue;
        const float *s = p.scores + row0 * max_tokens + static_cast<size_t>(t) * NR;
        if constexpr (NR == 1) {
          sc[u][0] = s[0];
        } else if constexpr (NR == 2) {
          const float2 v = *reinterpret_cast<const float2 *>(s);
          sc[u][0] = v.x, sc[u][1] = v.y;
        } else {
#pragma unroll
          for (int r = 0; r < NR; r += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(s + r);
            sc[u][r] = v.x, sc[u][r + 1] = v.y, sc[u][r + 2] = v.z, sc[u][r + 3] = v.w;
          }
        }
      }
    }
    float *dst[U];
    float sum[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + threadIdx.x + kFoldThreads * u;
      dst[u] = nullptr;
      sum[u] = 0.f;
      if (static_cast<unsigned>(page[u]) < static_cast<unsigned>(p.num_pages)) {
        dst[u] = p.weights + (static_cast<size_t>(page[u]) * p.n_kv_heads + g) * kPageSize +
                 t % kPageSize;  // (a bad page has been reported)
        if (t < tokens - p.fresh) sum[u] = *dst[u];
      }
    }
    float add[U];
#pragma unroll
    for (int u = 0; u < U; ++u) add[u] = 0.f;
    if constexpr (NR > 0) {
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float2 row = rows[r];
#pragma unroll
        for (int u = 0; u < U; ++u) add[u] += ex2(sc[u][r] - row.x) * row.y;
      }
    } else {
      for (int r0 = 0; r0 < p.group; r0 += p.tile_rows) {
        const int n_r = min(p.tile_rows, p.group - r0);
        for (int r = 0; r < n_r; ++r) {
          const float2 row = rows[r0 + r];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int t = t0 + threadIdx.x + kFoldThreads * u;
            if (dst[u])
              add[u] += ex2(p.scores[(row0 + r0) * max_tokens + static_cast<size_t>(t) * n_r + r] -
                            row.x) * row.y;
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dst[u]) *dst[u] = sum[u] + add[u];
  }
}

// The second and third kernel: CTA (list, part of its elements), CTA (list, segment).
template <int D>
__global__ void __launch_bounds__(kFoldThreads) weighted_fold_kernel(const WeightedParams p) {
  griddep_release();
  griddep_wait();  // the states
  const int bg = blockIdx.x / p.parts, part = blockIdx.x - bg * p.parts, n = p.group * (D / 4);
  fold_elements<D>(p, bg, part * kFoldElements, min(n, (part + 1) * kFoldElements),
                   p.rows + static_cast<size_t>(bg) * p.group);
}
template <int NR>
__global__ void __launch_bounds__(kFoldThreads) weighted_add_kernel(const WeightedParams p) {
  griddep_release();
  griddep_wait();  // the rows and the scores
  const int bg = blockIdx.x / p.segs;
  add_tokens<NR>(p, bg, blockIdx.x - bg * p.segs, p.rows + static_cast<size_t>(bg) * p.group);
}

// Both in one, a CTA a list: tables of two rounds at most.  A launch less: the host's call
// bounds those (1 x 512 tokens of 16 heads, calls on end: 15.0 us apart, 12.5 in one).
template <int D, int NR>
__global__ void __launch_bounds__(kFoldThreads) weighted_both_kernel(const WeightedParams p) {
  griddep_release();
  griddep_wait();
  float2 *rows = p.rows + static_cast<size_t>(blockIdx.x) * p.group;
  fold_elements<D>(p, blockIdx.x, 0, p.group * (D / 4), rows);
  __syncthreads();
  add_tokens<NR>(p, blockIdx.x, 0, rows);
}

// Row tiles of a group: as few as there can be, of nearly equal size.
void tiles_of(int group, int *n_sub, int *rows) {
  *n_sub = (group + kTile - 1) / kTile;
  *rows = (group + *n_sub - 1) / *n_sub;
  *n_sub = (group + *rows - 1) / *rows;
}

struct Layout {
  size_t span, rows, scores, bytes;
};
Layout layout_of(int batch, int n_q_heads, int n_kv_heads, int head_dim, int max_blocks,
                 int sms) {
  int n_sub, rows;
  tiles_of(n_q_heads / n_kv_heads, &n_sub, &rows);
  const size_t items = static_cast<size_t>(batch) * n_kv_heads * n_sub;
  Layout y;
  y.span = (items + static_cast<size_t>(sms) * kWarps) * kTile * (head_dim + 4) * sizeof(float);
  y.rows = (y.span + items * sizeof(int2) + 15) & ~size_t(15);
  y.scores = (y.rows + static_cast<size_t>(batch) * n_q_heads * sizeof(float2) + 15) & ~size_t(15);
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
  p.rows = reinterpret_cast<float2 *>(ws + y.rows);
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
  // a round of tokens a CTA, more where full tables would make it over 128 CTAs an SM
  const int64_t lists = static_cast<int64_t>(a.batch) * a.n_kv_heads;
  const int64_t rounds = (static_cast<int64_t>(a.max_blocks) * kPageSize + kFoldTokens - 1) /
                         kFoldTokens;
  const int64_t most = 128 * sms / lists > 1 ? 128 * sms / lists : 1;  // CTAs a list
  const bool both = rounds <= 2;
  p.workers = sms * kWarps;
  p.seg_tokens = static_cast<int>(both ? rounds : (rounds + most - 1) / most) * kFoldTokens;
  p.segs = (a.max_blocks * kPageSize + p.seg_tokens - 1) / p.seg_tokens;
  p.parts = (p.group * (D / 4) + kFoldElements - 1) / kFoldElements;
  if (launch_pdl(kern, dim3(sms), dim3(kWarps * 32), WeightedSmem<D>::kAlloc, stream, kmap, vmap,
                 p) != cudaSuccess)
    return PA_ERR_CUDA;
  const int rows_known = p.n_sub == 1 ? p.group : 0;
  const dim3 block(kFoldThreads);
  if (both) {
    auto kern2 = rows_known == 8 ? weighted_both_kernel<D, 8>
                 : rows_known == 4 ? weighted_both_kernel<D, 4>
                 : rows_known == 2 ? weighted_both_kernel<D, 2>
                 : rows_known == 1 ? weighted_both_kernel<D, 1> : weighted_both_kernel<D, 0>;
    return launch_pdl(kern2, dim3(static_cast<unsigned>(lists)), block, 0, stream, p) ==
                   cudaSuccess ? PA_OK : PA_ERR_CUDA;
  }
  if (launch_pdl(weighted_fold_kernel<D>, dim3(static_cast<unsigned>(lists) * p.parts), block, 0,
                 stream, p) != cudaSuccess)
    return PA_ERR_CUDA;
  auto add = rows_known == 8 ? weighted_add_kernel<8>
             : rows_known == 4 ? weighted_add_kernel<4>
             : rows_known == 2 ? weighted_add_kernel<2>
             : rows_known == 1 ? weighted_add_kernel<1> : weighted_add_kernel<0>;
  return launch_pdl(add, dim3(static_cast<unsigned>(lists) * p.segs), block, 0, stream, p) ==
                 cudaSuccess ? PA_OK : PA_ERR_CUDA;
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
