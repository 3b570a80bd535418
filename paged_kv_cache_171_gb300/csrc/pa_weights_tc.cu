// pa_weights_tc.cu -- attention weight that the queries of a chunk give each cached token,
// summed over the queries and over the heads of each kv head's group:
//
//   query i sees keys t <= ctx + i;   p = softmax(q K^T scale)
//   weights[t] = (t < ctx + n_new - fresh ? weights[t] : 0) + sum_{i, h} p[i][h][t]
//
// V is not needed.  Two passes over S = Q K^T on the tensor cores (tcgen05, accumulators
// in tensor memory), because a weight needs its row's final m and l, and S itself, at 4
// bytes a pair, would cost more to store and read than to compute twice.
//   rows pass     S[row][key]: a tile of 128 query rows stays in shared memory, K tiles of
//                 128 keys stream by; a thread owns a row and keeps its running max m and
//                 sum l.  Few rows: the keys are cut into ranges, one (m, l) each.
//   columns pass  S^T[key][row]: a tile of 128 keys stays, the query tiles stream by; a
//                 thread owns a key, so a weight is a sum within one thread, in a fixed
//                 order and without atomics: w += 2^(s - m_row) / l_row.  Each row's
//                 (m, 1 / l) comes from shared memory, the same for all lanes.
// A row is a (query, head) pair of one kv head's group; a query tile is a TMA box of hb
// heads x nq queries, so any group size and any stride of q goes.
//
// One kernel body does both: "held" tiles (HELD of them, one consumer warpgroup each) and
// a ring of streamed tiles.  Warp 0 loads, warp 1 issues the MMAs into two S buffers a
// held tile, warp 2 fetches the rows' (m, 1 / l) for the columns pass, warps 4 .. are the
// consumers.  Every hand-off is an mbarrier; every wait is bounded and gives up early once
// another role has raised the CTA's abort flag.
//
// Bound: the exponentials, two of them a pair (MUFU, 32 a cycle and SM), for chunks of
// many rows; K's bytes for few.
#include <type_traits>

#include "pa_device.cuh"
#include "pa_evict.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;
constexpr float kNoKey = -3.402823466e38f;  // running max of a row before its first key
constexpr int kRows = 128;                  // rows or keys of a tile

struct WeightsParams {
  const int32_t *block_table, *ctx_lens;
  float *weights;
  float2 *stats;  // [sequence x kv head][row tile][range][128]: m (log2), l
  int *status;
  float qscale;   // scale * log2 e
  int n_new, n_kv_heads, group, hb, nq, n_hsub, n_rt, batch, max_blocks, num_pages, fresh;
  int n_ranges;   // key ranges of the rows pass
  int groups;     // held-tile groups a (sequence, kv head) has
};

template <int D, int HELD>
struct WeightsSmem {
  static constexpr int kStages = HELD == 2 ? 4 : 2;
  static constexpr int kColBlk = kRows * 128;          // one 64-column block
  static constexpr int kTile = (D / 64) * kColBlk;
  static constexpr int kHeld = 0;
  static constexpr int kRing = HELD * kTile;
  static constexpr int kM = kRing + kStages * kTile;   // [stage][128]: -m
  static constexpr int kL = kM + kStages * kRows * 4;  // 1 / l
  static constexpr int kLim = kL + kStages * kRows * 4;  // last key the row sees
  static constexpr int kBars = kLim + kStages * kRows * 4;
  static constexpr int kSlot = kBars + 32 * 8;         // TMEM address, abort flag
  static constexpr int kAlloc = kSlot + 16 + 1024;
  static_assert(kAlloc <= 232448, "shared memory of an SM");
};

enum {
  kBarFull = 0,   // ring stage s landed
  kBarFree = 4,   // ring stage s read by the MMAs (commit)
  kBarHeld = 8,   // the held tiles landed
  kBarS = 9,      // S buffer 2 x + (j & 1) complete (commit)
  kBarSFree = 13, // S buffer read (one arrival a consumer warp of x)
  kBarT = 17,     // the rows' (m, 1 / l) of stage s are there
  kBarTFree = 21, // .. have been read (one arrival a consumer warp)
  kBarDrain = 25,
  kNumBars = 26
};

// What a CTA does.
struct Job {
  int b, g, ctx, T;  // T = ctx + n_new
  int held0;         // first held tile: row tile, or key tile
  int s0, n;         // first streamed tile, how many
  int range;
};

// One K tile (8 pages of one kv head) into shared memory.  The whole warp.
template <int D>
__device__ __forceinline__ void load_keys(const CUtensorMap *map, const WeightsParams &p,
                                          const Job &w, int tile, uint32_t dst, uint32_t bar,
                                          int lane) {
  const int n_pages = (w.T + kPageSize - 1) / kPageSize;
  if (lane < 8) {
    const int pg = 8 * tile + lane;
    int id = pg < n_pages ? p.block_table[static_cast<size_t>(w.b) * p.max_blocks + pg] : 0;
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) {
      record_error(p.status, PA_ERR_BAD_BLOCK);
      id = 0;
    }
#pragma unroll
    for (int x = 0; x < D / 64; ++x)
      tma_load_2d(dst + x * kRows * 128 + lane * 2048, map, 64 * x,
                  (id * p.n_kv_heads + w.g) * kPageSize, bar);
  }
  __syncwarp();
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, int u, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_"
      "tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar)
      : "memory");
}

// One tile of query rows: row r = query (rt / n_hsub) nq + r / hb, head (rt % n_hsub) hb +
// r % hb of the group.  Lane 0.
template <int D>
__device__ __forceinline__ void load_queries(const CUtensorMap *map, const WeightsParams &p,
                                             const Job &w, int rt, uint32_t dst, uint32_t bar) {
  const int qt = rt / p.n_hsub, hs = rt - qt * p.n_hsub;
#pragma unroll
  for (int x = 0; x < D / 64; ++x)
    tma_load_4d(dst + x * kRows * 128, map, 64 * x, w.g * p.group + hs * p.hb, qt * p.nq, w.b,
                bar);
}

// Query of row r of tile rt, or -1 past the chunk's end or the tile's rows.
__device__ __forceinline__ int query_of(const WeightsParams &p, int rt, int r) {
  const int q = (rt / p.n_hsub) * p.nq + r / p.hb;
  return r < p.hb * p.nq && q < p.n_new ? q : -1;
}

template <int D, bool BF16, int HELD, bool COLUMNS>
__global__ void __launch_bounds__(128 + 128 * HELD, HELD == 2 ? 1 : 2)
    weights_kernel(const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap, const WeightsParams p) {
  using L = WeightsSmem<D, HELD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) { return sb + L::kBars + 8 * i; };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_release();
  griddep_wait();

  Job w;
  {
    int at = blockIdx.x;
    w.range = COLUMNS ? 0 : at % p.n_ranges;
    if (!COLUMNS) at /= p.n_ranges;
    const int bg = at / p.groups;
    w.held0 = (at - bg * p.groups) * HELD;
    w.b = bg / p.n_kv_heads;
    w.g = bg - w.b * p.n_kv_heads;
    w.ctx = p.ctx_lens[w.b];
    const int most = p.max_blocks * kPageSize - p.n_new;
    if (w.ctx < 0 || w.ctx > most) {
      if (tid == 0) record_error(p.status, PA_ERR_BAD_CTX);
      w.ctx = w.ctx < 0 ? 0 : most;
    }
    w.T = w.ctx + p.n_new;
    if (COLUMNS) {
      if (w.held0 * kRows >= w.T) return;
      // query tiles whose last query sees the first held key
      const int q = max(0, w.held0 * kRows - w.ctx);
      w.s0 = q / p.nq * p.n_hsub;
      w.n = p.n_rt - w.s0;
    } else {
      // key tiles that the held rows see, cut into ranges
      const int last_rt = min(w.held0 + HELD, p.n_rt) - 1;
      const int last_q = min(p.n_new, (last_rt / p.n_hsub + 1) * p.nq) - 1;
      const int tiles = (w.ctx + last_q) / kRows + 1;
      const int per = (tiles + p.n_ranges - 1) / p.n_ranges;
      w.s0 = w.range * per;
      w.n = max(0, min(per, tiles - w.s0));
      if (w.n == 0) {  // nothing of the keys is left for this range
        for (int e = tid; e < HELD * kRows; e += blockDim.x) {
          const int rt = w.held0 + e / kRows;
          if (rt < p.n_rt)
            p.stats[((static_cast<size_t>(bg) * p.n_rt + rt) * p.n_ranges + w.range) * kRows +
                    e % kRows] = make_float2(kNoKey, 0.f);
        }
        return;
      }
    }
  }

  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kSlot + 4);
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bar(i), i >= kBarSFree && i < kBarT ? 4
                        : i >= kBarTFree && i < kBarDrain ? 4 * HELD : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tc::alloc(sb + L::kSlot, 256 * HELD);
    tc::relinquish();
  }
  // Rows of a query tile behind its box are never written by the copies: they hold zeros.
  if (p.hb * p.nq < kRows) {
    const int r0 = p.hb * p.nq, rows = kRows - r0;
    const int first = COLUMNS ? L::kRing : L::kHeld, n = COLUMNS ? L::kStages : HELD;
    for (int e = tid; e < n * (D / 64) * rows * 8; e += blockDim.x) {
      const int blk = e / (rows * 8), in = e - blk * rows * 8;
      st_shared_v4(sb + first + blk * L::kColBlk + (r0 + in / 8) * 128 + (in % 8) * 16, 0u, 0u,
                   0u, 0u);
    }
    fence_proxy_async_smem();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kSlot);
  const uint32_t q_bytes = (D / 64) * p.hb * p.nq * 128;

  if (warp == 0) {
    // ---- loads: the held tiles, then the ring
    bool ok = true;
    if (lane == 0) mbar_arrive_expect_tx(bar(kBarHeld), HELD * (COLUMNS ? L::kTile : q_bytes));
    __syncwarp();
    for (int x = 0; x < HELD; ++x) {
      const uint32_t dst = sb + L::kHeld + x * L::kTile;
      if (COLUMNS)
        load_keys<D>(&kmap, p, w, w.held0 + x, dst, bar(kBarHeld), lane);
      else if (lane == 0)
        // (a row tile past the last one reads it again; its rows are dropped)
        load_queries<D>(&qmap, p, w, min(w.held0 + x, p.n_rt - 1), dst, bar(kBarHeld));
    }
    int j = 0;
    for (; j < w.n; ++j) {
      const int s = j % L::kStages;
      if (j >= L::kStages &&
          !(ok = warp_wait(bar(kBarFree + s), ((j / L::kStages) - 1) & 1, abort_flag)))
        break;
      if (lane == 0) mbar_arrive_expect_tx(bar(kBarFull + s), COLUMNS ? q_bytes : L::kTile);
      __syncwarp();
      const uint32_t dst = sb + L::kRing + s * L::kTile;
      if (!COLUMNS)
        load_keys<D>(&kmap, p, w, w.s0 + j, dst, bar(kBarFull + s), lane);
      else if (lane == 0)
        load_queries<D>(&qmap, p, w, w.s0 + j, dst, bar(kBarFull + s));
    }
    if (!ok) {
      if (lane == 0) raise_abort(p.status, abort_flag);
      mbar_wait(bar(kBarHeld), 0);  // copies in flight still land
      for (int t = max(0, j - L::kStages); t < j; ++t)
        mbar_wait(bar(kBarFull + t % L::kStages), (t / L::kStages) & 1);
    }
  } else if (warp == 1) {
    // ---- S of every held tile against each streamed one
    constexpr uint32_t kId = tc::idesc_f16(BF16, kRows, kRows, false, false);
    const uint64_t held = tc::smem_desc_sw128(sb + L::kHeld, 16, 1024);
    const uint64_t ring = tc::smem_desc_sw128(sb + L::kRing, 16, 1024);
    bool ok = warp_wait(bar(kBarHeld), 0, abort_flag);
    for (int j = 0; j < w.n && ok; ++j) {
      const int s = j % L::kStages;
      if (!(ok = warp_wait(bar(kBarFull + s), (j / L::kStages) & 1, abort_flag))) break;
      for (int x = 0; x < HELD && ok; ++x) {
        const int buf = 2 * x + (j & 1);
        if (j >= 2 && !(ok = warp_wait(bar(kBarSFree + buf), ((j >> 1) - 1) & 1, abort_flag)))
          break;
        tc::fence_after_sync();
        if (lane == 0) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t off = ((k >> 2) * L::kColBlk + (k & 3) * 32) >> 4;
            tc::mma_f16(tmem + buf * kRows, held + ((x * L::kTile) >> 4) + off,
                        ring + ((s * L::kTile) >> 4) + off, kId, k > 0);
          }
          tc::commit(bar(kBarS + buf));
          if (x == HELD - 1) tc::commit(bar(kBarFree + s));
        }
        __syncwarp();
      }
    }
    if (!ok) {
      if (lane == 0) {
        raise_abort(p.status, abort_flag);
        tc::commit(bar(kBarDrain));
      }
      __syncwarp();
      mbar_wait(bar(kBarDrain), 0);
    }
  } else if (COLUMNS && warp == 2) {
    // ---- (-m, 1 / l) of the streamed tiles' rows, and the last key each one sees
    float *sm = reinterpret_cast<float *>(smem + L::kM);
    float *sl = reinterpret_cast<float *>(smem + L::kL);
    int *slim = reinterpret_cast<int *>(smem + L::kLim);
    const float2 *stats =
        p.stats + static_cast<size_t>(w.b * p.n_kv_heads + w.g) * p.n_rt * p.n_ranges * kRows;
    bool ok = true;
    for (int j = 0; j < w.n; ++j) {
      const int s = j % L::kStages, rt = w.s0 + j;
      if (j >= L::kStages &&
          !(ok = warp_wait(bar(kBarTFree + s), ((j / L::kStages) - 1) & 1, abort_flag)))
        break;
#pragma unroll
      for (int k = 0; k < kRows / 32; ++k) {
        const int r = lane + 32 * k, q = query_of(p, rt, r);
        const float2 *st = stats + static_cast<size_t>(rt) * p.n_ranges * kRows + r;
        float m = kNoKey, l = 0.f;
        if (q >= 0)
          for (int i = 0; i < p.n_ranges; ++i) {
            const float2 v = st[i * kRows];
            const float mn = fmaxf(m, v.x);
            l = l * ex2(m - mn) + v.y * ex2(v.x - mn);
            m = mn;
          }
        sm[s * kRows + r] = q >= 0 ? -m : 0.f;
        sl[s * kRows + r] = l == 0.f ? 0.f : 1.f / l;
        slim[s * kRows + r] = w.ctx + q;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarT + s));
    }
    if (!ok && lane == 0) raise_abort(p.status, abort_flag);
  } else if (warp >= 4) {
    // ---- consumers: lane r of held tile x is a row, or a key
    const int x = (warp - 4) >> 2, r = ((warp & 3) << 5) + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float qs = p.qscale;
    bool ok = true;
    if constexpr (!COLUMNS) {
      const int rt = w.held0 + x;
      const int q = query_of(p, rt, r);
      const int lim = w.ctx + max(q, 0);                            // last key row r sees
      const int lim_all = w.ctx + min(rt / p.n_hsub * p.nq, p.n_new - 1);  // every row of x does
      float m = kNoKey;
      float2 l2 = make_float2(0.f, 0.f);
      for (int j = 0; j < w.n; ++j) {
        const int buf = 2 * x + (j & 1);
        if (!(ok = warp_wait(bar(kBarS + buf), (j >> 1) & 1, abort_flag))) break;
        tc::fence_after_sync();
        uint32_t s[kRows];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tc::ld32(tmem + buf * kRows + lanes + 32 * c,
                   *reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
        tc::wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarSFree + buf));
        const int key0 = (w.s0 + j) * kRows;
        float cand;
        // the maximum of s qs (a negative scale: from the least s); masked keys never win
        auto extreme = [&](auto pick, float worst) {
          if (key0 + kRows - 1 > lim_all) {
            const int last = lim - key0;
#pragma unroll
            for (int c = 0; c < kRows; ++c)
              if (c > last) s[c] = __float_as_uint(worst);
          }
          float t0 = worst, t1 = worst, t2 = worst, t3 = worst;
#pragma unroll
          for (int c = 0; c < kRows; c += 8) {
            t0 = pick(t0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
            t1 = pick(t1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
            t2 = pick(t2, __uint_as_float(s[c + 4]), __uint_as_float(s[c + 5]));
            t3 = pick(t3, __uint_as_float(s[c + 6]), __uint_as_float(s[c + 7]));
          }
          return pick(pick(t0, t1, t2), t3, t3);
        };
        if (qs >= 0.f)
          cand = extreme([](float a, float b, float c) { return max3(a, b, c); }, -INFINITY);
        else
          cand = extreme([](float a, float b, float c) { return fminf(fminf(a, b), c); }, INFINITY);
        cand *= qs;  // (qs = 0: 0, or NaN where no key was seen)
        if (cand > m + kSlack) {
          const float corr = ex2(m - cand);
          m = cand;
          l2 = __fmul2_rn(l2, make_float2(corr, corr));
        }
        const float2 qs2 = make_float2(qs, qs), nm2 = make_float2(-m, -m);
        float2 e2 = make_float2(0.f, 0.f), f2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kRows; c += 4) {
          const float2 a = __ffma2_rn(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
                                      qs2, nm2);
          const float2 b = __ffma2_rn(
              make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), qs2, nm2);
          e2 = __fadd2_rn(e2, make_float2(ex2(a.x), ex2(a.y)));
          f2 = __fadd2_rn(f2, make_float2(ex2(b.x), ex2(b.y)));
        }
        l2 = __fadd2_rn(l2, __fadd2_rn(e2, f2));
      }
      if (ok && rt < p.n_rt)
        p.stats[((static_cast<size_t>(w.b * p.n_kv_heads + w.g) * p.n_rt + rt) * p.n_ranges +
                 w.range) * kRows + r] = make_float2(m, l2.x + l2.y);
    } else {
      const int key = (w.held0 + x) * kRows + r;
      const int key_end = (w.held0 + x) * kRows + kRows - 1;
      float2 sum = make_float2(0.f, 0.f);
      for (int j = 0; j < w.n; ++j) {
        const int buf = 2 * x + (j & 1), st = j % L::kStages, rt = w.s0 + j;
        if (!(ok = warp_wait2(bar(kBarS + buf), (j >> 1) & 1, bar(kBarT + st),
                              (j / L::kStages) & 1, abort_flag)))
          break;
        tc::fence_after_sync();
        // every row of the tile sees every key of this one?
        const bool all = key_end <= w.ctx + rt / p.n_hsub * p.nq;
        const uint32_t am = sb + L::kM + st * kRows * 4, al = sb + L::kL + st * kRows * 4;
        const uint32_t alim = sb + L::kLim + st * kRows * 4;
        float2 part = make_float2(0.f, 0.f), other = make_float2(0.f, 0.f);
        const float2 qs2 = make_float2(qs, qs);
#pragma unroll
        for (int c0 = 0; c0 < kRows; c0 += 32) {
          uint32_t s[32];
          tc::ld32(tmem + buf * kRows + lanes + c0, s);
          tc::wait_ld();
          if (c0 == kRows - 32) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarSFree + buf));
          }
          auto add = [&](auto masked) {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const uint4 m4 = lds128(am + (c0 + c) * 4), l4 = lds128(al + (c0 + c) * 4);
              const float2 a = __ffma2_rn(
                  make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), qs2,
                  make_float2(__uint_as_float(m4.x), __uint_as_float(m4.y)));
              const float2 b = __ffma2_rn(
                  make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), qs2,
                  make_float2(__uint_as_float(m4.z), __uint_as_float(m4.w)));
              float2 ea = make_float2(ex2(a.x), ex2(a.y)), eb = make_float2(ex2(b.x), ex2(b.y));
              if constexpr (decltype(masked)::value) {
                const uint4 k4 = lds128(alim + (c0 + c) * 4);
                if (key > static_cast<int>(k4.x)) ea.x = 0.f;
                if (key > static_cast<int>(k4.y)) ea.y = 0.f;
                if (key > static_cast<int>(k4.z)) eb.x = 0.f;
                if (key > static_cast<int>(k4.w)) eb.y = 0.f;
              }
              part = __ffma2_rn(ea, make_float2(__uint_as_float(l4.x), __uint_as_float(l4.y)),
                                part);
              other = __ffma2_rn(eb, make_float2(__uint_as_float(l4.z), __uint_as_float(l4.w)),
                                 other);
            }
          };
          if (all)
            add(std::false_type{});
          else
            add(std::true_type{});
        }
        sum = __fadd2_rn(sum, __fadd2_rn(part, other));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarTFree + st));
      }
      if (ok && key < w.T) {
        const int page =
            p.block_table[static_cast<size_t>(w.b) * p.max_blocks + key / kPageSize];
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) {  // else reported
          float *dst = p.weights + (static_cast<size_t>(page) * p.n_kv_heads + w.g) * kPageSize +
                       key % kPageSize;
          *dst = (key < w.T - p.fresh ? *dst : 0.f) + (sum.x + sum.y);
        }
      }
    }
    if (!ok && lane == 0) raise_abort(p.status, abort_flag);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::dealloc(tmem, 256 * HELD);
  }
}

struct Plan {
  int hb, nq, n_hsub, n_rt, ranges;
};
// Row tiles of a kv head's rows, and the key ranges that give about every SM a CTA of two
// of them.
Plan plan_of(int batch, int n_new, int n_q_heads, int n_kv_heads, int sms) {
  const int group = n_q_heads / n_kv_heads;
  Plan y;
  y.hb = group;
  if (y.hb > kRows)  // the largest divisor that fits a tile
    for (y.hb = kRows; group % y.hb; --y.hb) {
    }
  y.n_hsub = group / y.hb;
  y.nq = kRows / y.hb;
  y.n_rt = y.n_hsub * ((n_new + y.nq - 1) / y.nq);
  const int64_t ctas = static_cast<int64_t>(batch) * n_kv_heads * ((y.n_rt + 1) / 2);
  const int64_t r = sms / ctas;
  y.ranges = static_cast<int>(r < 1 ? 1 : r > 64 ? 64 : r);
  return y;
}

template <int D, bool BF16, int HELD, bool COLUMNS>
int launch_pass(const CUtensorMap &qmap, const CUtensorMap &kmap, const WeightsParams &p,
                int64_t ctas, cudaStream_t stream) {
  using L = WeightsSmem<D, HELD>;
  auto kern = weights_kernel<D, BF16, HELD, COLUMNS>;
  static ContextCache<bool> smem_set;
  if (set_smem_limit(kern, L::kAlloc, smem_set) != PA_OK) return PA_ERR_CUDA;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(128 + 128 * HELD), L::kAlloc,
                    stream, qmap, kmap, p) == cudaSuccess
             ? PA_OK : PA_ERR_CUDA;
}

template <int D, bool BF16>
int launch_t(const WeightsLaunch &a, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  const Plan y = plan_of(a.batch, a.n_new, a.n_q_heads, a.n_kv_heads, sms);
  CUtensorMap qmap, kmap;
  const uint64_t rows = static_cast<uint64_t>(a.num_pages) * a.n_kv_heads * kPageSize;
  if (make_rows_map(&kmap, a.k_cache, rows, D, kPageSize) != PA_OK) return PA_ERR_CUDA;
  if (make_query_map(&qmap, a.q, D, a.n_q_heads, a.n_new, a.batch, a.q_token_stride,
                     a.q_batch_stride, y.hb, y.nq) != PA_OK)
    return PA_ERR_CUDA;
  WeightsParams p;
  p.block_table = a.block_table;
  p.ctx_lens = a.ctx_lens;
  p.weights = a.weights;
  p.stats = static_cast<float2 *>(a.workspace);
  p.status = a.status;
  // (a zero scale becomes a factor small enough that every weight is the same: a masked
  // score, -inf, times zero would be NaN)
  p.qscale = a.scale * kLog2e;
  if (fabsf(p.qscale) < 1e-30f) p.qscale = a.scale < 0.f ? -1e-30f : 1e-30f;
  p.n_new = a.n_new;
  p.n_kv_heads = a.n_kv_heads;
  p.group = a.n_q_heads / a.n_kv_heads;
  p.hb = y.hb;
  p.nq = y.nq;
  p.n_hsub = y.n_hsub;
  p.n_rt = y.n_rt;
  p.batch = a.batch;
  p.max_blocks = a.max_blocks;
  p.num_pages = a.num_pages;
  p.fresh = a.fresh;
  p.n_ranges = y.ranges;
  const int64_t lists = static_cast<int64_t>(a.batch) * a.n_kv_heads;
  p.groups = (y.n_rt + 1) / 2;
  int rc = launch_pass<D, BF16, 2, false>(qmap, kmap, p, lists * p.groups * p.n_ranges, stream);
  if (rc) return rc;
  // few query tiles: one key tile a CTA and two CTAs an SM, so that one's start overlaps
  // the other's work; many: two key tiles, which halves what the query tiles cost L2
  const int key_tiles = (a.max_blocks * kPageSize + kRows - 1) / kRows;
  if (y.n_rt <= 4) {
    p.groups = key_tiles;
    return launch_pass<D, BF16, 1, true>(qmap, kmap, p, lists * p.groups, stream);
  }
  p.groups = (key_tiles + 1) / 2;
  return launch_pass<D, BF16, 2, true>(qmap, kmap, p, lists * p.groups, stream);
}

}  // namespace

size_t weights_workspace_bytes(int batch, int n_new, int n_q_heads, int n_kv_heads, int sms) {
  const Plan y = plan_of(batch, n_new, n_q_heads, n_kv_heads, sms);
  return static_cast<size_t>(batch) * n_kv_heads * y.n_rt * y.ranges * kRows * sizeof(float2);
}

int launch_weights(const WeightsLaunch &a, cudaStream_t stream) {
  if (a.head_dim == 128)
    return a.bf16 ? launch_t<128, true>(a, stream) : launch_t<128, false>(a, stream);
  return a.bf16 ? launch_t<64, true>(a, stream) : launch_t<64, false>(a, stream);
}

}  // namespace pa
