// pa_weights_tc.cu -- attention weight that the queries of a chunk give each cached token,
// summed over the queries and over the heads of each kv head's group:
//
//   query i sees keys t <= ctx + i;   p = softmax(q K^T scale)
//   weights[t] = (t < ctx + n_new - fresh ? weights[t] : 0) + sum_{i, h} p[i][h][t]
//
// V is not needed.  Two passes over S = Q K^T on the tensor cores (tcgen05, accumulators
// in tensor memory), because a weight needs its row's final m and l, and S itself, at 4
// bytes a pair, would cost more to store and read than to compute twice.
//   rows pass     S[row][key]: four tiles of 128 query rows are held in shared memory, K
//                 tiles of 128 keys stream by; a thread owns a row and keeps its running
//                 max m and sum l.  Few rows: the keys are cut into ranges, one (m, l) each.
//   columns pass  S^T[key][row]: a thread owns a key and sums 2^(s - lse_row), lse = m +
//                 log2 l, over the rows, in a fixed order and without atomics; the rows'
//                 lse come from shared memory, the same for all lanes.  Up to four row tiles
//                 (FEW): they are held and the keys stream, each once.  More (MANY): two key
//                 tiles are held, the row tiles stream, and a CTA goes from one pair of key
//                 tiles to the next.
// A row is a (query, head) pair of one kv head's group; a row tile is a TMA box of hb heads x
// nq queries, so any group size and any stride of q goes.
//
// Roles: warp 0 loads, warp 1 issues the MMAs, warps 4-19 are four consumer warpgroups, warps
// 2 and 3 add the columns pass's partial sums and update the pool.  Work reaches the consumers
// in chunks of 128 x 128 scores, which they read 64 columns at a time, so that a chunk's buffer
// in tensor memory is free again before its last scores have been worked off.  FEW: chunks go
// to the four warpgroups in turn, whatever their row tile (half a chunk each, in two pairs of
// warpgroups, pays each hand-off twice: 2 x 33 tokens of 64/8 heads over 32k 62 us, whole ones
// 42).  Rows pass: a warpgroup a row tile, or, of one or two row tiles, four or two in turn
// (128 and 256 rows over 32k: 67 -> 61 and 78 -> 71 us for both passes).  MANY: all four take
// 32 rows of both held key tiles (a load of lse then serves two keys).
// Rows that only fill a tile up cost no exponentials.  Every hand-off is an mbarrier; every
// wait is bounded and gives up early once another role has raised the CTA's abort flag.
//
// Bound: the exponentials, two of them a pair (MUFU), and the MMAs, about as long, for chunks
// of many rows: 4 x 512 tokens of 32/8 heads over 8192, 246 us (rows pass 119, columns pass
// 129), the exponential pipe busy 51 to 60% of the cycles and the tensor pipe 50 to 59%.  For
// few rows the same two with every hand-off in sight: 2 x 33 tokens of 64/8 heads over 32k,
// 89 us (44 and 44) for 134 MB of K read twice.
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
constexpr int kThreads = 640;
constexpr int kGroups = 4;                  // consumer warpgroups
constexpr int kNumBars = 36;
enum Pass { kRowsPass, kFew, kMany };

struct WeightsParams {
  const int32_t *block_table, *ctx_lens;
  float *weights;
  float2 *states;  // [sequence x kv head][row tile][range][128]: m (log2), l
  float *stats;    // [sequence x kv head][row tile][128]: -(m + log2 l), -inf for no row
  int *status;
  float qscale;    // |scale| * log2 e
  uint32_t negate; // bit of the instruction descriptor that turns the first operand's sign
  int n_new, n_kv_heads, group, hb, nq, n_hsub, n_rt, batch, max_blocks, num_pages, fresh;
  int n_ranges;    // key ranges of the rows pass
  int key_ranges;  // of the columns pass (FEW)
  int groups;      // row tile groups (rows pass), key tile pairs (MANY) of a list
  int items;       // lists x groups (MANY)
};

template <int D, int PASS>
struct WeightsSmem {
  static constexpr int kHeldTiles = PASS == kMany ? 2 : 4;
  // of the ring; held row tiles that there are not make room for more (up to 4)
  static constexpr int kStages = D == 128 && PASS != kMany ? 2 : 4;
  static constexpr int kColBlk = kRows * 128;          // one 64-column block
  static constexpr int kTile = (D / 64) * kColBlk;
  static constexpr int kStats = (kHeldTiles + kStages) * kTile;  // [row tile or stage][128]
  static constexpr int kPart = kStats + 4 * kRows * 4;        // [kPartBufs][kParts][keys] sums
  static constexpr int kPartKeys = PASS == kMany ? 2 * kRows : kRows;
  static constexpr int kParts = 4;  // sums a key: of each warpgroup (MANY) or row tile (FEW)
  // Buffers of sums.  FEW: four, so that a warpgroup that writes to one at key tile j, and
  // waits for it there, has done so at j - 4 too, and so never misses a phase of its barrier.
  static constexpr int kPartBufs = PASS == kMany ? 2 : 4;
  static constexpr int kBars = kPart + kPartBufs * kParts * kPartKeys * 4;
  static constexpr int kSlot = kBars + kNumBars * 8;          // TMEM address, abort flag
  static constexpr int kAlloc = kSlot + 16 + 1024;
  static_assert(kAlloc <= 232448, "shared memory of an SM");
};

enum {
  kBarFull = 0,       // ring stage s landed
  kBarFree = 4,       // ring stage s read (commit; MANY: and by the consumers' warps)
  kBarHeld = 8,       // the held tiles landed
  kBarHeldFree = 9,   // MANY: .. have been read by the pair's last MMA (commit)
  kBarS = 10,         // S buffer 0 .. 3 (MANY: pair 0, 1) complete (commit)
  kBarSFree = 18,     // .. read (one arrival a warp that reads it)
  kBarPart = 26,      // columns: the sums of buffer 0 .. are written
  kBarPartFree = 30,  // .. have been read (2 warps)
  kBarDrain = 34,
};

// What a CTA does at a time.
struct Job {
  int b, g, bg, ctx, T;  // T = ctx + n_new
  int held0, n_held;     // held tiles: row tiles, or (MANY) key tiles
  int s0, n;             // streamed tiles
  int range;
};

// Job number `at`; n = 0: nothing to do.
template <int PASS>
__device__ __forceinline__ Job job_of(const WeightsParams &p, int at, bool report) {
  Job w;
  if (PASS == kMany) {
    w.bg = at / p.groups;
    w.held0 = (at - w.bg * p.groups) * 2;
    w.n_held = 2;
    w.range = 0;
  } else {
    const int ranges = PASS == kRowsPass ? p.n_ranges : p.key_ranges;
    w.range = at % ranges;
    at /= ranges;
    w.bg = at / p.groups;
    w.held0 = (at - w.bg * p.groups) * 4;
    w.n_held = min(4, p.n_rt - w.held0);
  }
  w.b = w.bg / p.n_kv_heads;
  w.g = w.bg - w.b * p.n_kv_heads;
  w.ctx = p.ctx_lens[w.b];
  const int most = p.max_blocks * kPageSize - p.n_new;
  if (w.ctx < 0 || w.ctx > most) {
    if (report) record_error(p.status, PA_ERR_BAD_CTX);
    w.ctx = w.ctx < 0 ? 0 : most;
  }
  w.T = w.ctx + p.n_new;
  if (PASS == kMany) {
    // row tiles whose last query sees the first held key
    const int q = max(0, w.held0 * kRows - w.ctx);
    w.s0 = q / p.nq * p.n_hsub;
    w.n = w.held0 * kRows < w.T ? p.n_rt - w.s0 : 0;
  } else {
    // key tiles that the held rows see, cut into ranges
    const int ranges = PASS == kRowsPass ? p.n_ranges : p.key_ranges;
    const int last_q = min(p.n_new, ((w.held0 + w.n_held - 1) / p.n_hsub + 1) * p.nq) - 1;
    const int tiles = (w.ctx + last_q) / kRows + 1;
    const int per = (tiles + ranges - 1) / ranges;
    w.s0 = w.range * per;
    w.n = max(0, min(per, tiles - w.s0));
  }
  return w;
}

// The page that lane l < 8 copies of key tile `tile`.
__device__ __forceinline__ int page_of(const WeightsParams &p, const Job &w, int tile, int lane) {
  const int pg = 8 * tile + lane;  // past the end: page 0, masked
  int id = lane < 8 && pg * kPageSize < w.T
               ? p.block_table[static_cast<size_t>(w.b) * p.max_blocks + pg] : 0;
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) {
    record_error(p.status, PA_ERR_BAD_BLOCK);
    id = 0;
  }
  return id;
}
// One K tile (8 pages of one kv head) into shared memory.  The whole warp; an elected lane
// issues the copies (eight lanes, two each: a pass 1 to 2% longer).
template <int D>
__device__ __forceinline__ void load_keys(const CUtensorMap *map, const WeightsParams &p,
                                          const Job &w, int id, uint32_t dst, uint32_t bar,
                                          int lane) {
  const int row = (id * p.n_kv_heads + w.g) * kPageSize;
  int at[kRows / kPageSize];
#pragma unroll
  for (int k = 0; k < kRows / kPageSize; ++k) at[k] = __shfl_sync(0xffffffffu, row, k);
  if (tc::elect_one()) {
#pragma unroll
    for (int k = 0; k < kRows / kPageSize; ++k)
#pragma unroll
      for (int x = 0; x < D / 64; ++x)
        tma_load_2d(dst + x * kRows * 128 + k * 2048, map, 64 * x, at[k], bar);
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

// Rows of tile rt that are queries: the first ones.
__device__ __forceinline__ int rows_of(const WeightsParams &p, int rt) {
  return min(p.nq, p.n_new - rt / p.n_hsub * p.nq) * p.hb;
}

// -(m + log2 l); a row without a key, or none at all, weighs nothing.
__device__ __forceinline__ float stat_of(float m, float l) {
  return l == 0.f ? -INFINITY : -(m + log2f(l));
}

// A row's ranges folded.
__device__ __forceinline__ float folded(const WeightsParams &p, int bg, int rt, int r) {
  if (query_of(p, rt, r) < 0) return -INFINITY;
  const float2 *st =
      p.states + (static_cast<size_t>(bg) * p.n_rt + rt) * p.n_ranges * kRows + r;
  float m = kNoKey, l = 0.f;
#pragma unroll 4
  for (int i = 0; i < p.n_ranges; ++i) {
    const float2 v = st[static_cast<size_t>(i) * kRows];
    const float mn = fmaxf(m, v.x);
    l = l * ex2(m - mn) + v.y * ex2(v.x - mn);
    m = mn;
  }
  return stat_of(m, l);
}

// Joins the consumer warpgroups.
__device__ __forceinline__ void consumers_sync() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kGroups * kRows) : "memory");
}

// ---- rows pass: 64 scores of this thread's row at a time
struct RowState {
  float m;
  float2 l;
};
__device__ __forceinline__ void take_scores(uint32_t (&s)[64], int key0, int lim, int lim_all,
                                            float qs, RowState &st) {
  if (key0 + 63 > lim_all) {
    const int last = lim - key0;
#pragma unroll
    for (int c = 0; c < 64; ++c)
      if (c > last) s[c] = __float_as_uint(-INFINITY);
  }
  float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
  for (int c = 0; c < 64; c += 4) {
    t0 = max3(t0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
    t1 = max3(t1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
  }
  const float cand = fmaxf(t0, t1) * qs;
  if (cand > st.m + kSlack) {
    const float corr = ex2(st.m - cand);
    st.m = cand;
    st.l = __fmul2_rn(st.l, make_float2(corr, corr));
  }
  const float2 qs2 = make_float2(qs, qs), nm2 = make_float2(-st.m, -st.m);
  float2 e2 = make_float2(0.f, 0.f), f2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < 64; c += 4) {
    const float2 a = __ffma2_rn(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
                                qs2, nm2);
    const float2 b = __ffma2_rn(make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])),
                                qs2, nm2);
    e2 = __fadd2_rn(e2, make_float2(ex2(a.x), ex2(a.y)));
    f2 = __fadd2_rn(f2, make_float2(ex2(b.x), ex2(b.y)));
  }
  st.l = __fadd2_rn(st.l, __fadd2_rn(e2, f2));
}

// Rows from `until` on only fill a tile up: zeros, which weigh nothing (lse = inf), but whose
// score at a key with a value that is not finite is NaN, and with it the key's sum.  The last of
// 32 tells; their scores are set to 0 then.  The whole warp.  (4 x 512 of 32/8 heads over 7680: 223
// -> 225 us, 2 x 33 of 64/8 over 32k: 87 -> 89; masks in the sums themselves: 226 and 88, but 8%
// more for groups that leave each tile padded; these by themselves, from q and K, where a sum is
// NaN: 220 and 91.)
template <int KEYS>
__device__ __forceinline__ void clear_padding(uint32_t (&s)[KEYS][32], int until) {
  if (until >= 32) return;
  bool any = false;
#pragma unroll
  for (int x = 0; x < KEYS; ++x) any |= __uint_as_float(s[x][31]) != 0.f;
  if (!__any_sync(0xffffffffu, any)) return;
#pragma unroll
  for (int x = 0; x < KEYS; ++x)
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (c >= until) s[x][c] = 0u;
}

// ---- columns pass: the weights of 32 rows for KEYS keys of this thread, added to their
// sums (of even and odd rows).  at: the rows' -lse in shared memory; rows from `from` on see
// the key.
template <int KEYS, bool MASKED>
__device__ __forceinline__ void add_weights(const uint32_t (&s)[KEYS][32], uint32_t at,
                                            const int (&from)[KEYS], float qs,
                                            float2 (&sum)[KEYS]) {
  const float2 qs2 = make_float2(qs, qs);
  float2 even[KEYS], odd[KEYS];
#pragma unroll
  for (int x = 0; x < KEYS; ++x) even[x] = odd[x] = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
    const uint4 v = lds128(at + c * 4);
    const float2 v0 = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    const float2 v1 = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
#pragma unroll
    for (int x = 0; x < KEYS; ++x) {
      const float2 a = __ffma2_rn(
          make_float2(__uint_as_float(s[x][c]), __uint_as_float(s[x][c + 1])), qs2, v0);
      const float2 b = __ffma2_rn(
          make_float2(__uint_as_float(s[x][c + 2]), __uint_as_float(s[x][c + 3])), qs2, v1);
      float2 ea = make_float2(ex2(a.x), ex2(a.y)), eb = make_float2(ex2(b.x), ex2(b.y));
      if (MASKED) {
        if (c < from[x]) ea.x = 0.f;
        if (c + 1 < from[x]) ea.y = 0.f;
        if (c + 2 < from[x]) eb.x = 0.f;
        if (c + 3 < from[x]) eb.y = 0.f;
      }
      even[x] = __fadd2_rn(even[x], ea);
      odd[x] = __fadd2_rn(odd[x], eb);
    }
  }
#pragma unroll
  for (int x = 0; x < KEYS; ++x) sum[x] = __fadd2_rn(sum[x], __fadd2_rn(even[x], odd[x]));
}

template <int D, bool BF16, int PASS>
__global__ void __launch_bounds__(kThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap, const WeightsParams p) {
  using L = WeightsSmem<D, PASS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) { return sb + L::kBars + 8 * i; };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_release();
  griddep_wait();

  Job w = job_of<PASS>(p, blockIdx.x, tid == 0);
  if (PASS != kMany && w.n == 0) {  // nothing of the keys is left for this range
    if (PASS == kRowsPass)
      for (int e = tid; e < w.n_held * kRows; e += kThreads)
        p.states[((static_cast<size_t>(w.bg) * p.n_rt + w.held0 + e / kRows) * p.n_ranges +
                  w.range) * kRows + e % kRows] = make_float2(kNoKey, 0.f);
    return;
  }

  const int S = min(4, L::kHeldTiles + L::kStages - w.n_held);  // stages of the ring
  const uint32_t ring0 = sb + w.n_held * L::kTile;

  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kSlot + 4);
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      int n = 1;
      if (i >= kBarFree && i < kBarHeld) n = PASS == kMany ? 1 + 4 * kGroups : 1;
      if (i >= kBarSFree && i < kBarPart) n = PASS == kMany ? 4 * kGroups : 4;
      if (i >= kBarPartFree && i < kBarDrain) n = 2;
      if (i >= kBarPart && i < kBarPartFree) n = PASS == kMany ? 4 * kGroups : 4 * w.n_held;
      mbar_init(bar(i), n);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    __syncwarp();
    tc::alloc(sb + L::kSlot, 512);
    tc::relinquish();
  }
  // Rows of a query tile behind its box are never written by the copies: they hold zeros.
  if (p.hb * p.nq < kRows) {
    const int r0 = p.hb * p.nq, rows = kRows - r0;
    const int first = PASS == kMany ? L::kHeldTiles * L::kTile : 0;
    const int n = PASS == kMany ? L::kStages : w.n_held;
    for (int e = tid; e < n * (D / 64) * rows * 8; e += kThreads) {
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
  const uint32_t stats_bytes = kRows * sizeof(float);
  // Row tiles that the rows pass's warpgroups take in turn: one or two, or a warpgroup each.
  const int turns = w.n_held <= 2 ? w.n_held : kGroups;
  // the jobs of a CTA: one, or (MANY) every gridDim.x-th item
  auto next_job = [&](int &at) {
    for (at += gridDim.x; PASS == kMany && at < p.items; at += gridDim.x) {
      w = job_of<PASS>(p, at, false);
      if (w.n > 0) return true;
    }
    return false;
  };
  int at = blockIdx.x;
  bool more = true;
  if (PASS == kMany && w.n == 0) more = next_job(at);

  if (warp == 0) {
    // ---- loads
    bool ok = true;
    int c = 0, job = 0;  // tiles streamed, jobs done
    int s = 0;           // the next one's stage, and how often the ring has gone round
    uint32_t round = 0;
    for (; more && ok; more = next_job(at), ++job) {
      if (PASS == kMany && job > 0 &&
          !(ok = warp_wait(bar(kBarHeldFree), (job - 1) & 1, abort_flag)))
        break;
      if (lane == 0)
        mbar_arrive_expect_tx(bar(kBarHeld), w.n_held * (PASS == kMany ? L::kTile : q_bytes));
      __syncwarp();
      for (int x = 0; x < w.n_held; ++x) {
        if (PASS == kMany)
          load_keys<D>(&kmap, p, w, page_of(p, w, w.held0 + x, lane), sb + x * L::kTile,
                       bar(kBarHeld), lane);
        else if (lane == 0)
          load_queries<D>(&qmap, p, w, w.held0 + x, sb + x * L::kTile, bar(kBarHeld));
      }
      int id = PASS != kMany ? page_of(p, w, w.s0, lane) : 0;  // of the next key tile
      for (int j = 0; j < w.n; ++j, ++c) {
        const int here = id;
        if (PASS != kMany && j + 1 < w.n) id = page_of(p, w, w.s0 + j + 1, lane);
        if (c >= S && !(ok = warp_wait(bar(kBarFree + s), (round - 1) & 1, abort_flag))) break;
        const uint32_t full = bar(kBarFull + s), dst = ring0 + s * L::kTile;
        if (lane == 0)
          mbar_arrive_expect_tx(full, PASS == kMany ? q_bytes + stats_bytes : L::kTile);
        __syncwarp();
        if (PASS != kMany) {
          load_keys<D>(&kmap, p, w, here, dst, full, lane);
        } else if (lane == 0) {
          load_queries<D>(&qmap, p, w, w.s0 + j, dst, full);
          bulk_load(sb + L::kStats + s * stats_bytes,
                    p.stats + (static_cast<size_t>(w.bg) * p.n_rt + w.s0 + j) * kRows,
                    stats_bytes, full);
        }
        if (++s == S) s = 0, ++round;
      }
    }
    if (!ok) {
      if (lane == 0) raise_abort(p.status, abort_flag);
      mbar_wait(bar(kBarHeld), job & 1);  // copies in flight still land
      for (int t = max(0, c - S); t < c; ++t) mbar_wait(bar(kBarFull + t % S), (t / S) & 1);
    }
  } else if (warp == 1) {
    // ---- S of every held tile against each streamed one; the keys' tile is the first
    // operand in the columns pass, the rows' in the rows pass
    const uint32_t held = tc::desc_low(sb), ring = tc::desc_low(ring0);
    constexpr uint32_t kTileLow = L::kTile >> 4;
    const bool issuer = tc::elect_one();
    auto mma = [&](uint32_t dst, uint32_t a, uint32_t b, uint32_t id) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = ((k >> 2) * L::kColBlk + (k & 3) * 32) >> 4;
        tc::mma_f16_low(dst, a + off, b + off, id, k > 0);
      }
    };
    const uint32_t full_id = tc::idesc_f16(BF16, kRows, kRows, false, false) | p.negate;
    bool ok = true;
    int c = 0, job = 0, n = 0, s = 0;  // tiles, jobs, chunks, the tile's stage
    uint32_t round = 0;
    uint32_t ids[4];  // FEW: as many rows as are read
    if (PASS == kFew)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        ids[x] = tc::idesc_f16(BF16, kRows, (rows_of(p, x) + 31) & ~31, false, false) | p.negate;
    for (; more && ok; more = next_job(at), ++job) {
      ok = warp_wait(bar(kBarHeld), job & 1, abort_flag);
      for (int j = 0; j < w.n && ok; ++j, ++c) {
        if (!(ok = warp_wait(bar(kBarFull + s), round & 1, abort_flag))) break;
        const uint32_t tile = ring + s * kTileLow;
        if constexpr (PASS != kMany) {  // a chunk a row tile
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (x >= w.n_held) break;
            const int buf = PASS == kRowsPass && turns == kGroups ? x : n & 3;
            const int use = PASS == kRowsPass && turns == kGroups ? c : n >> 2;
            if (use > 0 && !(ok = warp_wait(bar(kBarSFree + buf), (use - 1) & 1, abort_flag)))
              break;
            tc::fence_after_sync();
            const uint32_t a = held + x * kTileLow;
            if (issuer) {
              mma(tmem + kRows * buf, PASS == kRowsPass ? a : tile, PASS == kRowsPass ? tile : a,
                  PASS == kRowsPass ? full_id : ids[x]);
              tc::commit(bar(kBarS + buf));
            }
            ++n;
          }
        } else {  // both key tiles' scores, in one of two pairs of buffers
          if (c >= 2 && !(ok = warp_wait(bar(kBarSFree + (c & 1)), ((c >> 1) - 1) & 1, abort_flag)))
            break;
          tc::fence_after_sync();
          if (issuer) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
              mma(tmem + kRows * (2 * (c & 1) + x), held + x * kTileLow, tile, full_id);
            tc::commit(bar(kBarS + (c & 1)));
            if (j == w.n - 1) tc::commit(bar(kBarHeldFree));
          }
        }
        if (ok && issuer) tc::commit(bar(kBarFree + s));
        if (++s == S) s = 0, ++round;
      }
    }
    if (!ok) {
      if (issuer) {
        raise_abort(p.status, abort_flag);
        tc::commit(bar(kBarDrain));
      }
      __syncwarp();
      mbar_wait(bar(kBarDrain), 0);
    }
  } else if (warp < 4) {
    if (PASS != kRowsPass) {
      // ---- the consumers' sums into the pool
      bool ok = true;
      constexpr int U = L::kPartKeys / 64;  // keys a thread
      struct Place {
        float *dst;
        float old;
      };
      // where key tid - 64 + 64 u of a tile lies, given its page, and what is there
      auto page_at = [&](int key) {
        return key < w.T ? p.block_table[static_cast<size_t>(w.b) * p.max_blocks + key / kPageSize]
                         : -1;
      };
      auto place_of = [&](int key, int page) {
        Place v = {nullptr, 0.f};
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) {  // else reported
          v.dst = p.weights + (static_cast<size_t>(page) * p.n_kv_heads + w.g) * kPageSize +
                  key % kPageSize;
          if (key < w.T - p.fresh) v.old = *v.dst;
        }
        return v;
      };
      int n = 0;  // sums taken
      for (; more && ok; more = next_job(at)) {
        const int tiles = PASS == kFew ? w.n : 1;
        const int key0 = (PASS == kFew ? w.s0 : w.held0) * kRows + tid - 64;
        // a tile's old weights are fetched a tile ahead, its pages two
        int page[U];
        Place next[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          next[u] = place_of(key0 + 64 * u, page_at(key0 + 64 * u));
          if (PASS == kFew) page[u] = page_at(key0 + kRows + 64 * u);
        }
        for (int j = 0; j < tiles; ++j, ++n) {
          Place here[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            here[u] = next[u];
            if (PASS == kFew) {
              const int key = key0 + (j + 1) * kRows + 64 * u;
              next[u] = place_of(key, page[u]);
              page[u] = page_at(key + kRows);
            }
          }
          const int buf = n % L::kPartBufs;
          if (!(ok = warp_wait(bar(kBarPart + buf), (n / L::kPartBufs) & 1, abort_flag))) break;
          const float *part = reinterpret_cast<const float *>(smem + L::kPart) +
                              buf * L::kParts * L::kPartKeys + tid - 64;
          float sum[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            sum[u] = 0.f;
#pragma unroll
            for (int y = 0; y < L::kParts; ++y)
              if (PASS == kMany || y < w.n_held) sum[u] += part[y * L::kPartKeys + 64 * u];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarPartFree + buf));
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (here[u].dst) *here[u].dst = here[u].old + sum[u];
        }
      }
      if (!ok && lane == 0) raise_abort(p.status, abort_flag);
    }
  } else {
    // ---- consumers
    const int y = (warp - 4) >> 2, r = ((warp & 3) << 5) + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float qs = p.qscale;
    bool ok = true;
    // the chunk in buffer `buf` has been read
    auto release = [&](int buf) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarSFree + buf));
    };
    if constexpr (PASS == kRowsPass) {
      // One or two row tiles: several warpgroups take the key tiles of one in turn.
      const int x = y % turns, step = kGroups / turns;
      const int rt = w.held0 + x, q0 = rt / p.n_hsub * p.nq;
      const int lim = w.ctx + min(q0 + r / p.hb, p.n_new - 1);  // the last key row r sees
      const int lim_all = w.ctx + q0;                           // .. that every row does
      const bool idle = 32 * (warp & 3) >= rows_of(p, rt);      // none of the warp's rows is one
      RowState st = {kNoKey, make_float2(0.f, 0.f)};
      if (x < w.n_held) {
        const uint32_t at = tmem + kRows * y + lanes;
        uint32_t uses = 0;  // of the buffer
        // 64 keys at a time, in one copy of the code: with four (unrolled over tiles) the
        // other warps' instructions left the cache, and each of their waits took 450 cycles
#pragma unroll 1
        for (int i = y / turns * 2; i < 2 * w.n;) {
          if ((i & 1) == 0) {
            if (!(ok = warp_wait(bar(kBarS + y), uses & 1, abort_flag))) break;
            ++uses;
            tc::fence_after_sync();
          }
          if (!idle) {
            uint32_t s[64];
            __syncwarp();  // lanes part where their maxima move; the loads want the whole warp
            tc::ld32(at + 64 * (i & 1), *reinterpret_cast<uint32_t(*)[32]>(s));
            tc::ld32(at + 64 * (i & 1) + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
            tc::wait_ld();
            if (i & 1) release(y);
            take_scores(s, w.s0 * kRows + 64 * i, lim, lim_all, qs, st);
          } else if (i & 1) {
            release(y);
          }
          i += (i & 1) ? 2 * step - 1 : 1;
        }
      }
      float m = st.m, l = st.l.x + st.l.y;
      if (step > 1) {
        // Their states folded, through the row tiles' place: every chunk is complete, so those
        // have been read.
        consumers_sync();
        float2 *all = reinterpret_cast<float2 *>(smem);
        all[y * kRows + r] = make_float2(m, l);
        consumers_sync();
        for (int k = y + turns; k < kGroups; k += turns) {
          const float2 v = all[k * kRows + r];
          const float mn = fmaxf(m, v.x);
          l = l * ex2(m - mn) + v.y * ex2(v.x - mn);
          m = mn;
        }
      }
      if (ok && y < w.n_held) {
        const size_t tile = static_cast<size_t>(w.bg) * p.n_rt + rt;
        p.states[(tile * p.n_ranges + w.range) * kRows + r] = make_float2(m, l);
        if (p.n_ranges == 1)
          p.stats[tile * kRows + r] = query_of(p, rt, r) < 0 ? -INFINITY : stat_of(m, l);
      }
    } else if constexpr (PASS == kFew) {
      float *part = reinterpret_cast<float *>(smem + L::kPart) + r;
      {  // the rows' statistics, a row a thread
        float *stats = reinterpret_cast<float *>(smem + L::kStats);
        const int e = tid - (kThreads - kGroups * kRows);
        if (e < w.n_held * kRows) stats[e] = folded(p, w.bg, e / kRows, e % kRows);
        consumers_sync();
      }
      const int chunks = w.n * w.n_held;
      int j = y / w.n_held, x = y - j * w.n_held;      // of chunk n
      const int last_rows = rows_of(p, w.n_held - 1);  // of the last query tile's
      for (int n = y; n < chunks && ok; n += kGroups) {
        if (!(ok = warp_wait(bar(kBarS + y), (n >> 2) & 1, abort_flag))) break;
        tc::fence_after_sync();
        const int key0 = (w.s0 + j) * kRows;
        const int rows = x >= w.n_held - p.n_hsub ? last_rows : p.hb * p.nq;
        const int q0 = (p.n_hsub == 1 ? x : x / p.n_hsub) * p.nq;  // the tile's first query
        const bool all = key0 + kRows - 1 <= w.ctx + q0;  // every row sees every key
        float2 sum[1] = {make_float2(0.f, 0.f)};
#pragma unroll 1
        for (int c0 = 0; c0 < rows; c0 += 64) {
          uint32_t s[2][1][32];
          const uint32_t at = tmem + kRows * y + lanes + c0;
          tc::ld32(at, s[0][0]);
          if (rows > c0 + 32) tc::ld32(at + 32, s[1][0]);
          tc::wait_ld();
          if (c0 + 64 >= rows) release(y);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (c0 + 32 * h >= rows) break;
            const uint32_t lse = sb + L::kStats + x * stats_bytes + (c0 + 32 * h) * 4;
            const int from[1] = {(key0 + r - w.ctx - q0) * p.hb - c0 - 32 * h};
            clear_padding(s[h], rows - c0 - 32 * h);
            if (all)
              add_weights<1, false>(s[h], lse, from, qs, sum);
            else
              add_weights<1, true>(s[h], lse, from, qs, sum);
          }
        }
        if (j >= 4 &&
            !(ok = warp_wait(bar(kBarPartFree + (j & 3)), ((j >> 2) - 1) & 1, abort_flag)))
          break;
        part[((j & 3) * L::kParts + x) * kRows] = sum[0].x + sum[0].y;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPart + (j & 3)));
        for (x += kGroups; x >= w.n_held; x -= w.n_held) ++j;
      }
    } else {
      float *part = reinterpret_cast<float *>(smem + L::kPart) + y * 2 * kRows + r;
      int c = 0, job = 0, st = 0;  // tiles, jobs, the tile's stage
      uint32_t round = 0;
      for (; more && ok; more = next_job(at), ++job) {
        const int key0 = w.held0 * kRows;
        float2 sum[2];
        sum[0] = sum[1] = make_float2(0.f, 0.f);
        for (int j = 0; j < w.n; ++j, ++c) {
          const int buf = c & 1;
          if (!(ok = warp_wait2(bar(kBarS + buf), (c >> 1) & 1, bar(kBarFull + st), round & 1,
                                abort_flag)))
            break;
          tc::fence_after_sync();
          uint32_t s[2][32];
#pragma unroll
          for (int x = 0; x < 2; ++x)
            tc::ld32(tmem + kRows * (2 * buf + x) + lanes + 32 * y, s[x]);
          tc::wait_ld();
          release(buf);
          const int q0 = (p.n_hsub == 1 ? w.s0 + j : (w.s0 + j) / p.n_hsub) * p.nq;
          const uint32_t lse = sb + L::kStats + st * stats_bytes + 32 * y * 4;
          int from[2];
#pragma unroll
          for (int x = 0; x < 2; ++x)
            from[x] = (key0 + x * kRows + r - w.ctx - q0) * p.hb - 32 * y;
          clear_padding(s, min(p.nq, p.n_new - q0) * p.hb - 32 * y);
          if (key0 + 2 * kRows - 1 <= w.ctx + q0)
            add_weights<2, false>(s, lse, from, qs, sum);
          else
            add_weights<2, true>(s, lse, from, qs, sum);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarFree + st));
          if (++st == S) st = 0, ++round;
        }
        if (!ok) break;
        if (job >= 2 &&
            !(ok = warp_wait(bar(kBarPartFree + (job & 1)), ((job >> 1) - 1) & 1, abort_flag)))
          break;
#pragma unroll
        for (int x = 0; x < 2; ++x)
          part[(job & 1) * L::kParts * 2 * kRows + x * kRows] = sum[x].x + sum[x].y;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPart + (job & 1)));
      }
    }
    if (!ok && lane == 0) raise_abort(p.status, abort_flag);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::dealloc(tmem, 512);
  }
}

// The rows' ranges folded for the columns pass of many row tiles.
__global__ void __launch_bounds__(kRows) stats_kernel(const WeightsParams p) {
  griddep_release();
  griddep_wait();
  const int bg = blockIdx.x / p.n_rt, rt = blockIdx.x - bg * p.n_rt, r = threadIdx.x;
  p.stats[static_cast<size_t>(blockIdx.x) * kRows + r] = folded(p, bg, rt, r);
}

// Ranges that `ctas` units of `tiles` key tiles each are cut into: the number whose waves
// of CTAs take least, a CTA's start counting as three tiles.
int ranges_of(int64_t ctas, int tiles, int sms) {
  if (ctas >= 8 * sms) return 1;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int r = 1; r <= 64 && r <= tiles; ++r) {
    const int waves = (static_cast<int>(ctas) * r + sms - 1) / sms;
    const int64_t cost = static_cast<int64_t>(waves) * ((tiles + r - 1) / r + 3);
    if (cost < least - least / 32) {  // more ranges only for more than 3%
      least = cost;
      best = r;
    }
  }
  return best;
}

struct Plan {
  int hb, nq, n_hsub, n_rt, ranges, key_ranges;
};
Plan plan_of(int batch, int n_new, int n_q_heads, int n_kv_heads, int max_blocks, int sms) {
  const int group = n_q_heads / n_kv_heads;
  Plan y;
  y.hb = group;
  if (y.hb > kRows)  // the largest divisor that fits a tile
    for (y.hb = kRows; group % y.hb; --y.hb) {
    }
  y.n_hsub = group / y.hb;
  y.nq = kRows / y.hb;
  y.n_rt = y.n_hsub * ((n_new + y.nq - 1) / y.nq);
  const int64_t lists = static_cast<int64_t>(batch) * n_kv_heads;
  const int tiles = (max_blocks * kPageSize + kRows - 1) / kRows;
  y.ranges = ranges_of(lists * ((y.n_rt + 3) / 4), tiles, sms);
  y.key_ranges = ranges_of(lists, tiles, sms);
  return y;
}

size_t states_bytes(int64_t lists, const Plan &y) {
  return static_cast<size_t>(lists) * y.n_rt * y.ranges * kRows * sizeof(float2);
}

template <int D, bool BF16, int PASS>
int launch_pass(const CUtensorMap &qmap, const CUtensorMap &kmap, const WeightsParams &p,
                int64_t ctas, cudaStream_t stream) {
  using L = WeightsSmem<D, PASS>;
  auto kern = weights_kernel<D, BF16, PASS>;
  static ContextCache<bool> smem_set;
  if (set_smem_limit(kern, L::kAlloc, smem_set) != PA_OK) return PA_ERR_CUDA;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), L::kAlloc, stream,
                    qmap, kmap, p) == cudaSuccess
             ? PA_OK : PA_ERR_CUDA;
}

template <int D, bool BF16>
int launch_t(const WeightsLaunch &a, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return PA_ERR_CUDA;
  const Plan y =
      plan_of(a.batch, a.n_new, a.n_q_heads, a.n_kv_heads, a.max_blocks, sms);
  CUtensorMap qmap, kmap;
  const uint64_t rows = static_cast<uint64_t>(a.num_pages) * a.n_kv_heads * kPageSize;
  if (make_rows_map(&kmap, a.k_cache, rows, D, kPageSize) != PA_OK) return PA_ERR_CUDA;
  if (make_query_map(&qmap, a.q, D, a.n_q_heads, a.n_new, a.batch, a.q_token_stride,
                     a.q_batch_stride, y.hb, y.nq) != PA_OK)
    return PA_ERR_CUDA;
  const int64_t lists = static_cast<int64_t>(a.batch) * a.n_kv_heads;
  WeightsParams p;
  p.block_table = a.block_table;
  p.ctx_lens = a.ctx_lens;
  p.weights = a.weights;
  p.states = static_cast<float2 *>(a.workspace);
  p.stats = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + states_bytes(lists, y));
  p.status = a.status;
  // The rows pass takes the maximum of the raw scores, so it needs a positive factor: a
  // negative scale turns the first operand's sign instead, and a zero scale becomes a factor
  // small enough that every weight is the same.
  p.qscale = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
  p.negate = a.scale < 0.f ? tc::kNegateA : 0u;
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
  p.key_ranges = y.key_ranges;
  p.groups = (y.n_rt + 3) / 4;
  p.items = 0;
  int rc = launch_pass<D, BF16, kRowsPass>(qmap, kmap, p, lists * p.groups * p.n_ranges, stream);
  if (rc) return rc;
  if (y.n_rt <= 4) {
    p.groups = 1;
    return launch_pass<D, BF16, kFew>(qmap, kmap, p, lists * p.key_ranges, stream);
  }
  if (y.ranges > 1 &&
      launch_pdl(stats_kernel, dim3(static_cast<unsigned>(lists * y.n_rt)), dim3(kRows), 0, stream,
                 p) != cudaSuccess)
    return PA_ERR_CUDA;
  const int key_tiles = (a.max_blocks * kPageSize + kRows - 1) / kRows;
  p.groups = (key_tiles + 1) / 2;
  p.items = static_cast<int>(lists * p.groups);
  return launch_pass<D, BF16, kMany>(qmap, kmap, p, p.items < sms ? p.items : sms, stream);
}

}  // namespace

size_t weights_workspace_bytes(int batch, int n_new, int n_q_heads, int n_kv_heads,
                               int max_blocks, int sms) {
  const Plan y = plan_of(batch, n_new, n_q_heads, n_kv_heads, max_blocks, sms);
  const int64_t lists = static_cast<int64_t>(batch) * n_kv_heads;
  return states_bytes(lists, y) + static_cast<size_t>(lists) * y.n_rt * kRows * sizeof(float);
}

int launch_weights(const WeightsLaunch &a, cudaStream_t stream) {
  if (a.head_dim == 128)
    return a.bf16 ? launch_t<128, true>(a, stream) : launch_t<128, false>(a, stream);
  return a.bf16 ? launch_t<64, true>(a, stream) : launch_t<64, false>(a, stream);
}

}  // namespace pa
