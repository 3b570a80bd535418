// pa_kv4_rows.cu -- attention over the 4-bit paged cache for few query rows a
// kv head: decode (one query a sequence) and short chunks (speculative verify).
//
// A row is a (query, head) pair of one kv head; o = softmax(q K^T scale) V with
// K = zero_k + scale_k (c - 8) and V alike, c the 4-bit codes.  The codes go
// into the tensor cores as they are (exact in 16 bits) and the scales and
// zeros are applied outside,
//   s_t = scale_k[t] (q . (c_t - 8)) + zero_k[t] sum q
//   O   = sum_t (p_t scale_v[t]) (c_t - 7.5),   z = sum_t p_t (zero_v[t] - scale_v[t] / 2)
// so a page costs no dequantisation beyond turning nibbles into 16-bit floats.
//
// Operand form.  mma.sync m16n8k16 with the tokens (then the head dimensions)
// as the 16 rows and 8 query rows as the columns.  That uses every tensor-core
// row for up to 8 query rows, keeps the output state in head_dim / 4 registers
// a thread, and needs no transpose of K or V: a thread loads whole 32-bit words
// of codes, and because the contraction index may be permuted freely (q, or the
// order of tokens, is permuted alike) two nibbles four places apart in one
// word, or the same nibble of two tokens' words, form an operand register.
// The tensor cores align the addends of a sum to the largest and round toward zero, so
// operands are centred first.  K: (x & 0x000f000f) | 0x64006400 is 1024 + c, minus 1032;
// (x & 0x00f000f0) | 0x64006400 is 1024 + 16 c, times 1/16 minus 72; both exact.
// V: the fp16 subnormals x & 0x000f000f = c 2^-24 and x & 0x00f000f0 = c 2^-20, by one
// FMA each (c - 7.5) 2^-9, exact too; codes of a row lie evenly about 7.5, so that the
// sums do not grow with the number of keys where the result's terms cancel (with c - 8
// rows over 131072 keys were off by 1.2e-5, so by 7e-7; plain fp32: 1e-6).
// Codes as they are (one AND) would save the subtractions, but sums that carry 8 sum q
// or 8 sum p lose the last bits of the result: for K measured 1.3e-6 of the result's
// norm against 2e-7 (8% faster), for V 1e-4.  q is scaled by a power of two a row (its
// largest magnitude near 2^15; exact in fp16 down to 2^-39 of that).
// The weights p scale_v enter as two fp16 terms (head and remainder, 22 bits), relative
// to a power of two above the largest |scale_v| so far and multiplied by 2^7: they stay
// below 2^15.  The remainder, at most 2^3, is multiplied by 2^12 and summed in an
// accumulator of its own, so it still holds weights below the head's range, in steps of
// 2^-43 of the largest (at the head's scale it ended where the head does: 32k keys beside
// one that takes 0.99 of the weight came out 4e-4 off, now 9e-7); and l keeps what its
// last rounding lost.  With at most 4 rows
// (WIDE false) columns 4-7 repeat columns 0-3 and carry the second terms: one MMA does
// both.  The weights, in the accumulator's layout (token, row), become the second
// product's operand (row, token) by movmatrix.  The sums of each two pages are taken in
// an accumulator of their own and added to the state with a rounding add, because the
// tensor cores' roundings toward zero add up along a long context (measured on 32k
// tokens, 8 rows, with c - 8: error 9e-6 of the result in one accumulator, 8e-7 so; with
// c - 7.5 2e-7).
//
// Work split.  The pages of all (sequence, kv head, row tile) items, laid end to
// end, are cut into equal runs: a ragged batch takes the time of its pages, not of
// its longest sequence.  An item counts 12 pages more than it has, for what starting
// and merging it costs (64 sequences of 128 to 8192 tokens: 97 -> 86 us when it came in;
// 3, 6, 10, 12 and 16 pages now take 80, 81, 82, 82 and 76 there, and 60, 51, 52, 52 and
// 53 for 4 x 32768 of 64 / 8 heads).  A run belongs to a team of 4 warps, and an SM holds 4
// teams in one CTA, so that they can keep step (below).  A team's warps take its
// run's pages two by two in turn, each with its own ring of stages filled by bulk
// copies, and merge their (m, l, O) states when an item ends.  An item cut between
// teams leaves one state a team, folded in order of position by a second kernel
// (results do not depend on timing).  Runs go round the SMs, so that a call with few
// of them has one an SM (1 x 512 tokens of 16 heads: 21.0 -> 14.8 us of device time).
//
// Bound: issue.  Turning a page's codes is some 150 of about 410 warp instructions a page
// (planning and merging included); 61% of the issue slots and 52% of the ALU's are taken,
// DRAM 43%.  Decode at head_dim 128, a call: 8 x 4096 tokens of 32 / 32 heads 42.2 us
// (143 MB, 3.4 TB/s), 64 sequences of 128 to 8192 of 32 / 8 heads 81 us (287 MB, 3.5
// TB/s), 4 x 32768 of 64 / 8 heads 51 us (143 MB, 2.8 TB/s); the 16-bit cache's bytes
// alone would take 79, 159 and 79 us at the copy's bandwidth.
#include "pa_device.cuh"
#include "pa_kv4.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleSlack = 8.0f;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kNoKey = -3.402823466e38f;  // running max of a row before its first key
constexpr float kRemLift = 4096.f;  // of the weights' remainders
constexpr int kWarps = 4, kStages = 2, kTile = 8;  // query rows a tile
constexpr int kPair = 2;         // pages a stage holds
constexpr int kTeams = 4;        // teams of kWarps warps a CTA, one CTA an SM
constexpr int kMinPages = kWarps * kPair;  // least pages a team takes
constexpr int kPartPages = 12;   // what a part's start and merge cost, in pages
constexpr uint32_t kLead = 2;         // chunks a warp may be ahead of the slowest team

struct RowsParams {
  const uint16_t *q;
  const uint8_t *cache;
  const int32_t *block_table, *ctx_lens;
  void *out;
  float *ws;     // [team][2][kTile][D + 4] partial states
  int4 *cut;     // [team][2] the item that starts in the team's run and leaves it
  int *status;
  float qscale;  // scale * log2 e
  int n_new, queries, n_q_heads, n_kv_heads, group, batch, max_blocks, num_pages;
  int n_rows, n_sub, tile_rows;  // rows a kv head, row tiles, rows a tile
  uint32_t page_bytes;           // all kv heads' blocks of a page
};

template <int D>
struct RowsSmem {
  static constexpr int kBlock = kv4::block_bytes(D);
  static constexpr int kStage = kPair * kBlock;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kRowStride = D + 4;  // floats a merged row
  static constexpr int kMergeO = kRing;
  static constexpr int kMergeM = kMergeO + kWarps * kTile * kRowStride * 4;
  static constexpr int kMergeL = kMergeM + kWarps * kTile * 4;
  static constexpr int kQ = kMergeL + kWarps * kTile * 4;      // [2][kTile][D], 16 bits
  static constexpr int kBars = kQ + 2 * kTile * D * 2;
  static constexpr int kParts = kBars + kWarps * kStages * 8;  // Part[4]
  static constexpr int kWalk = kParts + 4 * 64;                // Walk
  static constexpr int kFlags = kWalk + 64;
  static constexpr int kTeam = (kFlags + 64 + 127) & ~127;     // all of the above, a team
  static constexpr int kDone = kTeams * kTeam;  // chunks done, a team's first warp's
  static constexpr int kBytes = kDone + kTeams * 4;
  static_assert(kBlock % 128 == 0 && kQ % 16 == 0 && kBars % 8 == 0 && kParts % 16 == 0,
                "alignment");
  static_assert(kTeam % 128 == 0 && kBytes <= 232448, "shared memory of an SM");
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t sub_1032(uint32_t x) {
  const __half2 r = __hsub2(*reinterpret_cast<__half2 *>(&x), __float2half2_rn(1032.f));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t sixteenth_sub_72(uint32_t x) {
  const __half2 r = __hfma2(*reinterpret_cast<__half2 *>(&x), __float2half2_rn(0.0625f),
                            __float2half2_rn(-72.f));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// (c - 7.5) 2^-9 of the fp16 subnormals c 2^-K, exact.
template <int K>
__device__ __forceinline__ uint32_t centred(uint32_t x) {
  const __half2 r = __hfma2(*reinterpret_cast<__half2 *>(&x), __float2half2_rn(1 << (K - 9)),
                            __float2half2_rn(-7.5f / 512.f));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// d = a b, the accumulator starting at zero.
__device__ __forceinline__ void mma_from_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Physical token of score row r < 8 (row r + 8: 8 more).  The order makes the
// rows that neighbouring lanes read from a stage alternate between its even and
// odd rows, which is what shared memory's 32 banks want of 64-byte rows.
__device__ __forceinline__ int token_of(int r) {
  const int c = r >> 1, a = c >> 1, b = c & 1;
  return (r & 1) ? 4 * a + 3 - b : 4 * a + b;
}

// The part of one item that a team's run holds.
struct Part {
  int b, g;           // sequence, kv head
  int r0, n_r;        // rows of the kv head
  int pg0, n_pg;      // pages
  int tokens;         // keys of the sequence, the chunk's included
  int first, last;    // teams that hold the item
  int slot;           // of the first one's state: 0 when the item starts its run
  int more;           // the run goes on behind this part
};
static_assert(sizeof(Part) <= 64, "room in shared memory");

// The team's run [w, w1) of the flattened list of units, walked part by part by one
// thread, which keeps the others' registers free of it.  A boundary between runs in or
// right behind an item's kPartPages units counts as lying before the item, so that
// every part has a page.
struct Walk {
  int64_t w, w1, run, base;  // base: units of one (kv head, row tile) before sequence b
  int b, n_b, tokens;        // the sequence, its units and its tokens

  // Tokens of sequence b, the chunk's included (a clamped length is reported by
  // the first team's scan).
  static __device__ int tokens_of(const RowsParams &p, int b, bool report) {
    const int most = p.max_blocks * kPageSize - p.n_new;
    int t = p.ctx_lens[b];
    if (t < 0 || t > most) {
      if (report) record_error(p.status, PA_ERR_BAD_CTX);
      t = t < 0 ? 0 : most;
    }
    return t + p.n_new;
  }
  // An empty sequence counts one page, so that someone writes its zeros.
  static __device__ int pages_of(int tokens) {
    return max(1, (tokens + kPageSize - 1) / kPageSize);
  }
  // Units of an item in the list: its pages behind kPartPages of its own.
  static __device__ int units_of(int tokens) { return pages_of(tokens) + kPartPages; }
  // The whole warp: lane l sums the pages of sequences [l per, (l + 1) per), and a
  // scan finds the sequence in which the team's run starts.  False: no run.
  // Warp-uniform results; lane 0 keeps them in *out.
  static __device__ bool start(const RowsParams &p, int team, int n_teams, int lane, Walk *out) {
    Walk x;
    const int heads = p.n_kv_heads * p.n_sub;
    const int per = (p.batch + 31) / 32;
    const int b0 = min(p.batch, lane * per), b1 = min(p.batch, b0 + per);
    int64_t sum = 0;
    int tokens = 0;  // of sequence b0
#pragma unroll 4
    for (int i = b0; i < b1; ++i) {
      const int t = tokens_of(p, i, team == 0);
      sum += units_of(t);
      if (i == b0) tokens = t;
    }
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    const int64_t total = __shfl_sync(kFull, incl, 31) * heads;
    x.run = max(kv4::quotient(total + n_teams - 1, n_teams), static_cast<int64_t>(kMinPages));
    x.w = team * x.run;
    x.w1 = min(total, x.w + x.run);
    if (x.w >= x.w1) return false;
    const int src = __ffs(__ballot_sync(kFull, incl * heads > x.w)) - 1;
    x.b = __shfl_sync(kFull, b0, src);
    x.base = __shfl_sync(kFull, incl - sum, src);
    x.tokens = __shfl_sync(kFull, tokens, src);
    x.n_b = units_of(x.tokens);
    if (lane == 0) *out = x;
    return true;
  }
  // (A run that ends before its first item's pages begin: n_pg < 1.)
  __device__ void next(const RowsParams &p, volatile Part &s) {
    const int heads = p.n_kv_heads * p.n_sub;
    while ((base + n_b) * heads <= w) {
      base += n_b;
      tokens = tokens_of(p, ++b, false);
      n_b = units_of(tokens);
    }
    const int64_t rel = w - base * heads;
    const int item = static_cast<int>(kv4::quotient(rel, n_b));
    int u0 = static_cast<int>(rel - static_cast<int64_t>(item) * n_b);
    const int64_t i0 = w - u0;  // the item's first unit
    if (u0 <= kPartPages) u0 = 0;  // a boundary in an item's own units lies before it
    const int pg0 = max(0, u0 - kPartPages);
    const int u1 = static_cast<int>(min(static_cast<int64_t>(n_b), w1 - i0));
    const int g = item / p.n_sub, sub = item - g * p.n_sub;
    const int first = static_cast<int>(kv4::quotient(i0 + kPartPages, run));
    s.b = b;
    s.g = g;
    s.r0 = sub * p.tile_rows;
    s.n_r = min(p.tile_rows, p.n_rows - sub * p.tile_rows);
    s.pg0 = pg0;
    s.n_pg = u1 - kPartPages - pg0;
    s.tokens = tokens;
    s.first = first;
    s.last = static_cast<int>(kv4::quotient(i0 + n_b - 1, run));
    s.slot = i0 <= first * run ? 0 : 1;
    w = i0 + u1;
    s.more = w + kPartPages < w1;
  }
};

// One warp's ring of stages of two pages and the cursor that feeds it, which runs
// up to kStages chunks ahead of the page math and into the next part: the copies
// of a part's first pages are in flight while the part before it is merged.
// Chunk i of a part is, for warp w, pages kPair (kWarps i + w) and the one behind
// it (the last may be one page).  `issued` and `waited` number the chunks over the
// team's whole run, which gives the stage and the parity.
template <int D>
struct Feed {
  static constexpr int kBlock = kv4::block_bytes(D);
  uint32_t stage0, bar0;
  const uint8_t *cache;    // the kv head's block of page 0
  const int32_t *bt_row;   // the warp's first page of the part
  int i, n, pages;         // next chunk, chunks, pages of the part from bt_row on
  int ids_cur, ids_nxt;
  uint32_t issued, waited;  // chunks over the whole run

  // Lane l holds the id of page l & 1 of chunk 16 w + (l >> 1), w the window.
  static __device__ int fetch_ids(const int32_t *row, int pages, int w, int lane) {
    const int pg = kWarps * kPair * (16 * w + (lane >> 1)) + (lane & 1);
    return pg < pages ? row[pg] : 0;
  }
  static __device__ const int32_t *row_of(const RowsParams &p, const volatile Part &s, int warp) {
    return p.block_table + static_cast<size_t>(s.b) * p.max_blocks + s.pg0 + kPair * warp;
  }
  // Pages from this warp's first one on; none of an empty sequence's.
  static __device__ int pages_of(const volatile Part &s, int warp) {
    return s.tokens > 0 ? s.n_pg - kPair * warp : 0;
  }
  static __device__ int chunks_of(const volatile Part &s, int warp) {
    return max(0, (pages_of(s, warp) + kWarps * kPair - 1) / (kWarps * kPair));
  }
  // Turns to part s, whose first window of page ids is at hand.
  __device__ void turn_to(const RowsParams &p, const volatile Part &s, int ids, int warp,
                          int lane) {
    cache = p.cache + static_cast<size_t>(s.g) * kBlock;
    bt_row = row_of(p, s, warp);
    pages = pages_of(s, warp);
    n = chunks_of(s, warp);
    i = 0;
    ids_cur = ids;
    ids_nxt = n > 16 ? fetch_ids(bt_row, pages, 1, lane) : 0;
  }
  // The whole warp: the next chunk of the part (i < n) into its stage.
  __device__ void issue(const RowsParams &p, int lane) {
    if ((i & 15) == 0 && i > 0) {
      ids_cur = ids_nxt;
      ids_nxt = fetch_ids(bt_row, pages, (i >> 4) + 1, lane);
    }
    // lanes 0 and 1 copy a page each
    int id = __shfl_sync(kFull, ids_cur, 2 * (i & 15) + (lane & 1));
    const int here = min(2, pages - kWarps * kPair * i);
    if (lane < here) {
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) {
        record_error(p.status, PA_ERR_BAD_BLOCK);
        id = 0;  // read a page that exists; the result is flagged as invalid
      }
      const uint32_t s = issued % kStages, bar = bar0 + 8 * s;
      fence_proxy_async_smem();
      if (lane == 0) mbar_arrive_expect_tx(bar, here * kBlock);
      bulk_load(stage0 + s * (kPair * kBlock) + lane * kBlock,
                cache + static_cast<uint64_t>(static_cast<uint32_t>(id)) * p.page_bytes, kBlock,
                bar);
    }
    ++i;
    ++issued;
  }
  // Warp-uniform wait for the next chunk; its stage, or 0 when the wait ran out.
  __device__ uint32_t wait(const RowsParams &p, int lane) {
    const uint32_t s = waited % kStages, par = (waited / kStages) & 1;
    ++waited;
    if (__all_sync(kFull, mbar_wait(bar0 + 8 * s, par))) return stage0 + s * (kPair * kBlock);
    if (lane == 0) record_error(p.status, PA_ERR_TIMEOUT);
    for (uint32_t k = waited; k < issued; ++k)  // copies in flight still land
      mbar_wait(bar0 + 8 * (k % kStages), (k / kStages) & 1);
    return 0;
  }
};

// The kWarps states of each of n_r rows in shared memory, merged by the exponent
// law; fn(row, first of 4 dimensions, O, m, l).
template <int D, class Fn>
__device__ __forceinline__ void merge_rows(const float *o, const float *m, const float *l, int n_r,
                                           int tid, Fn fn) {
  for (int e = tid; e < n_r * (D / 4); e += kWarps * 32) {
    const int r = e / (D / 4), d = 4 * (e % (D / 4));
    float M = kNoKey;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) M = fmaxf(M, m[k * kTile + r]);
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float f = ex2(m[k * kTile + r] - M);
      const float4 v =
          *reinterpret_cast<const float4 *>(o + (k * kTile + r) * RowsSmem<D>::kRowStride + d);
      sum = fmaf(f, l[k * kTile + r], sum);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    fn(r, d, acc, M, sum);
  }
}

// O / l to the result's row; zeros when no key was seen (NaN stays NaN).
template <int D, bool BF16, bool OUT16>
__device__ __forceinline__ void store_row(const RowsParams &p, size_t row, int d, float4 v,
                                          float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  if constexpr (OUT16)
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + row * D + d) =
        make_uint2(pack2<BF16>(v.x, v.y), pack2<BF16>(v.z, v.w));
  else
    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + row * D + d) = v;
}

// Team c's state of an item: slot 0 when its part starts the team's run.
template <int D>
__device__ __forceinline__ float *state_of(const RowsParams &p, const volatile Part &s, int c) {
  const int slot = c > s.first ? 0 : s.slot;
  return p.ws + (static_cast<size_t>(c) * 2 + slot) * kTile * (D + 4);
}

__device__ __forceinline__ void team_sync(int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(kWarps * 32) : "memory");
}

template <int D, bool BF16, bool WIDE, bool OUT16>
__global__ void __launch_bounds__(kTeams * kWarps * 32, 1)
    kv4_rows_kernel(const RowsParams p) {
  using L = RowsSmem<D>;
  constexpr int MT = D / 16;   // row tiles of the second product (head dimensions)
  constexpr int KW = D / 32;   // 32-bit words of K codes a thread holds per token
  constexpr int VW = D / 64;   // of V codes
  extern __shared__ __align__(128) uint8_t smem_all[];
  // a team is a unit of its own from here on: own shared memory, own barrier
  const int team = threadIdx.x / (kWarps * 32), tid = threadIdx.x % (kWarps * 32);
  const int team_id = team * gridDim.x + blockIdx.x;
  uint8_t *smem = smem_all + team * L::kTeam;
  volatile uint32_t *done = reinterpret_cast<volatile uint32_t *>(smem_all + L::kDone);
  const uint32_t sb = smem_u32(smem);
  const int lane = tid & 31, warp = tid >> 5;
  const int ln = lane >> 2, lc = lane & 3;

  if (tid == 0) {
    for (int s = 0; s < kWarps * kStages; ++s) mbar_init(sb + L::kBars + 8 * s, 1);
    fence_mbar_init();
    done[team] = 0;
  }
  griddep_wait();  // inputs may come from the previous kernel in the stream
  griddep_release();
  __syncthreads();

  volatile Part *parts = reinterpret_cast<volatile Part *>(smem + L::kParts);
  volatile int *flags = reinterpret_cast<volatile int *>(smem + L::kFlags);
  Walk *walk = reinterpret_cast<Walk *>(smem + L::kWalk);
  if (warp == kWarps - 1) {  // the warp with the fewest pages plans, two parts ahead
    bool any = Walk::start(p, team_id, gridDim.x * kTeams, lane, walk);
    if (lane == 0) {
      if (any) walk->next(p, parts[0]);
      any = any && parts[0].n_pg > 0;
      if (any) {
        if (parts[0].more) walk->next(p, parts[1]);
      } else {
        done[team] = 0x7fffffff;
        p.cut[2 * team_id] = make_int4(0, 0, 0, 0);
      }
      flags[0] = any;
    }
  }
  team_sync(team);
  if (!flags[0]) return;

  // row r of a part's kv head: query r / G, head r % G
  auto q_row = [&](const volatile Part &s, int r) {
    return (static_cast<size_t>(s.b) * p.queries + r / p.group) * p.n_q_heads + s.g * p.group +
           r % p.group;
  };
  // a part's q rows to shared memory, 16 bytes a thread
  auto load_q = [&](const volatile Part &s, int buf) {
    constexpr int kChunks = D / 8;
    if (tid < s.n_r * kChunks)
      cp_async16(sb + L::kQ + buf * (kTile * D * 2) + tid * 16,
                 p.q + q_row(s, s.r0 + tid / kChunks) * D + (tid % kChunks) * 8);
  };

  Feed<D> feed;
  feed.stage0 = sb + warp * kStages * L::kStage;
  feed.bar0 = sb + L::kBars + warp * kStages * 8;
  feed.issued = feed.waited = 0;
  bool alive = true;  // false once a wait of this warp has run out
  feed.turn_to(p, parts[0],
               Feed<D>::fetch_ids(Feed<D>::row_of(p, parts[0], warp),
                                  Feed<D>::pages_of(parts[0], warp), 0, lane),
               warp, lane);
  load_q(parts[0], 0);
  for (int k = 0; k < kStages && feed.i < feed.n; ++k) feed.issue(p, lane);

  float *mer_o = reinterpret_cast<float *>(smem + L::kMergeO);
  float *mer_m = reinterpret_cast<float *>(smem + L::kMergeM);
  float *mer_l = reinterpret_cast<float *>(smem + L::kMergeL);
  const int tk = token_of(ln);
  // V rows of the tokens that score rows 2 lc and 2 lc + 1 stand for
  const int t0 = token_of(2 * lc) * kv4::row_bytes(D);
  const int t1 = token_of(2 * lc + 1) * kv4::row_bytes(D);
  cp_async_wait();
  team_sync(team);
  uint32_t chunks_done = 0;

  for (int turn = 0;; ++turn) {
    const volatile Part &part = parts[turn & 3];
    const volatile Part &then = parts[(turn + 1) & 3];
    int key0 = (part.pg0 + kPair * warp) * kPageSize;  // of the chunk at hand
    const int n_chunks = Feed<D>::chunks_of(part, warp);
    bool ahead = false;  // the feed has turned to the next part
    int ids_then = 0;
    if (part.more) {
      ids_then = Feed<D>::fetch_ids(Feed<D>::row_of(p, then, warp),
                                    Feed<D>::pages_of(then, warp), 0, lane);
      load_q(then, (turn + 1) & 1);
      if (tid == (kWarps - 1) * 32 && then.more) walk->next(p, parts[(turn + 2) & 3]);
    }
    // up to kStages chunks ahead, into the next part if need be
    auto feed_on = [&]() {
      if (ahead || !part.more) return;
      feed.turn_to(p, then, ids_then, warp, lane);
      ahead = true;
      while (feed.i < feed.n && feed.issued - feed.waited < kStages) feed.issue(p, lane);
    };

    // ---- q of this lane's column as the first product's operand
    const int n_r = part.n_r;
    uint32_t qb[2 * KW][2];
    float f0, f1, e0, e1;  // per column 2 lc, 2 lc + 1: score factor, scaled sum of q
    {
      const int col = WIDE ? ln : (ln & 3);
      float x[8 * KW];
      if (col < n_r) {
        const uint32_t row =
            sb + L::kQ + (turn & 1) * (kTile * D * 2) + col * (D * 2) + lc * (D / 2);
#pragma unroll
        for (int k = 0; k < KW; ++k) {
          const uint4 v = lds128(row + 16 * k);
          const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float2 f = unpack2<BF16>(vw[u]);
            x[8 * k + 2 * u] = f.x;
            x[8 * k + 2 * u + 1] = f.y;
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8 * KW; ++k) x[k] = 0.f;
      }
      float top = 0.f, total_q = 0.f;
#pragma unroll
      for (int k = 0; k < 8 * KW; ++k) {
        top = fmaxf(top, fabsf(x[k]));
        total_q += x[k];
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        total_q += __shfl_xor_sync(kFull, total_q, o);
      }
      // 2^ex brings the row's largest magnitude into [2^14, 2^15), or near 1 where that
      // is near the smallest of all
      const int ex = min(120, 14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127));
      const float up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
      for (int k = 0; k < KW; ++k)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int d0 = 8 * k + 2 * s;
          qb[2 * k + s][0] = pack2<false>(x[d0] * up, x[d0 + 4] * up);
          qb[2 * k + s][1] = pack2<false>(x[d0 + 1] * up, x[d0 + 5] * up);
        }
      const float f = p.qscale * __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
      const float e = p.qscale * total_q;
      f0 = __shfl_sync(kFull, f, 8 * lc);
      f1 = __shfl_sync(kFull, f, 8 * lc + 4);
      e0 = __shfl_sync(kFull, e, 8 * lc);
      e1 = __shfl_sync(kFull, e, 8 * lc + 4);
    }

    float2 o[MT][2];  // rows ln and ln + 8 of a row tile, columns 2 lc and 2 lc + 1
#pragma unroll
    for (int k = 0; k < MT; ++k) o[k][0] = o[k][1] = make_float2(0.f, 0.f);
    // per row 2 lc (x) and 2 lc + 1 (y): the running max, negated, the sums l and z
    float2 nm = make_float2(-kNoKey, -kNoKey);
    float2 l2 = make_float2(0.f, 0.f), z2 = make_float2(0.f, 0.f);
    float2 l_rest = make_float2(0.f, 0.f);  // what l lost to its last rounding
    float v_ref = 0.f, v_inv = 0.f;  // reference of scale_v (a power of two), 2^7 / it
    // !WIDE: columns 4-7 carry 2^12 (weight - head), the others the weight
    const float lift = lc < 2 ? 1.f : kRemLift, rem = lc < 2 ? 0.f : -kRemLift;

    // Keys that every row of the tile sees and this part holds end here.
    const int part_end = (part.pg0 + part.n_pg) * kPageSize;
    const int lim_all = min(part_end, OUT16 ? part.tokens - p.n_new + 1 + part.r0 / p.group
                                            : part.tokens);
    while (alive && feed.i < feed.n && feed.issued - feed.waited < kStages) feed.issue(p, lane);
    if (alive && feed.i == feed.n) feed_on();  // a short part: the next one's pages
    for (int i = 0; i < n_chunks && alive; ++i, key0 += kWarps * kPair * kPageSize) {
      // The schedulers favour older warps; without a check the first teams would
      // finish long before the last, and leave an SM with too few warps to fill it.
      if ((chunks_done & 1) == 0) {
        for (int k = 0; k < 64; ++k) {
          const uint4 all = lds128(smem_u32(smem_all + L::kDone));
          const uint32_t slowest = min(min(all.x, all.y), min(all.z, all.w));
          if (chunks_done <= slowest + kLead) break;
          __nanosleep(100);
        }
      }
      const uint32_t st = feed.wait(p, lane);
      if (st == 0) {
        alive = false;
        break;
      }

      // ---- scores S[token][row] of the two pages; this lane: tokens tk and tk + 8 of
      // each (index 2 page + half), rows 2 lc and 2 lc + 1
      float2 s[2 * kPair], d[2 * kPair];
      uint32_t vm[2 * kPair];
#pragma unroll
      for (int pg = 0; pg < kPair; ++pg) {
        const uint32_t blk = st + pg * L::kBlock;
        const uint32_t km0 = lds32(blk + kv4::meta_offset(D, 0, 0) + 4 * tk);
        const uint32_t km1 = lds32(blk + kv4::meta_offset(D, 0, 8) + 4 * tk);
        vm[2 * pg] = lds32(blk + kv4::meta_offset(D, 1, 0) + 4 * tk);
        vm[2 * pg + 1] = lds32(blk + kv4::meta_offset(D, 1, 8) + 4 * tk);
        const uint32_t row = blk + tk * kv4::row_bytes(D) + 4 * KW * lc;
        uint32_t ka[KW], kb[KW];
        if constexpr (KW == 4) {
          const uint4 a = lds128(row), b = lds128(row + 8 * kv4::row_bytes(D));
          ka[0] = a.x, ka[1] = a.y, ka[2] = a.z, ka[3] = a.w;
          kb[0] = b.x, kb[1] = b.y, kb[2] = b.z, kb[3] = b.w;
        } else {
          const uint2 a = lds64(row), b = lds64(row + 8 * kv4::row_bytes(D));
          ka[0] = a.x, ka[1] = a.y;
          kb[0] = b.x, kb[1] = b.y;
        }
        float acc[4];
#pragma unroll
        for (int k = 0; k < KW; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t xa = ka[k] >> (8 * h), xb = kb[k] >> (8 * h);
            const uint32_t a[4] = {sub_1032((xa & 0x000f000fu) | 0x64006400u),
                                   sub_1032((xb & 0x000f000fu) | 0x64006400u),
                                   sixteenth_sub_72((xa & 0x00f000f0u) | 0x64006400u),
                                   sixteenth_sub_72((xb & 0x00f000f0u) | 0x64006400u)};
            if (k + h == 0)
              mma_from_zero(acc, a, qb[0][0], qb[0][1]);
            else
              mma16816<false>(acc, a, qb[2 * k + h][0], qb[2 * k + h][1]);
          }
        const float2 k0 = unpack2<BF16>(km0), k1 = unpack2<BF16>(km1);
        // (f times acc might overflow where the key's scale brings it back)
        s[2 * pg].x = fmaf(k0.x * f0, acc[0], k0.y * e0);
        s[2 * pg].y = fmaf(k0.x * f1, acc[1], k0.y * e1);
        s[2 * pg + 1].x = fmaf(k1.x * f0, acc[2], k1.y * e0);
        s[2 * pg + 1].y = fmaf(k1.x * f1, acc[3], k1.y * e1);
      }
      const bool edge = key0 + kPair * kPageSize > lim_all;
      if (edge) {
        // last key (exclusive) each of this lane's two rows sees
        const int T = min(part.tokens, part_end);
        auto limit = [&](int col) {
          const int r = part.r0 + min(WIDE ? col : (col & 3), n_r - 1);
          return OUT16 ? min(T, part.tokens - p.n_new + 1 + r / p.group) : T;
        };
        const int lim0 = limit(2 * lc), lim1 = limit(2 * lc + 1);
#pragma unroll
        for (int u = 0; u < 2 * kPair; ++u) {
          const int t = key0 + tk + 8 * u;
          s[u].x = t < lim0 ? s[u].x : -INFINITY;
          s[u].y = t < lim1 ? s[u].y : -INFINITY;
          // rows past the end may hold anything: 0 * NaN must not enter
          if (t >= T) vm[u] = 0;
        }
      }
      float2 v[2 * kPair];
#pragma unroll
      for (int u = 0; u < 2 * kPair; ++u) {
        v[u] = unpack2<BF16>(vm[u]);
        d[u] = __fadd2_rn(s[u], nm);
      }

      // ---- move the references when a score or a scale outgrows them
      const float grow = fmaxf(fmaxf(fmaxf(d[0].x, d[0].y), fmaxf(d[1].x, d[1].y)),
                               fmaxf(fmaxf(d[2].x, d[2].y), fmaxf(d[3].x, d[3].y)));
      float vtop = fmaxf(fmaxf(fabsf(v[0].x), fabsf(v[1].x)),
                         fmaxf(fabsf(v[2].x), fabsf(v[3].x)));
      if (__any_sync(kFull, grow > kRescaleSlack || vtop > v_ref)) {
        float a = fmaxf(fmaxf(s[0].x, s[1].x), fmaxf(s[2].x, s[3].x));
        float b = fmaxf(fmaxf(s[0].y, s[1].y), fmaxf(s[2].y, s[3].y));
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          a = fmaxf(a, __shfl_xor_sync(kFull, a, x));
          b = fmaxf(b, __shfl_xor_sync(kFull, b, x));
          vtop = fmaxf(vtop, __shfl_xor_sync(kFull, vtop, x));
        }
        const float n0 = fmaxf(-nm.x, a), n1 = fmaxf(-nm.y, b);
        float2 c = make_float2(ex2(-nm.x - n0), ex2(-nm.y - n1));
        nm = make_float2(-n0, -n1);
        l2 = __fmul2_rn(l2, c);
        l_rest = __fmul2_rn(l_rest, c);
        z2 = __fmul2_rn(z2, c);
        if (vtop > v_ref) {
          // a power of two above it, and at least 2^-100
          const float up = fmaxf(
              __uint_as_float((__float_as_uint(vtop) + 0x007fffffu) & 0x7f800000u), 0x1p-100f);
          c = __fmul2_rn(c, make_float2(v_ref / up, v_ref / up));
          v_ref = up;
          v_inv = 128.f / up;
        }
#pragma unroll
        for (int k = 0; k < MT; ++k) {
          o[k][0] = __fmul2_rn(o[k][0], c);
          o[k][1] = __fmul2_rn(o[k][1], c);
        }
#pragma unroll
        for (int u = 0; u < 2 * kPair; ++u) d[u] = __fadd2_rn(s[u], nm);
      }

      // ---- weights, as the second product's operand
      uint32_t hi[2 * kPair], lo[2 * kPair];
      float2 sum = l_rest;  // small weights add up before they meet a large l
#pragma unroll
      for (int u = 0; u < 2 * kPair; ++u) {
        const float2 pr = make_float2(ex2(d[u].x), ex2(d[u].y));
        sum = __fadd2_rn(sum, pr);
        const float x = v[u].x * v_inv;
        float2 wt = make_float2(pr.x * x, pr.y * x);
        const float mid = fmaf(-0.5f, v[u].x, v[u].y);  // of the row
        float2 zt = make_float2(mid, mid);
        if (OUT16 && edge) {  // a key that this row does not see may not be finite
          if (s[u].x == -INFINITY) wt.x = zt.x = 0.f;
          if (s[u].y == -INFINITY) wt.y = zt.y = 0.f;
        }
        z2 = make_float2(fmaf(pr.x, zt.x, z2.x), fmaf(pr.y, zt.y, z2.y));
        const uint32_t head = pack2<false>(wt.x, wt.y);
        const float2 back = unpack2<false>(head);
        if constexpr (WIDE) {
          hi[u] = transpose8x8(head);
          lo[u] = transpose8x8(
              pack2<false>((wt.x - back.x) * kRemLift, (wt.y - back.y) * kRemLift));
        } else {  // the head term again, or the remainder
          const float2 mine = __ffma2_rn(make_float2(rem, rem), back,
                                         __fmul2_rn(wt, make_float2(lift, lift)));
          hi[u] = transpose8x8(pack2<false>(mine.x, mine.y));
          lo[u] = 0;
        }
      }

      {
        const float2 l_new = __fadd2_rn(l2, sum);
        l_rest = __fadd2_rn(sum, __fadd2_rn(l2, make_float2(-l_new.x, -l_new.y)));
        l2 = l_new;
      }

      // ---- O[dimension][row] += V^T P, the chunk's sum in an accumulator of its own
      uint32_t va[kPair][4][VW];
#pragma unroll
      for (int pg = 0; pg < kPair; ++pg) {
        const uint32_t col = st + pg * L::kBlock + kv4::code_offset(D, 1, 0) + 4 * VW * ln;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t at = col + (u & 1 ? t1 : t0) + 8 * (u >> 1) * kv4::row_bytes(D);
          if constexpr (VW == 2) {
            const uint2 x = lds64(at);
            va[pg][u][0] = x.x, va[pg][u][1] = x.y;
          } else {
            va[pg][u][0] = lds32(at);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < VW; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // nibbles 4 h .. 4 h + 3 of two tokens' words, one token a half
          uint32_t x[kPair], y[kPair];
#pragma unroll
          for (int pg = 0; pg < kPair; ++pg) {
            x[pg] = __byte_perm(va[pg][0][j], va[pg][1][j], h ? 0x7632 : 0x5410);
            y[pg] = __byte_perm(va[pg][2][j], va[pg][3][j], h ? 0x7632 : 0x5410);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t a[kPair][4];
#pragma unroll
            for (int pg = 0; pg < kPair; ++pg) {
              const uint32_t xs = x[pg] >> (8 * u), ys = y[pg] >> (8 * u);
              a[pg][0] = centred<24>(xs & 0x000f000fu);
              a[pg][1] = centred<20>(xs & 0x00f000f0u);
              a[pg][2] = centred<24>(ys & 0x000f000fu);
              a[pg][3] = centred<20>(ys & 0x00f000f0u);
            }
            float t[4];
            float2 (&ok)[2] = o[4 * j + 2 * h + u];
            if constexpr (WIDE) {
              mma_from_zero(t, a[0], lo[0], lo[1]);
              mma16816<false>(t, a[1], lo[2], lo[3]);
              const float2 down = make_float2(1.f / kRemLift, 1.f / kRemLift);
              ok[0] = __ffma2_rn(make_float2(t[0], t[1]), down, ok[0]);
              ok[1] = __ffma2_rn(make_float2(t[2], t[3]), down, ok[1]);
            }
            mma_from_zero(t, a[0], hi[0], hi[1]);
            mma16816<false>(t, a[1], hi[2], hi[3]);
            ok[0] = __fadd2_rn(ok[0], make_float2(t[0], t[1]));
            ok[1] = __fadd2_rn(ok[1], make_float2(t[2], t[3]));
          }
        }
      __syncwarp();  // the stage has been read by every lane
      if (feed.i < feed.n)
        feed.issue(p, lane);
      else
        feed_on();
      ++chunks_done;
      if (tid == 0) done[team] = chunks_done;
    }

    // ---- the warp's state to shared memory: O is O[d = (D / 8) ln + 2 k + {0, 1}]
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l2.x += __shfl_xor_sync(kFull, l2.x, x);
      l2.y += __shfl_xor_sync(kFull, l2.y, x);
      z2.x += __shfl_xor_sync(kFull, z2.x, x);
      z2.y += __shfl_xor_sync(kFull, z2.y, x);
    }
    cp_async_wait();  // the next part's q
    team_sync(team);  // the part before this one has been merged
    const float back = v_ref * 0x1p2f;  // V's operands are over 2^9, the weights over 2^-7
#pragma unroll
    for (int k = 0; k < MT; ++k) {
      float2 a = make_float2(o[k][0].x, o[k][1].x), b = make_float2(o[k][0].y, o[k][1].y);
      if constexpr (!WIDE) {  // columns 4-7 hold the remainder terms of 0-3
        a.x = fmaf(__shfl_xor_sync(kFull, a.x, 2), 1.f / kRemLift, a.x);
        a.y = fmaf(__shfl_xor_sync(kFull, a.y, 2), 1.f / kRemLift, a.y);
        b.x = fmaf(__shfl_xor_sync(kFull, b.x, 2), 1.f / kRemLift, b.x);
        b.y = fmaf(__shfl_xor_sync(kFull, b.y, 2), 1.f / kRemLift, b.y);
      }
      if (WIDE || lc < 2) {
        float *dst = mer_o + (warp * kTile + 2 * lc) * L::kRowStride + (D / 8) * ln + 2 * k;
        *reinterpret_cast<float2 *>(dst) =
            make_float2(fmaf(a.x, back, z2.x), fmaf(a.y, back, z2.x));
        *reinterpret_cast<float2 *>(dst + L::kRowStride) =
            make_float2(fmaf(b.x, back, z2.y), fmaf(b.y, back, z2.y));
      }
    }
    if (ln == 0 && (WIDE || lc < 2)) {
      mer_m[warp * kTile + 2 * lc] = -nm.x;
      mer_m[warp * kTile + 2 * lc + 1] = -nm.y;
      mer_l[warp * kTile + 2 * lc] = l2.x;
      mer_l[warp * kTile + 2 * lc + 1] = l2.y;
    }
    team_sync(team);

    const bool whole = part.first == part.last;
    // the warps' states of a row merged: dimensions d .. d + 3, and (m, l)
    merge_rows<D>(mer_o, mer_m, mer_l, n_r, tid, [&](int r, int d, float4 acc, float m, float l) {
      if (whole) {
        store_row<D, BF16, OUT16>(p, q_row(part, part.r0 + r), d, acc, l);
      } else {
        float *dst = state_of<D>(p, part, team_id) + r * (D + 4);
        *reinterpret_cast<float4 *>(dst + d) = acc;
        if (d == 0) *reinterpret_cast<float2 *>(dst + D) = make_float2(m, l);
      }
    });
    if (!part.more) {
      // the run's last part may start an item that later teams hold more of
      if (tid == 0) {
        const bool cut = part.last > team_id && part.first == team_id;
        p.cut[2 * team_id] = make_int4(cut ? part.last - team_id + 1 : 0, part.slot, part.n_r, 0);
        p.cut[2 * team_id + 1] = make_int4(part.b, part.g, part.r0, 0);
        done[team] = 0x7fffffff;
      }
      break;
    }
  }
}

// ---- items cut between teams: the states of one that starts in team c's run are
// folded by GROUPS groups of threads, a thread a (row, 4 dimensions), a few states a
// step; group g takes states g, g + GROUPS, ..  One group, one CTA a team; or, where
// few items have many states each, kTeams of each, so that a round of loads takes them
// all (launch_rows_t).
template <int D, bool BF16, bool OUT16, int GROUPS>
__global__ void __launch_bounds__(GROUPS * kTile * D / 4) kv4_fold_kernel(const RowsParams p) {
  constexpr int kBatch = GROUPS > 1 ? 5 : 4, kState = kTile * (D + 4), kRowD = kTile * D / 4;
  __shared__ float4 sums[GROUPS > 1 ? GROUPS - 1 : 1][kRowD];
  __shared__ float2 tops[GROUPS > 1 ? GROUPS - 1 : 1][kTile];
  const int g = threadIdx.x / kRowD, th = threadIdx.x % kRowD;
  const int r = th / (D / 4), d = 4 * (th % (D / 4));
  griddep_release();
  griddep_wait();  // the states
  int4 cuts[GROUPS];
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) cuts[i] = __ldcg(p.cut + 2 * (blockIdx.x + i * gridDim.x));
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) {
    const int4 cut = cuts[i];
    const int c = blockIdx.x + i * gridDim.x, n = cut.x;
    if (n == 0) continue;
    const bool real = r < cut.z;
    float m = kNoKey, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto fold = [&](float2 ml, float4 v) {
      const float mn = fmaxf(m, ml.x);
      const float a = ex2(m - mn), f = ex2(ml.x - mn);
      acc.x = fmaf(acc.x, a, v.x * f);
      acc.y = fmaf(acc.y, a, v.y * f);
      acc.z = fmaf(acc.z, a, v.z * f);
      acc.w = fmaf(acc.w, a, v.w * f);
      l = fmaf(l, a, ml.y * f);
      m = mn;
    };
    const float *first = p.ws + (static_cast<size_t>(c) * 2 + cut.y) * kState + r * (D + 4);
    const float *rest = p.ws + static_cast<size_t>(c) * 2 * kState + r * (D + 4);
    for (int k0 = g; k0 < n && real; k0 += kBatch * GROUPS) {
      float2 ml[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {  // past the last state, it again
        const int k = min(k0 + u * GROUPS, n - 1);
        const float *sp = k == 0 ? first : rest + static_cast<size_t>(k) * 2 * kState;
        ml[u] = __ldcg(reinterpret_cast<const float2 *>(sp + D));
        v[u] = __ldcg(reinterpret_cast<const float4 *>(sp + d));
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (k0 + u * GROUPS < n) fold(ml[u], v[u]);
    }
    if constexpr (GROUPS > 1) {
      if (i > 0) __syncthreads();  // the item before has been read
      if (g > 0) {
        sums[g - 1][th] = acc;
        if (d == 0) tops[g - 1][r] = make_float2(m, l);
      }
      __syncthreads();
      if (g > 0) continue;
#pragma unroll
      for (int k = 0; k < GROUPS - 1; ++k) fold(tops[k][r], sums[k][th]);
    }
    if (!real) continue;
    const int4 at = __ldcg(p.cut + 2 * c + 1);
    const int row = at.z + r;
    store_row<D, BF16, OUT16>(
        p, (static_cast<size_t>(at.x) * p.queries + row / p.group) * p.n_q_heads +
               at.y * p.group + row % p.group, d, acc, l);
  }
}

template <int D, bool BF16, bool WIDE, bool OUT16>
int launch_rows_t(const RowsParams &p, int ctas, cudaStream_t stream) {
  auto kern = kv4_rows_kernel<D, BF16, WIDE, OUT16>;
  static ContextCache<bool> smem_set;
  if (set_smem_limit(kern, RowsSmem<D>::kBytes, smem_set) != PA_OK) return PA_ERR_CUDA;
  if (launch_pdl(kern, dim3(ctas), dim3(kTeams * kWarps * 32), RowsSmem<D>::kBytes, stream, p) !=
          cudaSuccess)
    return PA_ERR_CUDA;
  // A CTA of kTeams groups looks after kTeams runs: worth it from about 20 states an item.
  // One group against kTeams, us a call (head_dim 128):
  //   76 states  1 x 131072 tokens, 8 / 1 heads  87.5 / 52.4   1 x 32768, 32 / 8  26.9 / 21.3
  //   38         2 x 16384, 64 / 8               24.8 / 23.0
  //   19         4 x 32768, 64 / 8               51.1 / 52.2   4 x 8192, 32 / 8   19.9 / 19.1
  //   10         4 x 2 queries over 32768, 64 / 8  84.8 / 92.0
  const bool few = static_cast<int64_t>(p.batch) * p.n_kv_heads * p.n_sub * 20 <=
                   static_cast<int64_t>(ctas) * kTeams;
  const cudaError_t e =
      few ? launch_pdl(kv4_fold_kernel<D, BF16, OUT16, kTeams>, dim3(ctas),
                       dim3(kTeams * kTile * D / 4), 0, stream, p)
          : launch_pdl(kv4_fold_kernel<D, BF16, OUT16, 1>, dim3(ctas * kTeams),
                       dim3(kTile * D / 4), 0, stream, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int D, bool BF16>
int launch_rows_d(const RowsParams &p, int ctas, cudaStream_t stream) {
  const bool wide = p.tile_rows > 4;
  if (p.n_new > 0)
    return wide ? launch_rows_t<D, BF16, true, true>(p, ctas, stream)
                : launch_rows_t<D, BF16, false, true>(p, ctas, stream);
  return wide ? launch_rows_t<D, BF16, true, false>(p, ctas, stream)
              : launch_rows_t<D, BF16, false, false>(p, ctas, stream);
}

size_t partials_bytes(int head_dim, int ctas) {
  return static_cast<size_t>(ctas) * kTeams * 2 * kTile * (head_dim + 4) * sizeof(float);
}

}  // namespace

size_t kv4_rows_workspace_bytes(int head_dim, int sms) {
  return partials_bytes(head_dim, sms) + static_cast<size_t>(sms) * kTeams * 2 * sizeof(int4);
}

int launch_kv4_rows(const Kv4AttentionLaunch &a, cudaStream_t stream) {
  const int ctas = sm_count();
  if (ctas <= 0) return PA_ERR_CUDA;
  RowsParams p;
  p.q = static_cast<const uint16_t *>(a.q);
  p.cache = a.cache;
  p.block_table = a.block_table;
  p.ctx_lens = a.ctx_lens;
  p.out = a.out;
  p.ws = static_cast<float *>(a.workspace);
  p.cut = reinterpret_cast<int4 *>(static_cast<char *>(a.workspace) +
                                   partials_bytes(a.head_dim, ctas));
  p.status = a.status;
  p.qscale = a.scale * kLog2e;
  p.n_new = a.n_new;
  p.queries = a.n_new > 0 ? a.n_new : 1;
  p.n_q_heads = a.n_q_heads;
  p.n_kv_heads = a.n_kv_heads;
  p.group = a.n_q_heads / a.n_kv_heads;
  p.batch = a.batch;
  p.max_blocks = a.max_blocks;
  p.num_pages = a.num_pages;
  p.page_bytes = static_cast<uint32_t>(a.n_kv_heads) * kv4::block_bytes(a.head_dim);
  p.n_rows = p.queries * p.group;
  p.n_sub = (p.n_rows + kTile - 1) / kTile;
  p.tile_rows = (p.n_rows + p.n_sub - 1) / p.n_sub;
  p.n_sub = (p.n_rows + p.tile_rows - 1) / p.tile_rows;
  if (a.head_dim == 128)
    return a.bf16 ? launch_rows_d<128, true>(p, ctas, stream)
                  : launch_rows_d<128, false>(p, ctas, stream);
  return a.bf16 ? launch_rows_d<64, true>(p, ctas, stream)
                : launch_rows_d<64, false>(p, ctas, stream);
}

}  // namespace pa
