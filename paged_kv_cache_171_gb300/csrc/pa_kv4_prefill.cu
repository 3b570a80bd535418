// pa_kv4_prefill.cu -- chunked-prefill attention over the 4-bit paged cache on the
// 5th-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// Query i of sequence b (0 <= i < n_new) attends keys 0 .. ctx_lens[b] + i of the
// values K = zero_k + scale_k (c - 8), V alike, c the 4-bit codes.  Per row tile and
// key tile: S = Q K^T (tcgen05, 128 x 128 x head_dim), an online softmax, and O +=
// P V with P in tensor memory.  All operands are fp16, 11 significant bits; a key
// tile is turned into operand tiles once for 256 query rows.
//
// Two forms, by the cache's type (EXACT below):
//  * bf16: the converters store scale (c - 8) of K, which fp16 holds exactly (8 bits times
//    3), and zero + scale (c - 8) of V, over a power of two above the largest magnitude of
//    32 keys (k_ref, v_ref).  zero_k sum q comes out of the same product: 16 columns more,
//    of which K has the zero twice and Q the sum in two terms.  So S is exact to fp32's
//    last bits (with K rounded like V, the error in the weights grew with the scores: rows
//    at scores of N(0, 10) were up to 1.1% off, now 0.24%); V is off by two half steps of
//    2^-11 and P by one, well below the bf16 result's own rounding of 2^-8; and the softmax
//    works on S as it comes: a factor for each 32 keys in its exponent.
//    Operands reach up to 2^-7 in fp16, which has all its bits down to 2^-14: where a
//    key's largest magnitude is below 2^-5 of the reference, that is lowered by as much
//    (K's by 2^15 at most, V's by 2^11, which P gives up), and each key is converted over
//    a power of two of its own before it is moved there.  At the common reference one key
//    1024 times the others, whatever its weight, left those 31 with an error of 1.3%.
//  * fp16: that would be as much as the result's rounding, so the codes enter the
//    products exactly, as 2 c - 15 ((x & 0x001e001e) | 0x64006400 is 1024 + 2 c, x the
//    word shifted left by one), and the softmax threads apply the rest: with the row's
//    middle mid = zero - scale / 2,
//      s_t = scale_k[t] / 2 S_t + mid_k[t] sum q,   P = p_t scale_v[t] / v_ref,
//      z += p_t mid_v[t],                           out = (O v_ref / 2 + z) / l,
//    reading each key's scales and middles from shared memory.  The operand is centred
//    because the tensor cores round O toward zero at every 16 keys: with c - 8, whose
//    mean over a row is near -1/2, O grew with the number of keys where the result's
//    terms cancel, and rows over 131072 keys were off by 0.28%; so by 0.03%.
// P carries v_ref over the largest v_ref so far; when that grows, O is rescaled like
// at a move of the running maximum.
//
// Tiles.  An item is 256 consecutive rows (query, head) of one kv head, whatever
// the group size: row r is query r / G, head r % G.  It is two row tiles A and B of
// 128 rows that share every key tile of 128 keys (8 pages).  The tensor pipe
// alternates between them: B's softmax of key tile j starts once A has handed over
// its weights of j, A's of j + 1 once B has handed over those of j.
//
// An item of at most 128 rows (a short chunk) has its rows in both tiles, which split
// the key tiles instead: A the even ones, B the odd ones, so that one's softmax still
// overlaps the other's products.  At the end A reads both O's (the lanes hold the same
// rows) and merges the two states.  Of at most 64 rows, the softmax warps of the upper
// rows have none: these four turn the odd key tiles' codes, the converters the even ones'
// (4 x 4 queries, 64 / 8 heads, over 32k keys: 114 -> 102 us when it came in).
//
// Warp roles (one CTA an SM): warps 0 and 1 issue the MMAs of row tiles A and B, warps
// 4-7 turn codes into the K and V operand tiles (two stages each): a warp 32 keys of
// each tile, from a ring of pages that it fills for itself by bulk copies.  Warps 8-11
// and 12-15 are the softmax of A and B, a thread a row.  Warp 2 plans the run's next
// part during this one.  Every hand-off is an mbarrier and every wait is bounded.
//
// Nibbles.  x & 0x000f000f holds nibbles 0 and 4 of a word in two 16-bit halves, and so
// on: a fp16 pair is made of nibbles four apart.  The operand tiles keep that order of
// dimensions (0 4 1 5 2 6 3 7 of each eight): Q is stored in it, and the result is put
// back into the natural one on its way out.
//
// Work split.  The key tiles of all items, laid end to end, are cut into equal runs,
// one an SM: 256 items on 152 SMs take 1.7 items' time, not two, and a single
// sequence's chunk over a long context fills the GPU.  An item counts a few key tiles
// more than it has (part_tiles), for what starting and ending it costs.  An item cut
// between CTAs leaves an fp32 state (O, m, l) a row and CTA, folded by a second kernel.
//
// Bound.  A long chunk: the chain of a key tile, from the codes over S and the softmax
// to P V (tensor pipe 45% busy, issue 49%): 4 x 512 queries of 32 / 8 heads over 8192
// tokens, bf16 288 us (2.84e11 operations, 0.99 PFLOP/s); fp16 468 us, whose softmax reads
// 16 bytes a key and thread from shared memory (tensor 27%, issue 40%).  Few rows: turning
// the codes (4 x 4 queries of 64 / 8 heads over 32k tokens 86 us, 1.7 TB/s of codes; fp16
// 126).  Where every 32 keys span a wide range, the bf16 calls take 474 and 146 us.
#include <float.h>

#include <atomic>

#include "pa_kv4.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// A row's running maximum moves once a score passes it by kSlack (powers of two); the
// weights enter the tensor cores times 2^kLift, 2^15 at most.  What fp16 has left below is
// for the keys beside one that takes nearly all of the weight (32k of them beside one of
// 0.999 weigh 2^-25 each): 11 bits down to 2^-25 of the reference, steps of 2^-35 below.
constexpr float kSlack = 4.0f, kLift = 11.0f;
static_assert(kSlack + kLift <= 15.0f, "a weight stays below fp16's largest value");
constexpr float kNoKey = -3.402823466e38f;  // running max of a row before its first key
constexpr unsigned kFull = 0xffffffffu;
constexpr int kRows = 128, kKeys = 128;     // a row tile, a key tile
constexpr int kItemRows = 2 * kRows;
constexpr int kStages = 2;                  // of K and of V
constexpr int kConvertWarp0 = 4, kSoftmaxWarp0 = 8;
constexpr int kThreads = 16 * 32;

struct PrefillParams {
  const uint16_t *q;
  const uint8_t *cache;
  const int32_t *block_table, *ctx_lens;
  uint16_t *out;
  float *ws;    // [CTA][2][kItemRows][D + 4] partial states
  int4 *cut;    // [CTA][2] the item that starts in the CTA's run and leaves it
  int *status;
  float qscale;     // |scale| * log2 e, at least 1e-30
  uint32_t qsign;   // 0x80008000 when scale < 0 (folded into Q), else 0
  int n_new, n_q_heads, n_kv_heads, group, batch, max_blocks, num_pages;
  int n_rows, n_items;  // rows a kv head, items a kv head
  int part_tiles;       // what a part's start and end cost, in key tiles
  uint32_t page_bytes;
};

template <int D, bool EXACT, bool FEW>
struct PrefillSmem {
  static constexpr int kRawPages = FEW ? 3 : 2;       // a converter warp's ring (below)
  static constexpr int kColBlk = kRows * 128;         // one 64-column block, 128 rows
  static constexpr int kTile = (D / 64) * kColBlk;    // 128 rows x D, 16 bits
  static constexpr int kQ = 0;                        // Q_A, Q_B
  static constexpr int kK = kQ + 2 * kTile;
  static constexpr int kV = kK + kStages * kTile;
  // EXACT: per stage and pair of keys scale_k / 2 x2, mid_k x2 (both times qscale),
  // scale_v / v_ref x2, mid_v x2.  Else the factor of each row's S.
  static constexpr int kMeta = kV + kStages * kTile;
  static constexpr int kMetaBytes = EXACT ? kStages * (kKeys / 2) * 32 : 2 * kRows * 4;
  // the converters' rings of pages: the first group's, and, where the two row tiles are
  // one and Q_B not needed, the second group's (two pages a warp are enough while it turns
  // a tile for 256 rows: 4 x 512 queries over 8192 tokens 277 us with three, 271 with two;
  // for few rows 85 and 88)
  static constexpr int kRing = 4 * kRawPages * kv4::block_bytes(D);
  static constexpr int kRaw = kMeta + kMetaBytes, kRaw1 = kQ + kTile;
  static_assert(kRing <= kTile, "room in Q_B");
  // Not EXACT: the 8 columns of zeros and sums behind Q's and K's, 16 bytes a row, and the
  // zeros that stand for 8 more.
  static constexpr int kExtra = EXACT ? 0 : kRows * 16;
  static constexpr bool kInQ = FEW && kRing + (1 + kStages) * kExtra <= kTile;
  static constexpr int kEnd = kRaw + kRing;
  static constexpr int kQX = kInQ ? kRaw1 + kRing : kEnd;       // of Q_A, Q_B
  static constexpr int kKX = kQX + (FEW ? 1 : 2) * kExtra;      // of the stages
  static constexpr int kZeros = kInQ ? kEnd : kKX + kStages * kExtra;
  // per stage: k_ref of each 32 keys, then v_ref
  static constexpr int kRef = kZeros + kExtra;
  static constexpr int kBars = kRef + kStages * 32;
  static constexpr int kSlot = kBars + 2 * 46 * 8;        // TMEM address, abort flag
  static constexpr int kPart = kSlot + 16;            // this part and the next
  static constexpr int kWalk = kPart + 2 * 64;
  static constexpr int kBytes = kWalk + 64;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 232448, "exceeds the per-CTA shared memory limit");
};

enum {
  kBarK = 0,       // K stage s converted, at + s (4 arrivals)
  kBarV = 2,       // V stage s and its references (4 arrivals)
  kBarKFree = 4,   // K stage s read by row tile x's S MMA (commit), at + 2 x + s
  kBarVFree = 8,   // V stage s read by row tile x's P V MMAs, at + 2 x + s
  kBarS = 12,      // S_x in TMEM (commit), at + x
  kBarP = 14,      // keys 64 h .. 64 h + 63 of P_x in TMEM, at + 2 x + h (4 arrivals)
  kBarO = 18,      // the last P_x V done (commit), at + x
  kBarDrain = 20,  // an MMA warp's own drain on its failure path, at + x
  kBarRaw = 22,    // page s of the ring of converter w of group c, at + 3 (4 c + w) + s
  kNumBars = 46
};

// The part of one item that a CTA's run holds.
struct TilePart {
  int b, g, row0;      // sequence, kv head, first row of the item
  int ctx;             // cached tokens of the sequence
  int t0, nt;          // key tiles
  int first, last;     // CTAs that hold the item
  int slot;            // of the first one's state: 0 when the item starts its run
  int more;            // the run goes on behind this part
};
static_assert(sizeof(TilePart) <= 64, "room in shared memory");

// How a part uses the two row tiles.
struct Tiling {
  int n_active;  // row tiles at work
  bool split;    // they hold the same rows and split the key tiles
  __device__ Tiling(int row0, int nt, int n_rows) {
    const bool one = row0 + kRows >= n_rows;
    split = one && nt >= 2;
    n_active = one && !split ? 1 : 2;
  }
  // The row tiles that read stage s (of tile t = s mod 2 when split): first and last.
  __device__ int first(int s) const { return split ? s : 0; }
  __device__ int last(int s) const { return split ? s : n_active - 1; }
};
static_assert(kStages == 2, "split key tiles: a stage belongs to one row tile");

// The CTA's run [w, w1) of the flattened list of units.  A boundary between runs in or
// right behind an item's part_tiles units counts as lying before the item, so that every
// part has a key tile.
struct TileWalk {
  int64_t w, w1, run, base;  // base: units of the sequences before b
  int b, ctx, per_head;      // the sequence; units of one of its kv heads

  static __device__ int ctx_of(const PrefillParams &p, int b, bool report) {
    const int most = p.max_blocks * kPageSize - p.n_new;
    int t = p.ctx_lens[b];
    if (t < 0 || t > most) {
      if (report) record_error(p.status, PA_ERR_BAD_CTX);
      t = t < 0 ? 0 : most;
    }
    return t;
  }
  // Units of item k (of a kv head) of a sequence with ctx cached tokens: the key tiles
  // that it sees behind part_tiles of its own.
  static __device__ int units_of(const PrefillParams &p, int ctx, int k) {
    const int last_row = min(p.n_rows, (k + 1) * kItemRows) - 1;
    return (ctx + last_row / p.group) / kKeys + 1 + p.part_tiles;
  }
  static __device__ int head_units(const PrefillParams &p, int ctx) {
    int n = 0;
    for (int k = 0; k < p.n_items; ++k) n += units_of(p, ctx, k);
    return n;
  }
  // The whole warp; lane 0 keeps the result in *out.  False: no run.
  static __device__ bool start(const PrefillParams &p, int lane, TileWalk *out) {
    TileWalk x;
    const int per = (p.batch + 31) / 32;
    const int b0 = min(p.batch, lane * per), b1 = min(p.batch, b0 + per);
    int64_t sum = 0;
    for (int i = b0; i < b1; ++i) sum += head_units(p, ctx_of(p, i, blockIdx.x == 0));
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    const int64_t total = __shfl_sync(kFull, incl, 31) * p.n_kv_heads;
    x.run = kv4::quotient(total + gridDim.x - 1, gridDim.x);
    x.w = blockIdx.x * x.run;
    x.w1 = min(total, x.w + x.run);
    if (x.w >= x.w1) return false;
    const int src = __ffs(__ballot_sync(kFull, incl * p.n_kv_heads > x.w)) - 1;
    x.b = __shfl_sync(kFull, b0, src);
    x.base = __shfl_sync(kFull, incl - sum, src) * p.n_kv_heads;
    x.ctx = ctx_of(p, x.b, false);
    x.per_head = head_units(p, x.ctx);
    if (lane == 0) *out = x;
    return true;
  }
  __device__ void next(const PrefillParams &p, TilePart &s) {
    while (base + static_cast<int64_t>(per_head) * p.n_kv_heads <= w) {
      base += static_cast<int64_t>(per_head) * p.n_kv_heads;
      ctx = ctx_of(p, ++b, false);
      per_head = head_units(p, ctx);
    }
    const int64_t rel = w - base;
    const int g = static_cast<int>(kv4::quotient(rel, per_head));
    int u0 = static_cast<int>(rel - static_cast<int64_t>(g) * per_head), k = 0, n;
    while (u0 >= (n = units_of(p, ctx, k))) {
      u0 -= n;
      ++k;
    }
    const int64_t i0 = w - u0;  // the item's first unit
    if (u0 <= p.part_tiles) u0 = 0;  // a boundary in an item's own units lies before it
    const int u1 = static_cast<int>(min(static_cast<int64_t>(n), w1 - i0));
    s.b = b;
    s.g = g;
    s.row0 = k * kItemRows;
    s.ctx = ctx;
    s.t0 = max(0, u0 - p.part_tiles);
    s.nt = u1 - p.part_tiles - s.t0;  // (below 1: the run ends before the item's tiles begin)
    s.first = static_cast<int>(kv4::quotient(i0 + p.part_tiles, run));
    s.last = static_cast<int>(kv4::quotient(i0 + n - 1, run));
    s.slot = i0 <= s.first * run ? 0 : 1;
    w = i0 + u1;
    s.more = w + p.part_tiles < w1;
  }
};

// Row r of a kv head in the [batch][n_new][n_q_heads] order of q and out.
__device__ __forceinline__ size_t row_at(const PrefillParams &p, int b, int g, int r) {
  return (static_cast<size_t>(b) * p.n_new + r / p.group) * p.n_q_heads + g * p.group +
         r % p.group;
}

// The eight codes of a word, in the order 0 4 1 5 2 6 3 7.  EXACT: as 2 c - 15.  Else as
// zero + scale (c - 8) over 2^7 ref: (x & 0x000f000f) is the fp16 subnormal pair
// c 2^-24 and (x & 0x00f000f0) is c 2^-20, so with s24 = scale 2^24, s20 = scale 2^20
// and z = zero - 8 scale (K: -8 scale) a pair is one AND and one FMA.
template <bool EXACT>
__device__ __forceinline__ uint4 operand(uint32_t x, __half2 s24, __half2 s20, __half2 z) {
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t w;
    __half2 r;
    if constexpr (EXACT) {
      w = ((k == 0 ? x << 1 : x >> (4 * k - 1)) & 0x001e001eu) | 0x64006400u;
      r = __hsub2(*reinterpret_cast<const __half2 *>(&w), __float2half2_rn(1039.f));
    } else {
      w = (x >> (8 * (k >> 1))) & ((k & 1) ? 0x00f000f0u : 0x000f000fu);
      r = __hfma2((k & 1) ? s20 : s24, *reinterpret_cast<const __half2 *>(&w), z);
    }
    o[k] = *reinterpret_cast<const uint32_t *>(&r);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A power of two of at least x >= 0, kept to 2^-100 .. 2^126 (x / 2^126 is below 4).
__device__ __forceinline__ float above(float x) {
  const float up = __uint_as_float((__float_as_uint(x) + 0x007fffffu) & 0x7f800000u);
  return fminf(fmaxf(up, 0x1p-100f), 0x1p126f);
}

// The exponent of a power of two, and 2^k for -126 <= k <= 127.
__device__ __forceinline__ int exponent(float x) {
  return static_cast<int>(__float_as_uint(x) >> 23) - 127;
}
__device__ __forceinline__ float exp2i(int k) {
  return __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
}

// Converter warp w of group c: keys 32 w .. 32 w + 31 (two pages) of the key tiles c,
// c + step, .., K then V, and their references and, in the exact form, scales and zeros.
// The pages come through a ring of the warp's own, by bulk copies a tile (FEW: 1.5) ahead.
//
// A row past the sequence's end stands for zeros (it may hold anything, and 0 * NaN is
// NaN).  A key or value row that is not finite makes its key's score NaN, which
// masking removes for the queries that do not see it, and its values zero.
template <int D, bool BF16, bool EXACT, bool FEW>
__device__ __forceinline__ void convert_tiles(int c, int step, int w, const PrefillParams &p,
                                              const TilePart &part, uint32_t sb, uint32_t bars,
                                              uint8_t *smem, const Tiling &tl,
                                              volatile int *abort_flag, int lane) {
  using L = PrefillSmem<D, EXACT, FEW>;
  constexpr int kRawPages = L::kRawPages;
  constexpr int kBlock = kv4::block_bytes(D);
  constexpr int kPieces = D / 32;                // 16-byte pieces of a row's codes
  constexpr int kIters = kPageSize * kPieces / 32;  // pieces a lane and page
  constexpr int kPagesTile = kKeys / kPageSize;
  auto bar = [&](int i) { return bars + 8 * i; };
  const int tokens = part.ctx + p.n_new;
  const int n_pages = (tokens + kPageSize - 1) / kPageSize;
  const int32_t *bt_row = p.block_table + static_cast<size_t>(part.b) * p.max_blocks;
  const uint8_t *head = p.cache + static_cast<size_t>(part.g) * kBlock;
  // the upper column block's pieces (head_dim 128) take another row than the lower's, so
  // that no two lanes of a store meet in a bank
  const int piece = lane % kPieces, row_l = (lane / kPieces) ^ (piece >= 2 ? 4 : 0);
  const uint32_t raw0 = sb + (c == 0 ? L::kRaw : L::kRaw1) + w * kRawPages * kBlock;
  const uint32_t raw_bar = bar(kBarRaw + kRawPages * (4 * c + w));

  // Page ids: lane l holds page l & 1 of the warp's two in its tile 16 v + (l >> 1), v
  // the window; past the sequence's end page 0, which is masked.
  auto ids_of = [&](int v) {
    const int t = c + (16 * v + (lane >> 1)) * step;
    const int pg = (part.t0 + t) * kPagesTile + 2 * w + (lane & 1);
    return t < part.nt && pg < n_pages ? bt_row[pg] : 0;
  };
  int ids = ids_of(0), ids_next = ids_of(1);
  int issued = 0;  // the warp's pages, 2 a tile; page i sits in ring slot i % kRawPages
  const int total = c < part.nt ? 2 * ((part.nt - c + step - 1) / step) : 0;
  // the next pages, as many as `most` (1 or 2), a lane each
  auto issue = [&](int most) {
    const int n = min(most, total - issued);
    if ((issued & 31) == 0 && issued > 0) {
      ids = ids_next;
      ids_next = ids_of((issued >> 5) + 1);
    }
    // the second page may be the next window's first
    const int from = (issued + (lane & 1)) & 31;
    int id = __shfl_sync(kFull, ids, from);
    const int id_next = __shfl_sync(kFull, ids_next, from);
    if ((issued & 31) == 31 && (lane & 1)) id = id_next;
    if (lane < n) {  // (behind a proxy fence, where a slot has been read)
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) {
        record_error(p.status, PA_ERR_BAD_BLOCK);
        id = 0;
      }
      const int s = (issued + lane) % kRawPages;
      mbar_arrive_expect_tx(raw_bar + 8 * s, kBlock);
      bulk_load(raw0 + s * kBlock,
                head + static_cast<uint64_t>(static_cast<uint32_t>(id)) * p.page_bytes, kBlock,
                raw_bar + 8 * s);
    }
    if (n == 2 && (issued & 31) == 31) {
      ids = ids_next;
      ids_next = ids_of(((issued + 1) >> 5) + 1);
    }
    issued += max(0, n);
  };
  issue(2);
  if constexpr (kRawPages > 2) issue(1);

  bool ok = true;
  int t = c;
  for (int i = 0; t < part.nt; t += step, i += 2) {
    const int s0 = i % kRawPages, s1 = (i + 1) % kRawPages;
    ok = warp_wait2(raw_bar + 8 * s0, (i / kRawPages) & 1, raw_bar + 8 * s1,
                    ((i + 1) / kRawPages) & 1, abort_flag);
    if (!ok) break;
    const uint32_t raw[2] = {raw0 + s0 * kBlock, raw0 + s1 * kBlock};
    // ---- scales and zeros of row `lane` of the warp's 32
    float2 k, v;
    {
      const uint32_t blk = lane < kPageSize ? raw[0] : raw[1];
      k = unpack2<BF16>(lds32(blk + kv4::meta_offset(D, 0, 0) + 4 * (lane % kPageSize)));
      v = unpack2<BF16>(lds32(blk + kv4::meta_offset(D, 1, 0) + 4 * (lane % kPageSize)));
    }
    // the codes into registers, the next pages into their slots
    uint4 codes[2 * kIters], v_codes[2 * kIters];
#pragma unroll
    for (int i = 0; i < 2 * kIters; ++i) {
      const uint32_t at = raw[i / kIters] +
                          ((i % kIters) * (32 / kPieces) + row_l) * kv4::row_bytes(D) + 16 * piece;
      codes[i] = lds128(at);
      v_codes[i] = lds128(at + kPageSize * kv4::row_bytes(D));
    }
    if ((part.t0 + t) * kKeys + 32 * w + lane >= tokens) {
      k = v = make_float2(0.f, 0.f);
    } else if (!(fabsf(k.x) <= FLT_MAX && fabsf(k.y) <= FLT_MAX && fabsf(v.x) <= FLT_MAX &&
                 fabsf(v.y) <= FLT_MAX)) {
      k = make_float2(0.f, __int_as_float(0x7fc00000));
      v = make_float2(0.f, 0.f);
    }
    // the row's largest magnitude (a NaN does not count) and the 32 rows'; no float is
    // negative here, so their bits are in their order
    const float k_own = EXACT ? 0.f : fmaxf(fmaf(8.f, fabsf(k.x), fabsf(k.y)), 0.f);
    const float v_own = fmaxf(EXACT ? fabsf(v.x) : fmaf(8.f, fabsf(v.x), fabsf(v.y)), 0.f);
    auto top_of = [](float own) {
      return above(__uint_as_float(__reduce_max_sync(kFull, __float_as_uint(own))));
    };
    const float k_ref = EXACT ? 1.f : top_of(k_own), v_ref = top_of(v_own);
    // How far the reference is lowered for rows below 2^-5 of it (other than zero).
    int k_span = 0, v_span = 0;
    auto small = [](float own, float ref) { return own > 0.f && own * 32.f < ref; };
    if (!EXACT && __builtin_expect(
                      __any_sync(kFull, small(k_own, k_ref) || small(v_own, v_ref)), 0)) {
      auto span_of = [](float own, float ref) {
        const uint32_t least =
            __reduce_min_sync(kFull, own > 0.f ? __float_as_uint(own) : 0x7f800000u);
        const int span = exponent(ref) - exponent(__uint_as_float(least));
        return span > 5 ? span : 0;
      };
      k_span = min(15, span_of(k_own, k_ref));
      v_span = min(11, span_of(v_own, v_ref));
    }

    const int s = t % kStages;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const int free = which ? kBarVFree : kBarKFree;
      if (t >= kStages)  // with one reader, its barrier twice
        ok = warp_wait2(bar(free + 2 * tl.first(s) + s), (t / kStages - 1) & 1,
                        bar(free + 2 * tl.last(s) + s), (t / kStages - 1) & 1, abort_flag);
      if (!ok) break;
      const int span = which ? v_span : k_span;
      const int ref = exponent(which ? v_ref : k_ref);
      int row_ref = ref;
      if (__builtin_expect(span, 0)) row_ref = exponent(above(which ? v_own : k_own));
      const float inv = exp2i(-row_ref);
      const float2 own = which ? v : k;
      // over 2^7 ref: |scale| 2^24 is at most 2^14
      const uint32_t scales = pack2<false>(own.x * inv * 0x1p17f, own.x * inv * 0x1p13f);
      // K's zero is not in its codes' operand but in the columns behind it
      const uint32_t zeros =
          pack2<false>(fmaf(-8.f, own.x, which ? own.y : 0.f) * inv * 0x1p-7f, 0.f);
      if (!EXACT && !which) {
        const float z = k.y * exp2i(-ref) * exp2i(span);
        st_shared_v4(sb + L::kKX + s * L::kExtra + (32 * w + lane) * 16,
                     pack2<false>(z, z * 0x1p-11f), 0, 0, 0);
      }
      if (which) {
        // V's stage is free once the softmax has read these for the tile before in it
        float *refs = reinterpret_cast<float *>(smem + L::kRef) + 8 * s;
        if (lane == 0) {
          refs[w] = k_ref * exp2i(-k_span);
          refs[4 + w] = v_ref * exp2i(-v_span);
        }
        if constexpr (EXACT) {
          const int row = 32 * w + lane;
          float *m = reinterpret_cast<float *>(smem + L::kMeta) + s * (kKeys / 2) * 8 +
                     (row >> 1) * 8 + (row & 1);
          m[0] = k.x * (0.5f * p.qscale);
          m[2] = fmaf(-0.5f, k.x, k.y) * p.qscale;
          m[4] = v.x * inv;
          m[6] = fmaf(-0.5f, v.x, v.y);
        }
      }
      const uint32_t dst = sb + (which ? L::kV : L::kK) + s * L::kTile;
#pragma unroll
      for (int i = 0; i < 2 * kIters; ++i) {
        // row of the warp's 32
        const int row = (i / kIters) * kPageSize + (i % kIters) * (32 / kPieces) + row_l;
        __half2 s24 = __float2half2_rn(0.f), s20 = s24, z = s24;
        if constexpr (!EXACT) {
          const uint32_t sc = __shfl_sync(kFull, scales, row);
          const uint32_t zr = __shfl_sync(kFull, zeros, row);
          const uint32_t a = __byte_perm(sc, sc, 0x1010), b = __byte_perm(sc, sc, 0x3232);
          const uint32_t c = __byte_perm(zr, zr, 0x1010);
          s24 = *reinterpret_cast<const __half2 *>(&a);
          s20 = *reinterpret_cast<const __half2 *>(&b);
          z = *reinterpret_cast<const __half2 *>(&c);
        }
        const uint32_t wd[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
        // 16-byte chunks 4 piece .. 4 piece + 3 of the row, swizzled
        const int at = 32 * w + row, c0 = 4 * piece;
        const uint32_t to = dst + (c0 >> 3) * L::kColBlk + swz128(at, c0);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 o = operand<EXACT>(wd[u], s24, s20, z);
          st_shared_v4(to ^ (u << 4), o.x, o.y, o.z, o.w);
        }
        codes[i] = v_codes[i];  // for the second round
      }
      if (!EXACT && __builtin_expect(span, 0)) {
        // what this thread wrote, from its rows' own references to the lowered one
        const float move = exp2i(max(-24, row_ref - ref + span));
        const uint32_t moves = pack2<false>(move, move);
#pragma unroll 1
        for (int i = 0; i < 8 * kIters; ++i) {
          const int k = i >> 2;
          const int row = (k / kIters) * kPageSize + (k % kIters) * (32 / kPieces) + row_l;
          const uint32_t by = __shfl_sync(kFull, moves, row);
          const uint32_t at =
              (dst + (piece >> 1) * L::kColBlk + swz128(32 * w + row, 4 * piece)) ^ ((i & 3) << 4);
          const uint4 o = lds128(at);
          auto times = [&](uint32_t x) {
            const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&x),
                                      *reinterpret_cast<const __half2 *>(&by));
            return *reinterpret_cast<const uint32_t *>(&r);
          };
          st_shared_v4(at, times(o.x), times(o.y), times(o.z), times(o.w));
        }
      }
      fence_proxy_async_smem();  // generic stores -> read by the tensor cores
      __syncwarp();
      if (lane == 0) mbar_arrive(bar((which ? kBarV : kBarK) + s));
      if (!which) issue(2);  // the pages' codes are in registers, and the fence covers it
    }
    if (!ok) break;
  }
  if (!ok) {
    if (lane == 0) raise_abort(p.status, abort_flag);
    for (int i = max(0, issued - kRawPages); i < issued; ++i)  // copies in flight still land
      mbar_wait(raw_bar + 8 * (i % kRawPages), (i / kRawPages) & 1);
    return;
  }
  // every MMA that reads a stage has committed before the part ends
  for (int i = max(c, t - kStages); i < t && ok; i += step)
    for (int x = tl.first(i % kStages); x <= tl.last(i % kStages) && ok; ++x)
      ok = warp_wait2(bar(kBarKFree + 2 * x + i % kStages), (i / kStages) & 1,
                      bar(kBarVFree + 2 * x + i % kStages), (i / kStages) & 1, abort_flag);
  if (!ok && lane == 0) raise_abort(p.status, abort_flag);
}

// MMA warp x (lane 0): S_x(0), then per key tile t: P_x(t) V_t in two key halves,
// S_x(t + 1), which overwrites P_x in TMEM: MMAs of one thread run in order.  (Split key
// tiles: t = x, x + 2, ..)
template <int D, bool EXACT, bool FEW>
__device__ __forceinline__ void mma_tiles(int x, bool split, int nt, uint32_t sb, uint32_t bars,
                                          uint32_t tmem, int *status, volatile int *abort_flag,
                                          int lane) {
  using L = PrefillSmem<D, EXACT, FEW>;
  constexpr uint32_t kIdS = tc::idesc_f16(false, kRows, kKeys, false, false);
  constexpr uint32_t kIdO = tc::idesc_f16(false, kRows, D, false, true);
  auto bar = [&](int i) { return bars + 8 * i; };
  const uint64_t dq = tc::smem_desc_sw128(sb + L::kQ + (FEW ? 0 : x) * L::kTile, 16, 1024);
  const uint64_t dk0 = tc::smem_desc_sw128(sb + L::kK, 16, 1024);
  const uint64_t dv0 = tc::smem_desc_sw128(sb + L::kV, L::kColBlk, 1024);
  // the columns behind: 8 of the tile, 8 of zeros (kZeros is behind the tiles)
  auto extra = [&](int at) { return tc::smem_desc_plain(sb + at, L::kZeros - at, 128); };
  const uint64_t dqx = extra(L::kQX + (FEW ? 0 : x) * L::kExtra);
  const uint64_t dkx0 = extra(L::kKX), dkx1 = extra(L::kKX + L::kExtra);
  const uint32_t tS = tmem + x * kKeys, tO = tmem + 2 * kKeys + x * D;
  const int step = split ? 2 : 1, t_first = split ? x : 0;
  auto s_mma = [&](int t) {
    if (lane == 0) {
      const uint64_t dk = dk0 + static_cast<uint64_t>(((t % kStages) * L::kTile) >> 4);
      if constexpr (!EXACT) tc::mma_f16(tS, dqx, t % kStages ? dkx1 : dkx0, kIdS, 0);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = static_cast<uint64_t>(((kk >> 2) * L::kColBlk + (kk & 3) * 32) >> 4);
        tc::mma_f16(tS, dq + off, dk + off, kIdS, !EXACT || kk > 0);
      }
      tc::commit(bar(kBarS + x));
      tc::commit(bar(kBarKFree + 2 * x + t % kStages));
    }
    __syncwarp();
  };
  auto pv_mma = [&](int t, int h) {
    if (lane == 0) {
      const uint64_t dv = dv0 + static_cast<uint64_t>(((t % kStages) * L::kTile) >> 4);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        tc::mma_f16_tmem_a(tO, tS + 32 * h + 8 * kk,
                           dv + static_cast<uint64_t>(((4 * h + kk) * 2048) >> 4), kIdO,
                           (t > t_first || h > 0 || kk > 0) ? 1u : 0u);
      if (h == 1) {
        tc::commit(bar(kBarVFree + 2 * x + t % kStages));
        if (t + step >= nt) tc::commit(bar(kBarO + x));
      }
    }
    __syncwarp();
  };
  bool ok = warp_wait(bar(kBarK + t_first), 0, abort_flag);
  if (ok) {
    tc::fence_after_sync();
    s_mma(t_first);
  }
  for (int t = t_first, j = 0; t < nt && ok; t += step, ++j) {  // the j-th tile of x
    for (int h = 0; h < 2 && ok; ++h) {
      ok = h ? warp_wait(bar(kBarP + 2 * x + 1), j & 1, abort_flag)
             : warp_wait2(bar(kBarV + t % kStages), (t / kStages) & 1, bar(kBarP + 2 * x), j & 1,
                          abort_flag);
      if (!ok) break;
      tc::fence_after_sync();
      pv_mma(t, h);
    }
    const int tn = t + step;
    if (ok && tn < nt &&
        (ok = warp_wait(bar(kBarK + tn % kStages), (tn / kStages) & 1, abort_flag))) {
      tc::fence_after_sync();
      s_mma(tn);
    }
  }
  if (!ok) {
    if (lane == 0) {
      raise_abort(status, abort_flag);
      tc::commit(bar(kBarDrain + x));  // arrives once every MMA issued so far is done
    }
    __syncwarp();
    mbar_wait(bar(kBarDrain + x), 0);
  }
}

__device__ __forceinline__ void row_tiles_sync() {  // both softmax warpgroups
  asm volatile("bar.sync 4, 256;" ::: "memory");
}

// Softmax warpgroup x: lane l of warp w owns row 32 (w mod 4) + l of row tile x.
template <int D, bool BF16, bool EXACT, bool FEW>
__device__ __forceinline__ void softmax_tiles(const PrefillParams &p,
                                              const volatile TilePart &part, int x,
                                              const Tiling &tl, uint32_t sb, uint32_t bars,
                                              uint32_t tmem, uint8_t *smem,
                                              volatile int *abort_flag, int warp, int lane) {
  using L = PrefillSmem<D, EXACT, FEW>;
  auto bar = [&](int i) { return bars + 8 * i; };
  const int r = ((warp & 3) << 5) + lane;
  // last key that the row sees, and that every row of the tile sees
  const int row0 = part.row0 + (tl.split ? 0 : x * kRows);
  const int lim = part.ctx + min(row0 + r, p.n_rows - 1) / p.group;
  const int lim_all = part.ctx + row0 / p.group;
  const int step = tl.split ? 2 : 1, t_first = tl.split ? x : 0;
  const int nt = part.nt;
  int key0 = (part.t0 + t_first) * kKeys;
  const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t tS = tmem + x * kKeys + lane_base;
  const uint32_t tO = tmem + 2 * kKeys + x * D + lane_base;

  const int xq = FEW ? 0 : x;  // whose Q
  float qsum = 0.f, row_f = 0.f;
  if constexpr (EXACT) {
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      const uint4 v = lds128(sb + L::kQ + xq * L::kTile + (c >> 3) * L::kColBlk + swz128(r, c));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2<false>(w[k]);
        qsum += f.x + f.y;
      }
    }
  } else {
    row_f = reinterpret_cast<const float *>(smem + L::kMeta)[xq * kRows + r];
  }
  const float2 q2 = make_float2(qsum, qsum);

  float m = kNoKey, v_ref = 0.f;
  float2 l2 = make_float2(0.f, 0.f), z2 = make_float2(0.f, 0.f);
  bool bad = false;
  for (int t = t_first, j = 0; t < nt; t += step, ++j, key0 += step * kKeys) {
    // the other row tile's turn first
    const int to = t - 1 + x;
    if (tl.n_active == 2 && !tl.split && to >= 0)
      bad = !warp_wait(bar(kBarP + 2 * (x ^ 1)), to & 1, abort_flag);
    if (bad || !warp_wait2(bar(kBarV + t % kStages), (t / kStages) & 1, bar(kBarS + x), j & 1,
                           abort_flag)) {
      bad = true;
      break;
    }
    tc::fence_after_sync();
    const uint32_t meta = sb + L::kMeta + (t % kStages) * (kKeys / 2) * 32;
    const float4 k_ref = *reinterpret_cast<const float4 *>(smem + L::kRef + 32 * (t % kStages));
    const float4 vr = *reinterpret_cast<const float4 *>(smem + L::kRef + 32 * (t % kStages) + 16);
    // scores = f[ch] S, of 32 keys each; P = 2^(score - m) v_ref[ch] / the largest so far
    const float kr[4] = {k_ref.x, k_ref.y, k_ref.z, k_ref.w};
    float f[4];
#pragma unroll
    for (int ch = 0; ch < 4; ++ch)  // never 0: a masked -inf stays -inf
      f[ch] = EXACT ? 1.f : fmaxf(row_f * kr[ch] * 128.f, FLT_MIN);
    const float v_top = fmaxf(fmaxf(fmaxf(vr.x, vr.y), fmaxf(vr.z, vr.w)), v_ref);
    const float grown =
        v_ref > 0.f ? exp2i(max(-126, exponent(v_ref) - exponent(v_top))) : 0.f;
    v_ref = v_top;

    // The scores of kHold keys at a time, the last ones first; the first ones stay, the
    // others are read again.  (Exact: with a whole row of them and the scales on their
    // way the registers do not suffice.)
    constexpr int kHold = EXACT || FEW ? 64 : kKeys;
    uint32_t s[kHold];
    auto scores = [&](int h, bool raw) {
#pragma unroll
      for (int cb = 0; cb < kHold / 32; ++cb)
        tc::ld32(tS + h * kHold + cb * 32, *reinterpret_cast<uint32_t(*)[32]>(s + cb * 32));
      tc::wait_ld();
      if (EXACT && raw) {  // scores from the raw sums, two keys an instruction
#pragma unroll
        for (int c = 0; c < kHold; c += 2) {
          const uint4 u = lds128(meta + (h * kHold + c) * 16);
          const float2 e = __ffma2_rn(
              make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
              make_float2(__uint_as_float(u.x), __uint_as_float(u.y)),
              __fmul2_rn(make_float2(__uint_as_float(u.z), __uint_as_float(u.w)), q2));
          s[c] = __float_as_uint(e.x);
          s[c + 1] = __float_as_uint(e.y);
        }
        if (h > 0) {
#pragma unroll
          for (int cb = 0; cb < kHold / 32; ++cb)
            tc::st32(tS + h * kHold + cb * 32, *reinterpret_cast<uint32_t(*)[32]>(s + cb * 32));
          tc::wait_st();
        }
      }
      if (key0 + (h + 1) * kHold - 1 > lim_all) {
        const int last = lim - key0 - h * kHold;  // keys past this one are masked for the row
#pragma unroll
        for (int c = 0; c < kHold; ++c)
          if (c > last) s[c] = __float_as_uint(-INFINITY);
      }
    };
    float cand = -INFINITY;
#pragma unroll
    for (int h = kKeys / kHold - 1; h >= 0; --h) {
      scores(h, true);
#pragma unroll
      for (int ch = 0; ch < kHold / 32; ++ch) {
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int c = 32 * ch; c < 32 * ch + 32; c += 4) {
          t0 = max3(t0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
          t1 = max3(t1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
        }
        cand = fmaxf(cand, fmaxf(t0, t1) * f[h * (kHold / 32) + ch]);
      }
    }
    float corr = 1.f;
    if (cand - m > kSlack) {
      corr = ex2(m - cand);  // 0 while m was no key's
      m = cand;
      l2 = __fmul2_rn(l2, make_float2(corr, corr));
      z2 = __fmul2_rn(z2, make_float2(corr, corr));
    }
    const bool need = corr != 1.f || grown != 1.f;
    corr *= grown;

    // ---- weights over the S columns, two keys a column; each 64-key half is handed
    // to the MMA warp as soon as it is written
    auto chunk = [&](int ch) {
      uint32_t ph[16];
      // v_ref[ch] over the largest, 2^by: into the exponent, out of the sum.  Below
      // 2^-60 these values no longer count, but their weights still do.
      const int by = max(-60, exponent(ch == 0 ? vr.x : ch == 1 ? vr.y : ch == 2 ? vr.z : vr.w) -
                                  exponent(v_ref));
      const float nb = static_cast<float>(by) + kLift - m, back = exp2i(-by);
      const float2 nm = make_float2(nb, nb), f2 = make_float2(f[ch], f[ch]);
      float2 sum = make_float2(0.f, 0.f), zs = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int c = (32 * ch) % kHold + 2 * k;
        const float2 sc = make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        const float2 e = EXACT ? __fadd2_rn(sc, nm) : __ffma2_rn(sc, f2, nm);
        const float2 pr = make_float2(ex2(e.x), ex2(e.y));
        sum = __fadd2_rn(sum, pr);
        if constexpr (EXACT) {
          const uint4 u = lds128(meta + (32 * ch + 2 * k) * 16 + 16);
          zs = __ffma2_rn(pr, make_float2(__uint_as_float(u.z), __uint_as_float(u.w)), zs);
          const float2 w =
              __fmul2_rn(pr, make_float2(__uint_as_float(u.x), __uint_as_float(u.y)));
          ph[k] = pack2<false>(w.x, w.y);
        } else {
          ph[k] = pack2<false>(pr.x, pr.y);
        }
      }
      const float2 undo = make_float2(back, back);
      l2 = __ffma2_rn(sum, undo, l2);
      if constexpr (EXACT) z2 = __ffma2_rn(zs, undo, z2);
      tc::st16(tS + 16 * ch, ph);
      if (ch == 1 && j > 0 && __any_sync(kFull, need)) {
        // P_x V of the tile before has completed: S_x was issued behind it
#pragma unroll
        for (int cb = 0; cb < D / 32; ++cb) {
          uint32_t o[32];
          tc::ld32(tO + cb * 32, o);
          tc::wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * corr);
          tc::st32(tO + cb * 32, o);
        }
      }
      if (ch & 1) {
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarP + 2 * x + (ch >> 1)));
        if (FEW && lane == 0) mbar_arrive(bar(kBarP + 2 * x + (ch >> 1)));  // two warps' worth
      }
    };
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
      if (ch > 0 && (32 * ch) % kHold == 0) scores(32 * ch / kHold, false);
      chunk(ch);
    }
  }
  if (!bad) bad = !warp_wait(bar(kBarO + x), 0, abort_flag);
  if (bad && lane == 0) raise_abort(p.status, abort_flag);
  // out = o_a O + o_b O_B + z, over l, all of lifted weights (V's operands are twice the
  // centred codes, or values over 2^7 v_ref)
  constexpr float kDown = 1.f / (1 << static_cast<int>(kLift));
  float l = (l2.x + l2.y) * kDown, z = (z2.x + z2.y) * kDown;
  float o_a = v_ref * (EXACT ? 0.5f * kDown : 128.f * kDown), o_b = 0.f;
  if (tl.split) {
    // B leaves its (m, l, z, reference) in Q_B, whose products are done; both
    // warpgroups always meet here, failed or not
    float4 *other = reinterpret_cast<float4 *>(smem + L::kQ + L::kTile) + r;
    if (x == 1 && !bad) *other = make_float4(m, l, z, o_a);
    tc::fence_before_sync();
    row_tiles_sync();
    bad = __any_sync(kFull, *abort_flag);
    if (x == 1) return;
    const float4 b = *other;
    const float mn = fmaxf(m, b.x), ca = ex2(m - mn), cb = ex2(b.x - mn);
    m = mn;
    l = ca * l + cb * b.y;
    z = ca * z + cb * b.z;
    o_a *= ca;
    o_b = cb * b.w;
  }
  if (bad) return;
  tc::fence_after_sync();

  // ---- the row's result in the natural order of dimensions, or its state
  const int row = row0 + r;
  const bool real = row < p.n_rows, whole = part.first == part.last;
  const float inv = !whole ? 1.f : (l == 0.f ? 0.f : 1.f / l);
  const int slot = static_cast<int>(blockIdx.x) > part.first ? 0 : part.slot;
  float *state = p.ws + ((static_cast<size_t>(blockIdx.x) * 2 + slot) * kItemRows +
                         (row - part.row0)) * (D + 4);
  uint16_t *dst = p.out + row_at(p, part.b, part.g, row) * D;
#pragma unroll 1
  for (int cb = 0; cb < D / 32; ++cb) {
    uint32_t o[32];
    tc::ld32(tO + cb * 32, o);
    tc::wait_ld();
    float f[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) f[k] = fmaf(__uint_as_float(o[k]), o_a, z);
    if (tl.split) {
      tc::ld32(tO + D + cb * 32, o);  // O_B is D columns to the right
      tc::wait_ld();
#pragma unroll
      for (int k = 0; k < 32; ++k) f[k] = fmaf(__uint_as_float(o[k]), o_b, f[k]);
    }
    if (!real) continue;
    constexpr int kAt[8] = {0, 2, 4, 6, 1, 3, 5, 7};  // where dimension k of eight is
    auto at = [&](int k) { return f[(k & ~7) + kAt[k & 7]] * inv; };
    if (whole) {
#pragma unroll
      for (int k = 0; k < 32; k += 8)
        *reinterpret_cast<uint4 *>(dst + cb * 32 + k) =
            make_uint4(pack2<BF16>(at(k), at(k + 1)), pack2<BF16>(at(k + 2), at(k + 3)),
                       pack2<BF16>(at(k + 4), at(k + 5)), pack2<BF16>(at(k + 6), at(k + 7)));
    } else {
#pragma unroll
      for (int k = 0; k < 32; k += 4)
        *reinterpret_cast<float4 *>(state + cb * 32 + k) =
            make_float4(at(k), at(k + 1), at(k + 2), at(k + 3));
    }
  }
  if (real && !whole) *reinterpret_cast<float2 *>(state + D) = make_float2(m, l);
}

// Row tile x of Q in the operand's order of dimensions, zeros past the rows (FEW: in
// the warps that have some; the others' S is not looked at), by 128 threads; not exact:
// as fp16 over a power of two a row, whose product with the score factor goes to kMeta.
// A thread copies chunks to where they belong and then turns its own in place.  The loops
// are hardly unrolled: this runs once a part, and straight-line code waits for its own
// instructions (measured 10 us a part with all 16 chunks unrolled, 4 so).
template <int D, bool BF16, bool EXACT, bool FEW>
__device__ __forceinline__ void load_q(const PrefillParams &p, const volatile TilePart &part,
                                       bool split, int x, uint32_t sb, uint8_t *smem, int th) {
  using L = PrefillSmem<D, EXACT, FEW>;
  constexpr int kChunks = D / 8;  // 16-byte chunks a row
  constexpr int kStep = 128 / kChunks;
  const int c = th % kChunks, row0 = part.row0 + (split ? 0 : x * kRows), b = part.b, g = part.g;
  const uint32_t dst = sb + L::kQ + x * L::kTile + (c >> 3) * L::kColBlk;
  const int rows = FEW ? kRows / 4 * ((p.n_rows + kRows / 4 - 1) / (kRows / 4)) : kRows;
#pragma unroll 1
  for (int r = th / kChunks; r < rows; r += kStep) {
    const uint32_t to = dst + swz128(r, c);
    if (row0 + r < p.n_rows)
      cp_async16(to, p.q + row_at(p, b, g, row0 + r) * D + c * 8);
    else
      st_shared_v4(to, 0, 0, 0, 0);
  }
  cp_async_wait();
#pragma unroll 1
  for (int r0 = th / kChunks; r0 < rows; r0 += 4 * kStep) {
    float sums[4] = {0.f, 0.f, 0.f, 0.f};  // of this thread's elements of four rows
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + i * kStep;
      if (r >= rows) break;
      const uint32_t at = dst + swz128(r, c);
      const uint4 v = lds128(at);
      uint32_t w[4] = {v.x ^ p.qsign, v.y ^ p.qsign, v.z ^ p.qsign, v.w ^ p.qsign};
      if constexpr (!EXACT) {
        float2 f[4];
        float top = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          f[u] = unpack2<BF16>(w[u]);
          top = fmaxf(top, fmaxf(fabsf(f[u].x), fabsf(f[u].y)));
        }
#pragma unroll
        for (int o = 1; o < kChunks; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        // 2^ex brings the row's largest magnitude into [2^14, 2^15), or near 1 where that
        // is near the smallest of all
        const int ex = min(120, 14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127));
        const float up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          w[u] = pack2<false>(f[u].x * up, f[u].y * up);
          const float2 h = unpack2<false>(w[u]);  // as the operand holds it
          sums[i] += h.x + h.y;
        }
        if (c == 0)
          reinterpret_cast<float *>(smem + L::kMeta)[x * kRows + r] =
              p.qscale * __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
      }
      st_shared_v4(at, __byte_perm(w[0], w[2], 0x5410), __byte_perm(w[0], w[2], 0x7632),
                   __byte_perm(w[1], w[3], 0x5410), __byte_perm(w[1], w[3], 0x7632));
    }
    if constexpr (!EXACT) {
      // the rows' sums: a quarter of their threads ends up with each of the four
      const bool upper = c & (kChunks / 2), odd = c & (kChunks / 4);
      float a = upper ? sums[2] : sums[0], b = upper ? sums[3] : sums[1];
      a += __shfl_xor_sync(kFull, upper ? sums[0] : sums[2], kChunks / 2);
      b += __shfl_xor_sync(kFull, upper ? sums[1] : sums[3], kChunks / 2);
      float sum = (odd ? b : a) + __shfl_xor_sync(kFull, odd ? a : b, kChunks / 4);
#pragma unroll
      for (int o = kChunks / 8; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      const int r = r0 + (2 * upper + odd) * kStep;
      if (c % (kChunks / 4) == 0 && r < rows) {  // over 2^7, in two terms
        sum *= 0x1p-7f;
        const float head = unpack2<false>(pack2<false>(sum, 0.f)).x;
        st_shared_v4(sb + L::kQX + x * L::kExtra + r * 16,
                     pack2<false>(sum, (sum - head) * 0x1p11f), 0, 0, 0);
      }
    }
  }
  fence_proxy_async_smem();  // generic stores -> read by the tensor cores
}

// All threads of the CTA, at named barrier N.
template <int N>
__device__ __forceinline__ void cta_sync() {
  asm volatile("bar.sync %0, %1;" ::"n"(N), "n"(kThreads) : "memory");
}

// Registers a thread after the split (not FEW): the softmax holds a whole row of scores.
constexpr int kRegsLaunch = 128, kRegsMma = 64, kRegsConvert = 96, kRegsSoftmax = 176;
static_assert(128 * (kRegsMma + kRegsConvert) + 256 * kRegsSoftmax <= kThreads * kRegsLaunch,
              "register split");
template <int N, bool UP>
__device__ __forceinline__ void set_registers() {
  if constexpr (UP)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// FEW: calls with at most 64 rows a kv head.  Both row tiles are the same rows (one Q),
// and warps 2 and 3 of the softmax warpgroups, whose rows are none, turn the odd key
// tiles' codes, through rings in Q_B's place.  All keep the registers of the launch, so
// that the two groups of converters are one copy of the code (two in the instruction
// caches, each at its own registers: 4 x 4 queries over 32k keys 97 us, so 86).
template <int D, bool BF16, bool FEW>
__global__ void __launch_bounds__(kThreads, 1) kv4_prefill_kernel(const PrefillParams p) {
  constexpr bool EXACT = !BF16;
  using L = PrefillSmem<D, EXACT, FEW>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kSlot + 4);
  volatile int *any = reinterpret_cast<volatile int *>(smem + L::kSlot + 8);
  TilePart *parts = reinterpret_cast<TilePart *>(smem + L::kPart);
  TileWalk *walk = reinterpret_cast<TileWalk *>(smem + L::kWalk);
  auto bars_of = [&](int turn) { return sb + L::kBars + (turn & 1) * (8 * kNumBars); };
  auto init_bars = [&](int turn) {
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bars_of(turn) + 8 * i, i < kBarKFree || (i >= kBarP && i < kBarP + 4) ? 4 : 1);
    fence_mbar_init();
  };

  if (!EXACT && tid < kRows) {
    st_shared_v4(sb + L::kZeros + tid * 16, 0, 0, 0, 0);
    fence_proxy_async_smem();  // read by the tensor cores
  }
  griddep_wait();  // inputs may come from the previous kernel in the stream
  griddep_release();
  if (warp == 0) {
    bool have = TileWalk::start(p, lane, walk);
    if (lane == 0) {
      if (have) walk->next(p, parts[0]);
      have = have && parts[0].nt > 0;
      if (!have) p.cut[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
      *any = have;
      *abort_flag = 0;
      init_bars(0);
    }
  }
  __syncthreads();
  if (!*any) return;
  if (warp == 0) {
    // S_A: columns 0-127, S_B: 128-255, O_A: 256 .. 256+D-1, O_B: 256+D .. 256+2D-1
    tc::alloc(sb + L::kSlot, 512);
    tc::relinquish();
  }

  // All walk the parts in step: barrier 1 when Q is in place, barrier 2 at the part's
  // end.  In between warp 2 plans the next one and readies its barriers.
  auto begin = [&] {
    tc::fence_before_sync();
    cta_sync<1>();
    tc::fence_after_sync();
    return *reinterpret_cast<volatile uint32_t *>(smem + L::kSlot);
  };
  auto finish = [&] {
    tc::fence_before_sync();
    cta_sync<2>();
    tc::fence_after_sync();
  };
  const int x = (warp - kSoftmaxWarp0) >> 2;  // of a softmax warpgroup
  auto own_q = [&](const volatile TilePart &part, const Tiling &tl) {
    if (!FEW || x == 0) load_q<D, BF16, EXACT, FEW>(p, part, tl.split, x, sb, smem, tid & 127);
    // what this thread left in Q_B, before copies into it
    if (FEW) fence_proxy_async_smem();
  };
  if (warp < kConvertWarp0) {
    if constexpr (!FEW) set_registers<kRegsMma, false>();
    for (int turn = 0;; ++turn) {
      const TilePart part = parts[turn & 1];
      const Tiling tl(part.row0, part.nt, p.n_rows);
      const uint32_t tmem = begin();
      if (warp < tl.n_active)
        mma_tiles<D, EXACT, FEW>(warp, tl.split, part.nt, sb, bars_of(turn), tmem, p.status,
                                 abort_flag, lane);
      if (warp == 2 && lane == 0 && part.more) {
        if (turn > 0)
          for (int i = 0; i < kNumBars; ++i)
            asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bars_of(turn + 1) + 8 * i)
                         : "memory");
        init_bars(turn + 1);
        walk->next(p, parts[(turn + 1) & 1]);
      }
      finish();
      if (!part.more || *abort_flag) {
        if (tid == 0) {
          // the run's last part may start an item that later CTAs hold more of
          const int c = blockIdx.x;
          const bool cut = part.last > c && part.first == c;
          p.cut[2 * c] = make_int4(cut ? part.last - c + 1 : 0, part.slot, part.row0, 0);
          p.cut[2 * c + 1] = make_int4(part.b, part.g, 0, 0);
        }
        break;
      }
    }
  } else if (warp < kSoftmaxWarp0 || (FEW && (warp & 2))) {
    if constexpr (!FEW) set_registers<kRegsConvert, false>();
    const int c = FEW && warp >= kSoftmaxWarp0 ? 1 : 0;
    for (int turn = 0;; ++turn) {
      const TilePart part = parts[turn & 1];
      const Tiling tl(part.row0, part.nt, p.n_rows);
      if (c == 1) own_q(part, tl);
      begin();
      if (c == 0 || tl.split)
        convert_tiles<D, BF16, EXACT, FEW>(c, FEW && tl.split ? 2 : 1,
                                      c == 0 ? warp - kConvertWarp0 : 2 * x + (warp & 1), p, part,
                                      sb, bars_of(turn), smem, tl, abort_flag, lane);
      if (c == 1 && tl.split) row_tiles_sync();
      finish();
      if (!part.more || *abort_flag) break;
    }
  } else {
    if constexpr (!FEW) set_registers<kRegsSoftmax, true>();
    for (int turn = 0;; ++turn) {
      const volatile TilePart &part = parts[turn & 1];
      const Tiling tl(part.row0, part.nt, p.n_rows);
      own_q(part, tl);
      const uint32_t tmem = begin();
      if (x < tl.n_active)
        softmax_tiles<D, BF16, EXACT, FEW>(p, part, x, tl, sb, bars_of(turn), tmem, smem,
                                           abort_flag, warp, lane);
      const bool more = part.more;
      finish();
      if (!more || *abort_flag) break;
    }
  }
  __syncthreads();
  if (warp == 0) tc::dealloc(*reinterpret_cast<volatile uint32_t *>(smem + L::kSlot), 512);
}

// ---- items cut between CTAs: block (c, y) folds the states of rows kFoldRows y .. of
// the item that starts in CTA c's run (if any), a thread a (row, 4 dimensions)
constexpr int kFoldRows = 16;
template <int D, bool BF16>
__global__ void __launch_bounds__(kFoldRows * D / 4) kv4_prefill_fold_kernel(
    const PrefillParams p) {
  griddep_release();
  griddep_wait();  // the states
  const int c = blockIdx.x;
  const int4 cut = __ldcg(p.cut + 2 * c);
  const int n = cut.x;
  if (n == 0) return;
  const int4 at = __ldcg(p.cut + 2 * c + 1);
  const int r = blockIdx.y * kFoldRows + threadIdx.x / (D / 4);
  const int d = 4 * (threadIdx.x % (D / 4)), row = cut.z + r;
  if (row >= p.n_rows) return;
  constexpr int kBatch = 4;
  constexpr size_t kState = static_cast<size_t>(kItemRows) * (D + 4);
  float m = kNoKey, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const float *first = p.ws + (static_cast<size_t>(c) * 2 + cut.y) * kState + r * (D + 4);
  const float *rest = p.ws + static_cast<size_t>(c) * 2 * kState + r * (D + 4);
  for (int k0 = 0; k0 < n; k0 += kBatch) {
    float2 ml[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int k = min(k0 + u, n - 1);  // past the last state, it again
      const float *sp = k == 0 ? first : rest + static_cast<size_t>(k) * 2 * kState;
      ml[u] = __ldcg(reinterpret_cast<const float2 *>(sp + D));
      v[u] = __ldcg(reinterpret_cast<const float4 *>(sp + d));
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (k0 + u >= n) break;
      const float mn = fmaxf(m, ml[u].x);
      const float a = ex2(m - mn), f = ex2(ml[u].x - mn);
      acc.x = fmaf(acc.x, a, v[u].x * f);
      acc.y = fmaf(acc.y, a, v[u].y * f);
      acc.z = fmaf(acc.z, a, v[u].z * f);
      acc.w = fmaf(acc.w, a, v[u].w * f);
      l = fmaf(l, a, ml[u].y * f);
      m = mn;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2 *>(p.out + row_at(p, at.x, at.y, row) * D + d) =
      make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
}

size_t states_bytes(int head_dim, int ctas) {
  return static_cast<size_t>(ctas) * 2 * kItemRows * (head_dim + 4) * sizeof(float);
}

template <int D, bool BF16, bool FEW>
int launch_t(const PrefillParams &p, int ctas, cudaStream_t stream) {
  auto kern = kv4_prefill_kernel<D, BF16, FEW>;
  static ContextCache<bool> smem_set;
  constexpr int kSmem = PrefillSmem<D, !BF16, FEW>::kAlloc;
  if (set_smem_limit(kern, kSmem, smem_set) != PA_OK) return PA_ERR_CUDA;
  // the split draws on what the block was launched with; less of it would never come free
  static std::atomic<bool> enough{FEW};
  if (!enough) {
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, kern) != cudaSuccess || attr.numRegs < kRegsLaunch)
      return PA_ERR_CUDA;
    enough = true;
  }
  if (launch_pdl(kern, dim3(ctas), dim3(kThreads), kSmem, stream, p) !=
          cudaSuccess ||
      launch_pdl(kv4_prefill_fold_kernel<D, BF16>,
                 dim3(ctas, (min(p.n_rows, kItemRows) + kFoldRows - 1) / kFoldRows),
                 dim3(kFoldRows * D / 4), 0, stream, p) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}

template <int D, bool BF16>
int launch_d(const PrefillParams &p, int ctas, cudaStream_t stream) {
  return p.n_rows <= kRows / 2 ? launch_t<D, BF16, true>(p, ctas, stream)
                               : launch_t<D, BF16, false>(p, ctas, stream);
}

}  // namespace

size_t kv4_tiles_workspace_bytes(int head_dim, int sms) {
  return states_bytes(head_dim, sms) + static_cast<size_t>(sms) * 2 * sizeof(int4);
}

int launch_kv4_tiles(const Kv4AttentionLaunch &a, cudaStream_t stream) {
  const int ctas = sm_count();
  if (ctas <= 0) return PA_ERR_CUDA;
  PrefillParams p;
  p.q = static_cast<const uint16_t *>(a.q);
  p.cache = a.cache;
  p.block_table = a.block_table;
  p.ctx_lens = a.ctx_lens;
  p.out = static_cast<uint16_t *>(a.out);
  p.ws = static_cast<float *>(a.workspace);
  p.cut = reinterpret_cast<int4 *>(static_cast<char *>(a.workspace) +
                                   states_bytes(a.head_dim, ctas));
  p.status = a.status;
  // The maximum is taken over raw sums, so their factor has to be positive: a negative
  // scale flips the sign of Q instead, a zero scale becomes one that makes every weight 1.
  p.qscale = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
  p.qsign = a.scale < 0.f ? 0x80008000u : 0u;
  p.n_new = a.n_new;
  p.n_q_heads = a.n_q_heads;
  p.n_kv_heads = a.n_kv_heads;
  p.group = a.n_q_heads / a.n_kv_heads;
  p.batch = a.batch;
  p.max_blocks = a.max_blocks;
  p.num_pages = a.num_pages;
  p.n_rows = a.n_new * p.group;
  p.n_items = (p.n_rows + kItemRows - 1) / kItemRows;
  // Us for 0, 1, 2, 4 tiles: 4 x 32 queries of 64 / 8 heads over 32k tokens 151, 149, 147,
  // 143, 4 x 512 of 32 / 8 over 8192 within 1%; up to 64 rows, whose tiles are the shorter
  // ones, for 3, 6, 10, 14: 87, 86, 87, 88.
  p.part_tiles = p.n_rows <= kRows / 2 ? 6 : 4;
  p.page_bytes = static_cast<uint32_t>(a.n_kv_heads) * kv4::block_bytes(a.head_dim);
  if (a.head_dim == 128)
    return a.bf16 ? launch_d<128, true>(p, ctas, stream) : launch_d<128, false>(p, ctas, stream);
  return a.bf16 ? launch_d<64, true>(p, ctas, stream) : launch_d<64, false>(p, ctas, stream);
}

}  // namespace pa
