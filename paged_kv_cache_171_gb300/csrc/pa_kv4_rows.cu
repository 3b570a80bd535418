// pa_kv4_rows.cu -- attention over the 4-bit paged cache for few query rows a
// kv head: decode (one query a sequence) and short chunks (speculative verify).
//
// A row is a (query, head) pair of one kv head; o = softmax(q K^T scale) V with
// K = zero_k + scale_k (c - 8) and V alike, c the 4-bit codes.  The codes go
// into the tensor cores as they are (exact in 16 bits) and the scales and
// zeros are applied outside,
//   s_t = scale_k[t] (q . c_t - 8 sum q) + zero_k[t] sum q
//   O   = sum_t (p_t scale_v[t]) (c_t - 8),   z = sum_t p_t zero_v[t]
// so a page costs no dequantisation beyond turning nibbles into 16-bit floats.
//
// Operand form.  mma.sync m16n8k16 with the tokens (then the head dimensions)
// as the 16 rows and 8 query rows as the columns.  That uses every tensor-core
// row for up to 8 query rows, keeps the output state in head_dim / 4 registers
// a thread, and needs no transpose of K or V: a thread loads whole 32-bit words
// of codes, and because the contraction index may be permuted freely (q, or the
// order of tokens, is permuted alike) two nibbles four places apart in one
// word, or the same nibble of two tokens' words, form an operand register.
//   K: x & 0x000f000f as fp16 is the subnormal c 2^-24, x & 0x00f000f0 is
//      c 2^-20: one AND gives two elements.  q is scaled by a power of two a
//      row (its largest magnitude near 2^15, exact in fp16 down to 2^-39 of the
//      row's largest) with the slots of the second kind divided by 16.
//   V: the accumulation over tokens is long, and tensor-core sums round toward
//      zero, so the codes are centred first: (x & 0x000f000f) | 0x64006400 is
//      1024 + c, minus 1032; (x & 0x00f000f0) | 0x64006400 is 1024 + 16 c,
//      times 1/16 minus 72; both exact.  Uncentred, the sum of 8 p would drown
//      a diffuse row's result in rounding.
// The weights p scale_v enter as two fp16 terms (head and remainder, 22 bits).
// Products of a head term and a code have 15 bits, so their sums hardly ever
// round; a remainder added to such a sum always would, toward zero, so the two
// are accumulated apart (4 rows or fewer) or page by page in an accumulator of
// their own that is added to the state with a rounding add (measured on the 32k
// rows at 8 rows a tile: error 9e-6 of the result in one accumulator).
// They are taken relative to a power of two above the largest |scale_v| so far
// and multiplied by 2^7, so that they stay below 2^15 and the second term
// reaches 2^-32 of the largest.  With at most 4 rows (WIDE false) columns 4-7
// repeat columns 0-3 and carry the second terms: one MMA does both.  The
// weights, in the accumulator's layout (token, row), become the second
// product's operand (row, token) by movmatrix.
//
// Work split.  The pages of all (sequence, kv head, row tile) items, laid end to
// end, are cut into equal runs, one a CTA, as many CTAs as fit the GPU at once:
// a ragged batch takes the time of its pages, not of its longest sequence.  A
// CTA's 4 warps take its run's pages in turn, each with its own ring of stages
// filled by bulk copies, and merge their (m, l, O) states when an item ends.  An
// item cut between CTAs leaves one state a CTA, and the last of them to arrive
// merges them in order of position, so results do not depend on timing.
#include "pa_device.cuh"
#include "pa_kv4.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleSlack = 8.0f;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kNoKey = -3.402823466e38f;  // running max of a row before its first key
constexpr int kWarps = 4, kStages = 3, kTile = 8;  // query rows a tile
constexpr int kPair = 2;         // pages a stage holds
constexpr int kCtasPerSm = 4;
constexpr int kMinPages = kWarps * kPair;  // least pages a CTA takes

struct RowsParams {
  const uint16_t *q;
  const uint8_t *cache;
  const int32_t *block_table, *ctx_lens;
  void *out;
  float *ws;     // [CTA][2][kTile][D + 4] partial states
  int *ctr;      // [CTA] arrivals of the item that starts in the CTA's run and leaves it
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
  // The warps' states at the end of a part, over the ring: no copy is in flight then.
  static constexpr int kRowStride = D + 4;  // floats a merged row
  static constexpr int kMergeO = 0;
  static constexpr int kMergeM = kMergeO + kWarps * kTile * kRowStride * 4;
  static constexpr int kMergeL = kMergeM + kWarps * kTile * 4;
  static_assert(kMergeL + kWarps * kTile * 4 <= kRing, "merge area must fit in the ring");
  static constexpr int kBars = kRing;
  static constexpr int kParts = kBars + kWarps * kStages * 8;  // Part[2]
  static constexpr int kWalk = kParts + 2 * 64;                // Walk
  static constexpr int kLast = kWalk + 64;
  static constexpr int kBytes = kLast + 16;
  static_assert(kBlock % 16 == 0 && kBars % 8 == 0 && kParts % 16 == 0, "alignment");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

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

// Physical token of score row r < 8 (row r + 8: 8 more).  The order makes the
// rows that neighbouring lanes read from a stage alternate between its even and
// odd rows, which is what shared memory's 32 banks want of 64-byte rows.
__device__ __forceinline__ int token_of(int r) {
  const int c = r >> 1, a = c >> 1, b = c & 1;
  return (r & 1) ? 4 * a + 3 - b : 4 * a + b;
}

// One warp's ring of stages of two pages.  Chunk i of an item's part is pages
// kWarps kPair i and the one behind it of bt_row (the last may be one page);
// `issued` and `waited` number the chunks over the CTA's whole run, which gives
// the stage and the parity.
template <int D>
struct BlockRing {
  static constexpr int kBlock = kv4::block_bytes(D);
  uint32_t stage0, bar0;
  const uint8_t *cache;    // the kv head's block of page 0
  const int32_t *bt_row;   // the warp's first page of the part
  int n, pages;            // chunks of the warp; pages of the part from bt_row on
  int ids_cur, ids_nxt;
  uint32_t issued, waited;  // chunks over the whole run

  // Lane l holds the id of page l & 1 of chunk 16 w + (l >> 1), w the window.
  __device__ int fetch_id(int w, int lane) const {
    const int pg = kWarps * kPair * (16 * w + (lane >> 1)) + (lane & 1);
    return pg < pages ? __ldg(bt_row + pg) : 0;
  }
  __device__ void start(int lane) {
    ids_cur = fetch_id(0, lane);
    ids_nxt = n > 16 ? fetch_id(1, lane) : 0;
  }
  // Called by the whole warp with i = 0, 1, 2, ... of the part's chunks.
  __device__ void issue(int i, int lane, const RowsParams &p) {
    if ((i & 15) == 0 && i > 0) {
      ids_cur = ids_nxt;
      ids_nxt = fetch_id((i >> 4) + 1, lane);
    }
    int id0 = __shfl_sync(kFull, ids_cur, 2 * (i & 15));
    int id1 = __shfl_sync(kFull, ids_cur, 2 * (i & 15) + 1);
    if (lane == 0) {
      const bool two = kWarps * kPair * i + 1 < pages;
      if (static_cast<unsigned>(id0) >= static_cast<unsigned>(p.num_pages) ||
          static_cast<unsigned>(id1) >= static_cast<unsigned>(p.num_pages)) {
        record_error(p.status, PA_ERR_BAD_BLOCK);
        id0 = id1 = 0;  // read a page that exists; the result is flagged as invalid
      }
      const uint32_t s = issued % kStages, bar = bar0 + 8 * s;
      const uint32_t dst = stage0 + s * (kPair * kBlock);
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(bar, two ? 2 * kBlock : kBlock);
      bulk_load(dst, cache + static_cast<uint64_t>(static_cast<uint32_t>(id0)) * p.page_bytes,
                kBlock, bar);
      if (two)
        bulk_load(dst + kBlock,
                  cache + static_cast<uint64_t>(static_cast<uint32_t>(id1)) * p.page_bytes,
                  kBlock, bar);
    }
    ++issued;
  }
  // Warp-uniform wait for the next chunk; its stage, or 0 when the wait ran out.
  __device__ uint32_t wait(int lane, const RowsParams &p) {
    const uint32_t s = waited % kStages, par = (waited / kStages) & 1;
    ++waited;
    if (__all_sync(kFull, mbar_wait(bar0 + 8 * s, par))) return stage0 + s * (kPair * kBlock);
    if (lane == 0) record_error(p.status, PA_ERR_TIMEOUT);
    for (uint32_t k = waited; k < issued; ++k)  // copies in flight still land
      mbar_wait(bar0 + 8 * (k % kStages), (k / kStages) & 1);
    return 0;
  }
};

// The part of one item that a CTA's run holds.
struct Part {
  int b, g;           // sequence, kv head
  int r0, n_r;        // rows of the kv head
  int pg0, n_pg;      // pages
  int tokens;         // keys of the sequence, the chunk's included
  int first, last;    // CTAs that hold the item
  int slot;           // of the first one's state: 0 when the item starts its run
  int more;           // the run goes on behind this part
};
static_assert(sizeof(Part) <= 64, "room in shared memory");

// The CTA's run [w, w1) of the flattened page list, walked part by part by one
// thread, which keeps the others' registers free of it.
struct Walk {
  int64_t w, w1, run, base;  // base: pages of one (kv head, row tile) before sequence b
  int b, n_b;

  // Tokens of sequence b, the chunk's included (a clamped length is reported by
  // the first CTA's scan).
  static __device__ int tokens(const RowsParams &p, int b, bool report) {
    const int most = p.max_blocks * kPageSize - p.n_new;
    int t = __ldg(p.ctx_lens + b);
    if (t < 0 || t > most) {
      if (report) record_error(p.status, PA_ERR_BAD_CTX);
      t = t < 0 ? 0 : most;
    }
    return t + p.n_new;
  }
  // An empty sequence counts one page, so that someone writes its zeros.
  static __device__ int pages(int tokens) {
    return max(1, (tokens + kPageSize - 1) / kPageSize);
  }
  // The whole warp: lane l sums the pages of sequences [l per, (l + 1) per), and a
  // scan finds the sequence in which this CTA's run starts.  False: no run.
  // Warp-uniform results; lane 0 keeps them in *out.
  static __device__ bool start(const RowsParams &p, int lane, Walk *out) {
    Walk x;
    const int heads = p.n_kv_heads * p.n_sub;
    const int per = (p.batch + 31) / 32;
    const int b0 = min(p.batch, lane * per), b1 = min(p.batch, b0 + per);
    int64_t sum = 0;
#pragma unroll 4
    for (int i = b0; i < b1; ++i) sum += pages(tokens(p, i, blockIdx.x == 0));
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    const int64_t total = __shfl_sync(kFull, incl, 31) * heads;
    x.run = max((total + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(kMinPages));
    x.w = blockIdx.x * x.run;
    x.w1 = min(total, x.w + x.run);
    if (x.w >= x.w1) return false;
    const int src = __ffs(__ballot_sync(kFull, incl * heads > x.w)) - 1;
    x.b = __shfl_sync(kFull, b0, src);
    x.base = __shfl_sync(kFull, incl - sum, src);
    x.n_b = pages(tokens(p, x.b, false));
    if (lane == 0) *out = x;
    return true;
  }
  __device__ void next(const RowsParams &p, volatile Part &s) {
    const int heads = p.n_kv_heads * p.n_sub;
    while ((base + n_b) * heads <= w) {
      base += n_b;
      n_b = pages(tokens(p, ++b, false));
    }
    const int64_t rel = w - base * heads;
    const int item = static_cast<int>(rel / n_b);
    const int pg0 = static_cast<int>(rel - static_cast<int64_t>(item) * n_b);
    const int n_pg = static_cast<int>(min(static_cast<int64_t>(n_b - pg0), w1 - w));
    const int64_t i0 = w - pg0;  // the item's first page
    s.b = b;
    s.g = item / p.n_sub;
    s.r0 = (item % p.n_sub) * p.tile_rows;
    s.n_r = min(p.tile_rows, p.n_rows - (item % p.n_sub) * p.tile_rows);
    s.pg0 = pg0;
    s.n_pg = n_pg;
    s.tokens = tokens(p, b, false);
    s.first = static_cast<int>(i0 / run);
    s.last = static_cast<int>((i0 + n_b - 1) / run);
    s.slot = i0 % run == 0 ? 0 : 1;
    w += n_pg;
    s.more = w < w1;
  }
};

template <int D, bool BF16, bool WIDE, bool OUT16>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm)
    kv4_rows_kernel(const RowsParams p) {
  using L = RowsSmem<D>;
  constexpr int MT = D / 16;   // row tiles of the second product (head dimensions)
  constexpr int KW = D / 32;   // 32-bit words of K codes a thread holds per token
  constexpr int VW = D / 64;   // of V codes
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ln = lane >> 2, lc = lane & 3;

  if (tid == 0) {
    for (int s = 0; s < kWarps * kStages; ++s) mbar_init(sb + L::kBars + 8 * s, 1);
    fence_mbar_init();
  }
  griddep_release();
  griddep_wait();  // inputs may come from the previous kernel in the stream
  __syncthreads();

  volatile Part *parts = reinterpret_cast<volatile Part *>(smem + L::kParts);
  volatile int *s_last = reinterpret_cast<volatile int *>(smem + L::kLast);
  Walk *walk = reinterpret_cast<Walk *>(smem + L::kWalk);
  if (warp == kWarps - 1) {  // the warp with the fewest pages plans
    const bool any = Walk::start(p, lane, walk);
    if (lane == 0) {
      if (any) walk->next(p, parts[0]);
      *s_last = any;
    }
  }
  __syncthreads();
  if (!*s_last) return;

  BlockRing<D> ring;
  ring.stage0 = sb + warp * kStages * L::kStage;
  ring.bar0 = sb + L::kBars + warp * kStages * 8;
  ring.issued = ring.waited = 0;
  bool alive = true;  // false once a wait of this warp has run out

  float *mer_o = reinterpret_cast<float *>(smem + L::kMergeO);
  float *mer_m = reinterpret_cast<float *>(smem + L::kMergeM);
  float *mer_l = reinterpret_cast<float *>(smem + L::kMergeL);
  const int tk = token_of(ln);
  // V rows of the tokens that score rows 2 lc and 2 lc + 1 stand for
  const int t0 = token_of(2 * lc) * kv4::row_bytes(D);
  const int t1 = token_of(2 * lc + 1) * kv4::row_bytes(D);

  for (int turn = 0;; turn ^= 1) {
    volatile Part &part = parts[turn];
    const int first_page = part.pg0 + kPair * warp;
    int key0 = first_page * kPageSize;  // of the chunk at hand
    {
      const int b = part.b;
      ring.bt_row = p.block_table + static_cast<size_t>(b) * p.max_blocks + first_page;
      ring.cache = p.cache + static_cast<size_t>(part.g) * L::kBlock;
      ring.pages = part.tokens > 0 && alive ? part.n_pg - kPair * warp : 0;
      ring.n = max(0, (ring.pages + kWarps * kPair - 1) / (kWarps * kPair));
    }
    ring.start(lane);
    for (int i = 0; i < kStages && i < ring.n; ++i) ring.issue(i, lane, p);
    if (tid == (kWarps - 1) * 32 && part.more) walk->next(p, parts[turn ^ 1]);

    // ---- q of this lane's column as the first product's operand
    // row r of the kv head: query r / G, head r % G
    auto q_row = [&](int r) {
      return (static_cast<size_t>(part.b) * p.queries + r / p.group) * p.n_q_heads +
             part.g * p.group + r % p.group;
    };
    const int n_r = part.n_r;
    uint32_t qb[2 * KW][2];
    float f0, f1, e0, e1;  // per column 2 lc, 2 lc + 1: score factor, scaled sum of q
    {
      const int col = WIDE ? ln : (ln & 3);
      float x[8 * KW];
      if (col < n_r) {
        const uint4 *src4 =
            reinterpret_cast<const uint4 *>(p.q + q_row(part.r0 + col) * D + (D / 4) * lc);
#pragma unroll
        for (int k = 0; k < KW; ++k) {
          const uint4 v = __ldg(src4 + k);
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
      // 2^ex brings the row's largest magnitude into [2^14, 2^15)
      const int ex = min(90, max(-90, 14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127)));
      const float up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
      const float up16 = up * 0.0625f;
#pragma unroll
      for (int k = 0; k < KW; ++k)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int d0 = 8 * k + 2 * s;
          qb[2 * k + s][0] = pack2<false>(x[d0] * up, x[d0 + 4] * up);
          qb[2 * k + s][1] = pack2<false>(x[d0 + 1] * up16, x[d0 + 5] * up16);
        }
      const float f = p.qscale * __uint_as_float(static_cast<uint32_t>(127 + 24 - ex) << 23);
      const float e = p.qscale * total_q;
      f0 = __shfl_sync(kFull, f, 8 * lc);
      f1 = __shfl_sync(kFull, f, 8 * lc + 4);
      e0 = __shfl_sync(kFull, e, 8 * lc);
      e1 = __shfl_sync(kFull, e, 8 * lc + 4);
    }

    float o[MT][4];
#pragma unroll
    for (int k = 0; k < MT; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
    // per row 2 lc (x) and 2 lc + 1 (y): the running max, negated, the sums l and z
    float2 nm = make_float2(-kNoKey, -kNoKey);
    float2 l2 = make_float2(0.f, 0.f), z2 = make_float2(0.f, 0.f);
    float v_ref = 0.f, v_inv = 0.f;  // reference of scale_v (a power of two), 2^7 / it
    const float2 f2 = make_float2(f0, f1), e2 = make_float2(e0, e1);
    const float2 e8 = make_float2(-8.f * e0, -8.f * e1);
    const float rem = lc < 2 ? 0.f : -1.f;  // this lane's columns carry remainder terms

    // Keys that every row of the tile sees and this part holds end here.
    const int part_end = (part.pg0 + part.n_pg) * kPageSize;
    const int lim_all = min(part_end, OUT16 ? part.tokens - p.n_new + 1 + part.r0 / p.group
                                            : part.tokens);
    for (int i = 0; i < ring.n; ++i, key0 += kWarps * kPair * kPageSize) {
      const uint32_t st = ring.wait(lane, p);
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
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KW; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t xa = ka[k] >> (8 * h), xb = kb[k] >> (8 * h);
            const uint32_t a[4] = {xa & 0x000f000fu, xb & 0x000f000fu, xa & 0x00f000f0u,
                                   xb & 0x00f000f0u};
            mma16816<false>(acc, a, qb[2 * k + h][0], qb[2 * k + h][1]);
          }
        const float2 k0 = unpack2<BF16>(km0), k1 = unpack2<BF16>(km1);
        s[2 * pg] = __ffma2_rn(make_float2(k0.x, k0.x),
                               __ffma2_rn(f2, make_float2(acc[0], acc[1]), e8),
                               __fmul2_rn(make_float2(k0.y, k0.y), e2));
        s[2 * pg + 1] = __ffma2_rn(make_float2(k1.x, k1.x),
                                   __ffma2_rn(f2, make_float2(acc[2], acc[3]), e8),
                                   __fmul2_rn(make_float2(k1.y, k1.y), e2));
      }
      if (key0 + kPair * kPageSize > lim_all) {
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
          o[k][0] *= c.x;
          o[k][1] *= c.y;
          o[k][2] *= c.x;
          o[k][3] *= c.y;
        }
#pragma unroll
        for (int u = 0; u < 2 * kPair; ++u) d[u] = __fadd2_rn(s[u], nm);
      }

      // ---- weights, as the second product's operand
      uint32_t hi[2 * kPair], lo[2 * kPair];
#pragma unroll
      for (int u = 0; u < 2 * kPair; ++u) {
        const float2 pr = make_float2(ex2(d[u].x), ex2(d[u].y));
        l2 = __fadd2_rn(l2, pr);
        z2 = __ffma2_rn(pr, make_float2(v[u].y, v[u].y), z2);
        const float x = v[u].x * v_inv;
        const float2 wt = __fmul2_rn(pr, make_float2(x, x));
        const uint32_t head = pack2<false>(wt.x, wt.y);
        const float2 back = unpack2<false>(head);
        if constexpr (WIDE) {
          hi[u] = transpose8x8(head);
          lo[u] = transpose8x8(pack2<false>(wt.x - back.x, wt.y - back.y));
        } else {  // the head term again, or the remainder
          const float2 mine = __ffma2_rn(make_float2(rem, rem), back, wt);
          hi[u] = transpose8x8(pack2<false>(mine.x, mine.y));
          lo[u] = 0;
        }
      }

      // ---- O[dimension][row] += V^T P
#pragma unroll
      for (int pg = 0; pg < kPair; ++pg) {
        const uint32_t col = st + pg * L::kBlock + kv4::code_offset(D, 1, 0) + 4 * VW * ln;
        uint32_t va[4][VW];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t at = col + (u & 1 ? t1 : t0) + 8 * (u >> 1) * kv4::row_bytes(D);
          if constexpr (VW == 2) {
            const uint2 x = lds64(at);
            va[u][0] = x.x, va[u][1] = x.y;
          } else {
            va[u][0] = lds32(at);
          }
        }
#pragma unroll
        for (int j = 0; j < VW; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // nibbles 4 h .. 4 h + 3 of two tokens' words, one token a half
            const uint32_t x = __byte_perm(va[0][j], va[1][j], h ? 0x7632 : 0x5410);
            const uint32_t y = __byte_perm(va[2][j], va[3][j], h ? 0x7632 : 0x5410);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t xs = x >> (8 * u), ys = y >> (8 * u);
              const uint32_t a[4] = {sub_1032((xs & 0x000f000fu) | 0x64006400u),
                                     sixteenth_sub_72((xs & 0x00f000f0u) | 0x64006400u),
                                     sub_1032((ys & 0x000f000fu) | 0x64006400u),
                                     sixteenth_sub_72((ys & 0x00f000f0u) | 0x64006400u)};
              float (&ok)[4] = o[4 * j + 2 * h + u];
              if constexpr (WIDE) {
                float t[4] = {0.f, 0.f, 0.f, 0.f};
                mma16816<false>(t, a, lo[2 * pg], lo[2 * pg + 1]);
                mma16816<false>(t, a, hi[2 * pg], hi[2 * pg + 1]);
                ok[0] += t[0], ok[1] += t[1], ok[2] += t[2], ok[3] += t[3];
              } else {
                mma16816<false>(ok, a, hi[2 * pg], hi[2 * pg + 1]);
              }
            }
          }
      }
      __syncwarp();  // the stage has been read by every lane
      if (i + kStages < ring.n) ring.issue(i + kStages, lane, p);
    }

    // ---- the warp's state to shared memory: O is O[d = (D / 8) ln + 2 k + {0, 1}]
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l2.x += __shfl_xor_sync(kFull, l2.x, x);
      l2.y += __shfl_xor_sync(kFull, l2.y, x);
      z2.x += __shfl_xor_sync(kFull, z2.x, x);
      z2.y += __shfl_xor_sync(kFull, z2.y, x);
    }
    __syncthreads();  // every warp is done with the ring
    const float back = v_ref * 0x1p-7f;
#pragma unroll
    for (int k = 0; k < MT; ++k) {
      float2 a = make_float2(o[k][0], o[k][2]), b = make_float2(o[k][1], o[k][3]);
      if constexpr (!WIDE) {  // columns 4-7 hold the remainder terms of 0-3
        a.x += __shfl_xor_sync(kFull, a.x, 2);
        a.y += __shfl_xor_sync(kFull, a.y, 2);
        b.x += __shfl_xor_sync(kFull, b.x, 2);
        b.y += __shfl_xor_sync(kFull, b.y, 2);
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
    __syncthreads();

    // ---- the item's CTAs: the first holds its start, the last its end
    const int first = part.first, last = part.last;
    auto store = [&](int r, int d, float4 v) {  // row r of the tile, dimensions d .. d + 3
      const size_t at = q_row(part.r0 + r) * D + d;
      if constexpr (OUT16)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
            make_uint2(pack2<BF16>(v.x, v.y), pack2<BF16>(v.z, v.w));
      else
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = v;
    };
    // CTA c's state of this item: slot 0 when its part starts the CTA's run.
    auto state = [&](int c, int r) {
      const int slot = c > first ? 0 : part.slot;
      return p.ws + ((static_cast<size_t>(c) * 2 + slot) * kTile + r) * (D + 4);
    };
    for (int e = tid; e < n_r * (D / 4); e += kWarps * 32) {
      const int r = e / (D / 4), d = 4 * (e % (D / 4));
      float M = kNoKey;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) M = fmaxf(M, mer_m[k * kTile + r]);
      float l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float lk = mer_l[k * kTile + r];
        const float f = ex2(mer_m[k * kTile + r] - M);
        const float4 v =
            *reinterpret_cast<const float4 *>(mer_o + (k * kTile + r) * L::kRowStride + d);
        l = fmaf(f, lk, l);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
      }
      if (first == last) {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // no key: zeros; NaN stays NaN
        store(r, d, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
      } else {
        float *dst = state(blockIdx.x, r);
        *reinterpret_cast<float4 *>(dst + d) = acc;
        if (d == 0) *reinterpret_cast<float2 *>(dst + D) = make_float2(M, l);
      }
    }
    if (first != last) {
      // The last of the item's CTAs to arrive merges their states.  One thread
      // arrives with an acquire-release add behind the barrier, so the CTA's
      // states are visible before its arrival counts, and every other CTA's
      // states to the last one.
      __syncthreads();
      if (tid == 0) *s_last = atomic_add_acq_rel_gpu(p.ctr + first, 1) == last - first;
      __syncthreads();
      if (*s_last) {
        for (int e = tid; e < n_r * (D / 4); e += kWarps * 32) {
          const int r = e / (D / 4), d = 4 * (e % (D / 4));
          float m = kNoKey, l = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          constexpr int kBatch = 4;
          for (int c = first; c <= last; c += kBatch) {
            float2 ml[kBatch];
            float4 v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
              if (c + u <= last) {
                const float *sp = state(c + u, r);
                ml[u] = __ldcg(reinterpret_cast<const float2 *>(sp + D));
                v[u] = __ldcg(reinterpret_cast<const float4 *>(sp + d));
              }
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
              if (c + u <= last && ml[u].y != 0.f) {
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
          store(r, d, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        }
      }
    }
    if (!part.more) break;
    fence_proxy_async_smem();  // the merge area's last reads, before copies over it
    __syncthreads();           // ... and the next part is planned
  }
}

template <int D, bool BF16, bool WIDE, bool OUT16>
int launch_rows_t(const RowsParams &p, int ctas, cudaStream_t stream) {
  auto kern = kv4_rows_kernel<D, BF16, WIDE, OUT16>;
  static ContextCache<bool> smem_set;
  if (set_smem_limit(kern, RowsSmem<D>::kBytes, smem_set) != PA_OK) return PA_ERR_CUDA;
  return launch_pdl(kern, dim3(ctas), dim3(kWarps * 32), RowsSmem<D>::kBytes, stream, p) ==
                 cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
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
  return static_cast<size_t>(ctas) * 2 * kTile * (head_dim + 4) * sizeof(float);
}

}  // namespace

size_t kv4_rows_workspace_bytes(int head_dim, int sms) {
  const int ctas = sms * kCtasPerSm;
  return partials_bytes(head_dim, ctas) + static_cast<size_t>(ctas) * sizeof(int);
}

int launch_kv4_rows(const Kv4AttentionLaunch &a, cudaStream_t stream) {
  const int ctas = sm_count() * kCtasPerSm;
  if (ctas <= 0) return PA_ERR_CUDA;
  RowsParams p;
  p.q = static_cast<const uint16_t *>(a.q);
  p.cache = a.cache;
  p.block_table = a.block_table;
  p.ctx_lens = a.ctx_lens;
  p.out = a.out;
  p.ws = static_cast<float *>(a.workspace);
  p.ctr = reinterpret_cast<int *>(static_cast<char *>(a.workspace) +
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
  if (launch_clear_counters(p.ctr, ctas, stream) != PA_OK) return PA_ERR_CUDA;
  if (a.head_dim == 128)
    return a.bf16 ? launch_rows_d<128, true>(p, ctas, stream)
                  : launch_rows_d<128, false>(p, ctas, stream);
  return a.bf16 ? launch_rows_d<64, true>(p, ctas, stream)
                : launch_rows_d<64, false>(p, ctas, stream);
}

}  // namespace pa
