// pa_kv4_append.cu -- appends that rotate (into the 16-bit cache, or quantised
// into the 4-bit one), the read of 4-bit rows as values, and the page copy of
// the 4-bit cache.
//
// Rotation (rotary position embedding): the first rot_dim dimensions of a row
// form rot_dim / 2 pairs (a, b), each turned by its angle at the token's
// position,
//   a' = a cos - b sin,   b' = b cos + a sin,
// with cos and sin from an fp32 table, the products and the sums each rounded
// to fp32 and the result rounded once (to 16 bits, or to a 4-bit code).
//
// Quantisation of a row x (fp32 after the rotation): scale = r16((max - min) /
// 15), zero = r16(min + 8 scale), code = rint((x - zero) / scale) + 8 clamped
// to 0 .. 15, the codes of the formula evaluated step by step in fp32 (a product
// with the reciprocal decides where it is clear, an IEEE division where it is not).
// A scale of 0 gives code 8 (x = zero); a row whose range, scale or zero is not
// finite gives scale = zero = NaN.
//
// Bound: memory.  A row is head_dim / 16 threads of 16 dimensions; thread t
// holds the two 8-element chunks that pair with each other, so a rotation
// needs no exchange, the row's extremes take log2(head_dim / 16) shuffles, and
// the thread's 8 cosines and 8 sines serve each of the NR rows of one token
// that it handles.  NR = 1 while the call is small (more threads: the latency
// of one dependent chain), 4 once there are enough rows to fill the GPU.
// Small CTAs at 80 registers keep 24 warps an SM and the last wave short: 4 x 512 tokens
// 12.4 -> 11.0 us against CTAs of 256 at the compiler's 95, 4 x 2048 quantised and read
// back 55.6 -> 48.3, although the quantising form spills some (56 bytes stored, 72 to 96
// loaded a thread); at 64 registers 17.4 and 51.5.
// Measured: rotation alone, 4 x 512 tokens of 32 / 8 heads of 128: 11.0 us a call
// (51.4 MB, 4.7 TB/s); 8191 tokens of 16 / 16 heads of 64: 19.9 us (101.7 MB, 5.1
// TB/s).  Quantising 4 x 2048 tokens (32 / 8 heads of 128): 37 us for 169 MB, where
// the codes' arithmetic and the loads take turns.
#include <cuda_bf16.h>
#include <float.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_kv4.cuh"

namespace pa {
namespace {

constexpr int kAppendThreads = 128;

struct AppendParams {
  const uint16_t *k_new, *v_new, *q;
  uint16_t *q_out, *k_cache, *v_cache;
  uint8_t *kv4;
  const int32_t *block_table, *seq_idx, *pos;
  const int32_t *turn_pos;  // or null: pos
  const float *cos_sin;
  int *status;
  int64_t k_stride, v_stride, q_stride, total;
  int n_q_heads, n_kv_heads, batch, max_blocks, num_pages;
  int max_pos, rot_dim, rows, row_lanes;
  bool interleaved;
};

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// x rounded to the 16-bit type: its bits, and the value they stand for.
template <bool BF16>
__device__ __forceinline__ uint32_t round16(float x, float &back) {
  const uint32_t w = pack2<BF16>(x, 0.f) & 0xffffu;
  back = unpack1<BF16>(static_cast<uint16_t>(w));
  return w;
}

// Row r of a token: K of kv head r, then V of kv head r - Hkv, then q.
// Thread t of the row holds chunks c0 and c1 (8 elements each).
template <int D, bool BF16, bool KV4, int NR>
__global__ void __launch_bounds__(kAppendThreads, 6) append_rope_kernel(const AppendParams p) {
  constexpr int TPR = D / 16;  // threads per row
  griddep_release();
  griddep_wait();  // the rows may come from the previous kernel in the stream
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= p.total) return;
  const int t = static_cast<int>(idx % TPR);
  const int64_t unit = idx / TPR;
  const int64_t j = p.total >> 32 ? unit / p.row_lanes
                                  : static_cast<uint32_t>(unit) / static_cast<uint32_t>(p.row_lanes);
  const int r0 = static_cast<int>(unit - j * p.row_lanes);

  const int b = p.seq_idx[j], pos = p.pos[j];
  const int at = p.turn_pos ? p.turn_pos[j] : pos;  // the position it is rotated by
  const bool turn = p.cos_sin != nullptr;
  const int half_chunks = p.rot_dim / 16;         // chunks of rotated first elements
  const bool mine = turn && t < half_chunks;      // this thread's chunks are rotated
  const bool split = mine && !p.interleaved;      // pairs (i, i + rot / 2)
  const int rc0 = split ? t : 2 * t, rc1 = split ? t + half_chunks : 2 * t + 1;
  // the rows, on their way while the place is looked up
  uint4 in[NR][2];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = r0 + i * p.row_lanes;
    if (r >= p.rows) break;
    const bool is_v = r >= p.n_kv_heads && r < 2 * p.n_kv_heads;
    const uint16_t *src =
        r < p.n_kv_heads ? p.k_new + j * p.k_stride + static_cast<int64_t>(r) * D
        : is_v ? p.v_new + j * p.v_stride + static_cast<int64_t>(r - p.n_kv_heads) * D
               : p.q + j * p.q_stride + static_cast<int64_t>(r - 2 * p.n_kv_heads) * D;
    const uint4 *s4 = reinterpret_cast<const uint4 *>(src);
    in[i][0] = s4[is_v ? 2 * t : rc0];
    in[i][1] = s4[is_v ? 2 * t + 1 : rc1];
  }

  const bool reporter = t == 0 && r0 == 0;
  if (b < 0 || b >= p.batch || pos < 0 || pos >= p.max_blocks * kPageSize ||
      (turn && (at < 0 || at >= p.max_pos))) {
    if (reporter) record_error(p.status, PA_ERR_BAD_INDEX);
    return;
  }
  const int page = p.block_table[static_cast<size_t>(b) * p.max_blocks + pos / kPageSize];
  float cs[8], sn[8];
  if (mine) {
    const float4 *row = reinterpret_cast<const float4 *>(
        p.cos_sin + static_cast<size_t>(at) * p.rot_dim);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 c = row[2 * t + k], s = row[p.rot_dim / 8 + 2 * t + k];
      cs[4 * k] = c.x, cs[4 * k + 1] = c.y, cs[4 * k + 2] = c.z, cs[4 * k + 3] = c.w;
      sn[4 * k] = s.x, sn[4 * k + 1] = s.y, sn[4 * k + 2] = s.z, sn[4 * k + 3] = s.w;
    }
  }
  if (page < 0 || page >= p.num_pages) {
    if (reporter) record_error(p.status, PA_ERR_BAD_BLOCK);
    return;
  }
  const int slot = pos % kPageSize;

#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = r0 + i * p.row_lanes;
    if (r >= p.rows) break;
    const bool is_v = r >= p.n_kv_heads && r < 2 * p.n_kv_heads;
    const bool is_q = r >= 2 * p.n_kv_heads;
    const int c0 = is_v ? 2 * t : rc0, c1 = is_v ? 2 * t + 1 : rc1;
    float x[16];
    {
      const uint32_t w[8] = {in[i][0].x, in[i][0].y, in[i][0].z, in[i][0].w,
                             in[i][1].x, in[i][1].y, in[i][1].z, in[i][1].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 f = unpack2<BF16>(w[k]);
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
    }
    if (mine && !is_v) {
      auto turn_pair = [&](float &xa, float &xb, int k) {
        const float a = xa, bb = xb;
        xa = __fsub_rn(__fmul_rn(a, cs[k]), __fmul_rn(bb, sn[k]));
        xb = __fadd_rn(__fmul_rn(bb, cs[k]), __fmul_rn(a, sn[k]));
      };
      if (p.interleaved) {
#pragma unroll
        for (int k = 0; k < 8; ++k) turn_pair(x[2 * k], x[2 * k + 1], k);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) turn_pair(x[k], x[8 + k], k);
      }
    }
    const int g = is_v ? r - p.n_kv_heads : r;
    if (!KV4 || is_q) {
      uint16_t *dst;
      if (is_q) {
        dst = p.q_out + (j * p.n_q_heads + (r - 2 * p.n_kv_heads)) * D;
      } else {
        dst = (is_v ? p.v_cache : p.k_cache) +
              ((static_cast<size_t>(page) * p.n_kv_heads + g) * kPageSize + slot) * D;
      }
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = pack2<BF16>(x[2 * k], x[2 * k + 1]);
      uint4 *d4 = reinterpret_cast<uint4 *>(dst);
      // chunks that are not rotated keep their bits (NaN payloads included)
      d4[c0] = (mine && !is_v) ? make_uint4(o[0], o[1], o[2], o[3]) : in[i][0];
      d4[c1] = (mine && !is_v) ? make_uint4(o[4], o[5], o[6], o[7]) : in[i][1];
    } else {
      float mn = x[0], mx = x[0];
#pragma unroll
      for (int k = 1; k < 16; ++k) {
        mn = min_nan(mn, x[k]);
        mx = max_nan(mx, x[k]);
      }
      const int lane = threadIdx.x & 31;
      const unsigned grp = ((1u << TPR) - 1u) << (lane & ~(TPR - 1));  // the row's lanes
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) {
        mn = min_nan(mn, __shfl_xor_sync(grp, mn, o));
        mx = max_nan(mx, __shfl_xor_sync(grp, mx, o));
      }
      const float range = __fsub_rn(mx, mn);
      float s, z;
      uint32_t sb = round16<BF16>(__fmul_rn(range, 1.0f / 15.0f), s);
      uint32_t zb = round16<BF16>(__fmaf_rn(8.f, s, mn), z);
      const bool fine = fabsf(range) <= FLT_MAX && fabsf(s) <= FLT_MAX && fabsf(z) <= FLT_MAX;
      if (!fine) sb = zb = BF16 ? 0x7fc0u : 0x7e00u;
      // (x - z) / s by the reciprocal, off by two half steps, 2^-23 of the quotient: at
      // most 2^-20 up to 8, and a larger one (the zero's own rounding against a small
      // scale) is clamped.  A row with an element within 1e-4 of the border between two
      // codes is divided out.
      const bool step = fine && s > 0.f;
      const float inv = step ? __fdiv_rn(1.f, s) : 0.f;
      float c[16];
      bool near = false;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float y = __fsub_rn(x[k], z) * inv;
        c[k] = rintf(y);
        near |= !(fabsf(y - c[k]) < 0.4999f);
      }
      if (near && step) {
#pragma unroll
        for (int k = 0; k < 16; ++k) c[k] = rintf(__fdiv_rn(__fsub_rn(x[k], z), s));
      }
      uint32_t code[2] = {0u, 0u};
#pragma unroll
      for (int k = 0; k < 16; ++k)
        code[k >> 3] |= static_cast<uint32_t>(step ? fminf(fmaxf(c[k] + 8.f, 0.f), 15.f) : 8.f)
                        << (4 * (k & 7));
      uint8_t *blk = p.kv4 + (static_cast<size_t>(page) * p.n_kv_heads + g) *
                                 kv4::block_bytes(D);
      uint32_t *row = reinterpret_cast<uint32_t *>(blk + kv4::code_offset(D, is_v, slot));
      row[c0] = code[0];
      row[c1] = code[1];
      if (t == 0)
        *reinterpret_cast<uint32_t *>(blk + kv4::meta_offset(D, is_v, slot)) = sb | (zb << 16);
    }
  }
}

template <int D, bool BF16, bool KV4>
int launch_append_t(const AppendRopeLaunch &a, cudaStream_t stream) {
  AppendParams p;
  p.k_new = static_cast<const uint16_t *>(a.k_new);
  p.v_new = static_cast<const uint16_t *>(a.v_new);
  p.q = static_cast<const uint16_t *>(a.q);
  p.q_out = static_cast<uint16_t *>(a.q_out);
  p.k_cache = static_cast<uint16_t *>(a.k_cache);
  p.v_cache = static_cast<uint16_t *>(a.v_cache);
  p.kv4 = a.kv4_cache;
  p.block_table = a.block_table;
  p.seq_idx = a.seq_idx;
  p.pos = a.pos;
  p.turn_pos = a.turn_pos;
  p.cos_sin = a.cos_sin;
  p.status = a.status;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.q_stride = a.q_stride;
  p.n_q_heads = a.n_q_heads;
  p.n_kv_heads = a.n_kv_heads;
  p.batch = a.batch;
  p.max_blocks = a.max_blocks;
  p.num_pages = a.num_pages;
  p.max_pos = a.max_pos;
  p.rot_dim = a.rot_dim;
  p.interleaved = a.interleaved;
  p.rows = 2 * a.n_kv_heads + (a.q ? a.n_q_heads : 0);
  constexpr int TPR = D / 16, kThreads = kAppendThreads;
  // One row a thread until the threads would fill about two waves of the GPU.
  const bool many = static_cast<int64_t>(a.n_tok) * p.rows * TPR > 2 * 152 * 2048;
  const int nr = many ? 4 : 1;
  p.row_lanes = (p.rows + nr - 1) / nr;
  p.total = static_cast<int64_t>(a.n_tok) * p.row_lanes * TPR;
  const int64_t blocks = (p.total + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return PA_ERR_SHAPE;
  const dim3 grid(static_cast<unsigned>(blocks));
  const cudaError_t e =
      many ? launch_pdl(append_rope_kernel<D, BF16, KV4, 4>, grid, dim3(kThreads), 0, stream, p)
           : launch_pdl(append_rope_kernel<D, BF16, KV4, 1>, grid, dim3(kThreads), 0, stream, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// Bound: issue (44 instructions per 16 bytes).  16 x 1000 tokens of 8 heads of 128: 17.9
// us a call for 86 MB, 4.8 TB/s.
// ---- read: a CTA takes `per_cta` tokens, whose places its first threads look up for
// all; a thread 8 dimensions (16 bytes out) of four rows at a time
struct ReadParams {
  const uint8_t *cache;
  const int32_t *block_table, *seq_idx, *pos;
  uint16_t *k_out, *v_out;
  int *status;
  int n_tok, per_cta, n_kv_heads, batch, max_blocks, num_pages;
};
constexpr int kReadThreads = 256, kReadTokens = 64;  // tokens a CTA at most

// zero + scale (code - 8) of a word's eight codes, rounded once: nibbles k and k + 4 as
// the two halves of a 16-bit pair (its bits under those of 2^10 or 2^7 are 1024 + code or
// 128 + code), whose difference from 1032 or 136 is exact, and one FMA.
template <bool BF16>
__device__ __forceinline__ uint4 values_of(uint32_t code, uint32_t meta) {
  using H = std::conditional_t<BF16, __nv_bfloat162, __half2>;
  const uint32_t ss = __byte_perm(meta, meta, 0x1010), zz = __byte_perm(meta, meta, 0x3232);
  const uint32_t eight = BF16 ? 0x43084308u : 0x64086408u;  // 128 + 8, 1024 + 8
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w = ((code >> (4 * k)) & 0x000f000fu) | (BF16 ? 0x43004300u : 0x64006400u);
    const H c = __hsub2(*reinterpret_cast<const H *>(&w), *reinterpret_cast<const H *>(&eight));
    const H x = __hfma2(*reinterpret_cast<const H *>(&ss), c, *reinterpret_cast<const H *>(&zz));
    o[k] = *reinterpret_cast<const uint32_t *>(&x);
  }
  return make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410),
                    __byte_perm(o[0], o[1], 0x7632), __byte_perm(o[2], o[3], 0x7632));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kReadThreads) read_kv4_kernel(const ReadParams p) {
  constexpr int TPR = D / 8, kUnroll = 4;
  __shared__ const uint8_t *place[kReadTokens];  // the token's page, or null
  __shared__ int slots[kReadTokens];
  griddep_release();
  griddep_wait();
  const int j0 = blockIdx.x * p.per_cta, n = min(p.per_cta, p.n_tok - j0);
  const int64_t page_bytes = static_cast<int64_t>(p.n_kv_heads) * kv4::block_bytes(D);
  if (threadIdx.x < n) {
    const int b = p.seq_idx[j0 + threadIdx.x], pos = p.pos[j0 + threadIdx.x];
    const uint8_t *at = nullptr;
    if (b < 0 || b >= p.batch || pos < 0 || pos >= p.max_blocks * kPageSize) {
      record_error(p.status, PA_ERR_BAD_INDEX);
    } else {
      const int page = p.block_table[static_cast<size_t>(b) * p.max_blocks + pos / kPageSize];
      if (page < 0 || page >= p.num_pages)
        record_error(p.status, PA_ERR_BAD_BLOCK);
      else
        at = p.cache + page * page_bytes;
    }
    place[threadIdx.x] = at;
    slots[threadIdx.x] = pos & (kPageSize - 1);
  }
  __syncthreads();
  // unit (token, K or V, kv head, 8 dimensions), the last fastest: a thread's next one is
  // kReadThreads / TPR rows on
  const uint32_t heads = p.n_kv_heads, per_token = 2 * heads, t = threadIdx.x % TPR;
  constexpr uint32_t kStep = kReadThreads / TPR;
  const uint32_t step_j = kStep / per_token, step_r = kStep % per_token;
  uint32_t j = threadIdx.x / TPR / per_token, r = threadIdx.x / TPR % per_token;
  while (j < n) {
    uint32_t code[kUnroll], meta[kUnroll];
    uint4 *dst[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      dst[i] = nullptr;
      const uint8_t *blk = j < n ? place[j] : nullptr;
      if (blk) {
        const uint32_t which = r >= heads, g = r - (which ? heads : 0);
        const int slot = slots[j];
        blk += g * static_cast<uint32_t>(kv4::block_bytes(D));
        auto word = [&](int at) { return reinterpret_cast<const uint32_t *>(blk + at); };
        code[i] = __ldcg(word(kv4::code_offset(D, which, slot)) + t);
        meta[i] = __ldcg(word(kv4::meta_offset(D, which, slot)));
        dst[i] = reinterpret_cast<uint4 *>(which ? p.v_out : p.k_out) +
                 (static_cast<size_t>(j0 + j) * heads + g) * TPR + t;
      }
      j += step_j;
      r += step_r;
      if (r >= per_token) r -= per_token, ++j;
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      if (dst[i]) *dst[i] = values_of<BF16>(code[i], meta[i]);
  }
}

template <int D, bool BF16>
int launch_read_t(const ReadKv4Launch &a, cudaStream_t stream) {
  ReadParams p;
  p.cache = a.cache;
  p.block_table = a.block_table;
  p.seq_idx = a.seq_idx;
  p.pos = a.pos;
  p.k_out = static_cast<uint16_t *>(a.k_out);
  p.v_out = static_cast<uint16_t *>(a.v_out);
  p.status = a.status;
  p.n_tok = a.n_tok;
  p.n_kv_heads = a.n_kv_heads;
  p.batch = a.batch;
  p.max_blocks = a.max_blocks;
  p.num_pages = a.num_pages;
  // As few tokens a CTA as leave about one wave of CTAs, eight an SM.
  const int tokens = min(kReadTokens, (a.n_tok - 1) / (152 * 8) + 1);
  p.per_cta = tokens;
  const int blocks = (a.n_tok - 1) / tokens + 1;
  return launch_pdl(read_kv4_kernel<D, BF16>, dim3(blocks), dim3(kReadThreads), 0, stream, p) ==
                 cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

// ---- whole pages src[i] -> dst[i], every kv head, 16 bytes a thread
__global__ void __launch_bounds__(256)
    copy_pages_kv4_kernel(uint4 *cache, const int32_t *src, const int32_t *dst, int num_pages,
                          int64_t page_vecs, int *status) {
  griddep_release();
  griddep_wait();
  const int s = src[blockIdx.x], d = dst[blockIdx.x];
  if (s < 0 || s >= num_pages || d < 0 || d >= num_pages) {
    if (threadIdx.x == 0) record_error(status, PA_ERR_BAD_BLOCK);
    return;
  }
  const uint4 *from = cache + s * page_vecs;
  uint4 *to = cache + d * page_vecs;
  for (int64_t e = threadIdx.x; e < page_vecs; e += blockDim.x) to[e] = from[e];
}

}  // namespace

int launch_append_rope(const AppendRopeLaunch &a, cudaStream_t stream) {
  const bool k4 = a.kv4_cache != nullptr;
  if (a.head_dim == 128) {
    if (k4) return a.bf16 ? launch_append_t<128, true, true>(a, stream)
                          : launch_append_t<128, false, true>(a, stream);
    return a.bf16 ? launch_append_t<128, true, false>(a, stream)
                  : launch_append_t<128, false, false>(a, stream);
  }
  if (k4) return a.bf16 ? launch_append_t<64, true, true>(a, stream)
                        : launch_append_t<64, false, true>(a, stream);
  return a.bf16 ? launch_append_t<64, true, false>(a, stream)
                : launch_append_t<64, false, false>(a, stream);
}

int launch_read_kv4(const ReadKv4Launch &a, cudaStream_t stream) {
  if (a.head_dim == 128)
    return a.bf16 ? launch_read_t<128, true>(a, stream) : launch_read_t<128, false>(a, stream);
  return a.bf16 ? launch_read_t<64, true>(a, stream) : launch_read_t<64, false>(a, stream);
}

int launch_copy_pages_kv4(uint8_t *cache, const int32_t *src, const int32_t *dst, int *status,
                          int n, int n_kv_heads, int head_dim, int num_pages,
                          cudaStream_t stream) {
  const int64_t vecs = static_cast<int64_t>(n_kv_heads) * kv4::block_bytes(head_dim) / 16;
  return launch_pdl(copy_pages_kv4_kernel, dim3(n), dim3(256), 0, stream,
                    reinterpret_cast<uint4 *>(cache), src, dst, num_pages, vecs,
                    status) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // namespace pa
