// Shared by the attention operators (attn_rope.cu, attn_rows.cu, attn_chunk.cu,
// attn_join.cu): the views of head rows, paged cache and batch that the C-ABI
// layer fills in, and the device helpers that read them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace nvmoe {

// bf16 rows [T, heads, head_dim] with strides in elements.
struct HeadRows {
  void* data;
  int64_t token_stride, head_stride;
  int heads;
};

struct KvCacheView {
  void* k;
  void* v;
  bool fp8;                 // E4M3, else bf16
  int heads, head_dim;
  int page_shift;           // page_size = 1 << page_shift
  int64_t num_pages;
  int64_t page_stride, token_stride, head_stride;   // elements
  const float* k_scale;     // [heads] or null
  const float* v_scale;
};

struct BatchView {
  int batch, max_new;
  int64_t tokens, max_pages;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* page_table;
};

// Norm and rotation of head rows (the weights are bf16 [head_dim] or null).
struct HeadTransform {
  const float* rope;        // [rope_positions, rotary_dim] or null
  int64_t rope_positions;
  int rotary_dim, interleaved;
  const __nv_bfloat16* q_weight;
  const __nv_bfloat16* k_weight;
  float eps;
};

// q and k (either may have 0 heads) to q_out and k_out at given positions.
cudaError_t launch_qk_norm_rope(const HeadRows& q, const HeadRows& k, int64_t T, int head_dim,
                                const int32_t* positions, const HeadTransform& tr,
                                const HeadRows& q_out, const HeadRows& k_out, int* status,
                                cudaStream_t stream);
// k and v into the cache (and q, if it has heads, to q_out) at the cache
// positions of the batch.
cudaError_t launch_kv_append(const HeadRows& q, const HeadRows& k, const HeadRows& v,
                             const KvCacheView& cache, const BatchView& batch,
                             const HeadTransform& tr, const HeadRows& q_out, int* status,
                             cudaStream_t stream);

// Keys of a tile: the unit in which attention work is shared out.
constexpr int kAttnTileKeys = 128;

// A segment (the keys that one block of rows sees) cut by borders between
// CTAs: begun by CTA b (as its last piece, slot 1), ended by CTA `last`; the
// CTAs after b hold their part in slot 0.  rows = 0: CTA b begins none.
struct AttnPiece {
  int rows;          // valid rows
  int head;          // key head
  int64_t first;     // first token of the request
  int row0;          // first row: row i is token first + (row0 + i) / group
  int last;
};

// Where a CTA of the chunk kernel starts: `left` tiles from tile `tile` of the
// segment (request, key head, row block).
struct AttnStart {
  long long left;
  int request, head, block, tile;
  int last;                   // the CTA that ends the segment which this one leaves cut
};

// First tile of share c when `total` tiles are dealt to g <= total takers (so
// that none is without).
__device__ __forceinline__ long long share_begin(long long total, int c, int g) {
  if (total < (1 << 22))       // (c <= g <= 256: the product fits 32 bits)
    return static_cast<uint32_t>(total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(g);
  return total * c / g;
}
// Takers among `grid` CTAs.
__device__ __forceinline__ int share_takers(long long total, int grid) {
  return total < grid ? static_cast<int>(total) : grid;
}

// x / d for 0 <= x < 2^31 by a product and shifts (Granlund and Montgomery,
// "Division by invariant integers using multiplication", 1994).
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t divisor) : d(divisor), shift(0) {
    while ((uint64_t{1} << shift) < divisor) ++shift;              // ceil(log2 d)
    mul = static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{1} << shift) - divisor)) /
                                    divisor + 1);
  }
  __device__ __forceinline__ int operator()(int x) const {
    const uint32_t t = __umulhi(mul, static_cast<uint32_t>(x));
    const uint32_t half = (static_cast<uint32_t>(x) - t) >> (shift > 0 ? 1 : 0);
    return static_cast<int>((t + half) >> (shift > 0 ? shift - 1 : 0));
  }
};

struct AttnArgs {
  HeadRows q;
  HeadRows out;
  float* lse;               // [tokens, q heads] or null
  KvCacheView cache;
  BatchView batch;
  float scale;
  int window;
  int* status;
  FastDiv group;            // query heads of a key head
  // pieces of cut segments: [grid], [grid][2][piece_rows][D] sums before the
  // division, [grid][2][piece_rows] (maximum in powers of two, weight sum)
  AttnPiece* pieces;
  float* piece_o;
  float2* piece_ml;
  int piece_rows;
  // chunk kernel: blocks before each request [batch + 1], cost in tiles of those
  // before each block [max_blocks + 1] (one key head), the CTAs' starts [grid]
  int* plan_block0;
  long long* plan_cost0;
  AttnStart* starts;
  int max_blocks;
  bool plan_here;           // in the chunk kernel itself; else by attn_plan_kernel
};
constexpr int kAttnTileRows = 128;    // query rows of a tile (block) of the chunk kernel
// Rows of a segment up to which attention_rows_kernel takes the call: one m16 tile.
// Two such tiles against the chunk kernel at 28 rows, bf16 and E4M3 caches: 64
// requests of up to 16384 tokens 273 and 257 us against 244 and 169, of 2000 tokens
// 70 and 70 against 56 and 64, 2 of 131072 171 and 158 against 181 and 115; one of
// 1000, bf16, 15 against 19.
constexpr int kAttnFewRows = 16;
// map_k, map_v: [num_pages, heads, page_size, D] by strides, boxes of up to
// 128 tokens of one page and head.
cudaError_t launch_attention_rows(const AttnArgs& args, const CUtensorMap& map_k,
                                  const CUtensorMap& map_v, int grid, cudaStream_t stream);
// Blocks and requests up to which the chunk kernel's CTAs plan for themselves: a
// thread for each (of 384 or 512).
constexpr int kAttnPlanHere = 384;
cudaError_t launch_attn_plan(const AttnArgs& args, int grid, cudaStream_t stream);
cudaError_t launch_attention_chunk(const AttnArgs& args, const CUtensorMap& map_k,
                                   const CUtensorMap& map_v, int grid, cudaStream_t stream);
cudaError_t launch_attn_combine(const AttnArgs& args, int grid, cudaStream_t stream);

// New tokens and cached length of request r as the kernels take them, kept
// inside the buffers whatever q_start and kv_len hold: rows [first, first + n)
// of q, the first of them at cache position pos0 (negative if the length is
// below n), `len` keys.  Tokens past the ends of q count for the positions.
struct Request {
  int64_t first;
  int n;
  int pos0, len;
};
__device__ __forceinline__ Request load_request(const BatchView& b, int page_shift, int r,
                                                int* status) {
  Request q;
  const int64_t begin = b.q_start[r], end = b.q_start[r + 1];
  int64_t a = begin, e = end;
  const int64_t cap = b.max_pages << page_shift;   // < 2^31, checked on the host
  int64_t len = b.kv_len[r];
  if (a < 0) a = 0;
  if (e > b.tokens) e = b.tokens;
  int64_t n = e > a ? e - a : 0;
  const int64_t pos0 = n > 0 ? len - (end - a) : len;
  if (n > b.max_new || len > cap || begin < 0 || end < begin || end > b.tokens)
    record_status(status, kErrBadIndex);
  if (n > b.max_new) n = b.max_new;
  if (len > cap) len = cap;
  if (len < 0) len = 0;
  q.first = a;
  q.n = static_cast<int>(n);
  q.pos0 = pos0 < -(int64_t{1} << 30) ? -(1 << 30) : static_cast<int>(pos0);
  q.len = static_cast<int>(len);
  return q;
}

// First key that a row at cache position pos sees, which may be negative (window up to
// 2^31 - 1, 0: no window).
__device__ __forceinline__ int first_key(int pos, int window) {
  return window > 0 && pos >= window ? pos - window + 1 : 0;
}

// Of the boxes of `box` keys that make up a tile from key0 on, how many hold a
// key of [kbeg, kend).
__device__ __forceinline__ int boxes_of(int key0, int box, int kbeg, int kend) {
  const int first = max(0, kbeg - key0) / box;
  const int last = (min(kAttnTileKeys, max(0, kend - key0)) + box - 1) / box;
  return max(0, last - first);
}

// Eight bf16 of a 16-byte word as floats.
__device__ __forceinline__ void bf16x8_to_float(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two E4M3 (satfinite, nearest even; NaN stays NaN), `lo` in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two E4M3 (low 16 bits) as two fp16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
  return r;
}

// 2^x (relative error about 2^-22; 0 at -inf).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Pairs of fp32 in one register pair (one instruction for both).
__device__ __forceinline__ uint64_t f32x2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Natural logarithm of sum * 2^m, -inf for a row that saw no key.
__device__ __forceinline__ float lse_of(float m, float sum) {
  return sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994531f;
}


// ---- values that are not finite ----
// The kernels multiply whole tiles, in which a key that a row does not see has
// weight 0, and 0 * inf is not 0.  They note whether any sum is not finite, and if
// so come here after the last segment.  What a row does see may make it infinite or
// NaN all the same; only rows with such a value at a key that they do not see are done
// once more, key by key.  (A test of each partly visible tile before its product cost
// 5 to 25 % of a chunk; the note costs nothing that shows.)

// This lane's D / 32 neighbouring elements of the cache row at element offset `at`;
// zeros for a row that is not there (-1).
template <int D, bool FP8>
__device__ __forceinline__ void load_part(const void* base, int64_t at, float (&x)[D / 32]) {
  constexpr int kPer = D / 32;
  if (at < 0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = 0.0f;
    return;
  }
  at += (threadIdx.x & 31) * kPer;
  if constexpr (FP8) {
    uint32_t u;
    if constexpr (kPer == 4) u = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(base) + at);
    else u = *reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(base) + at);
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = e4m3_to_float((u >> (8 * i)) & 0xFFu);
  } else {
    const uint32_t* p =
        reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(base) + at);
    uint32_t u[kPer / 2];
    if constexpr (kPer == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      u[0] = v.x;
      u[kPer / 2 - 1] = v.y;
    } else {
      u[0] = *p;
    }
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      x[i] = __uint_as_float(u[i / 2] << 16);
      x[i + 1] = __uint_as_float(u[i / 2] & 0xFFFF0000u);
    }
  }
}

// Dot product of the bf16 row q and the cache row at element offset `at`.
template <int D, bool FP8>
__device__ __forceinline__ float dot_of(const __nv_bfloat16* q, const void* base, int64_t at) {
  float s[2] = {0.0f, 0.0f};
#pragma unroll 4
  for (int d = 0; d < D; d += 16) {
    float x[16], k[16];
    bf16x8_to_float(*reinterpret_cast<const uint4*>(q + d), reinterpret_cast<float (&)[8]>(x[0]));
    bf16x8_to_float(*reinterpret_cast<const uint4*>(q + d + 8),
                    reinterpret_cast<float (&)[8]>(x[8]));
    if constexpr (FP8) {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + at + d);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const uint32_t h = e4m3x2_to_f16x2(w[i >> 2] >> ((i & 2) * 8));
        const float2 f = __half22float2(reinterpret_cast<const __half2&>(h));
        k[i] = f.x;
        k[i + 1] = f.y;
      }
    } else {
      const uint4* p =
          reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at + d);
      bf16x8_to_float(p[0], reinterpret_cast<float (&)[8]>(k[0]));
      bf16x8_to_float(p[1], reinterpret_cast<float (&)[8]>(k[8]));
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i & 1] = fmaf(x[i], k[i], s[i & 1]);
  }
  return s[0] + s[1];
}

// Element offset of a key (below the request's length) of request r and head h; -1 in
// a page out of range, which has been reported and reads as zeros.
__device__ __forceinline__ int64_t place_of(const AttnArgs& a, int r, int h, int key) {
  const int64_t page = a.batch.page_table[r * a.batch.max_pages + (key >> a.cache.page_shift)];
  if (page < 0 || page >= a.cache.num_pages) return -1;
  return page * a.cache.page_stride +
         (key & ((1 << a.cache.page_shift) - 1)) * a.cache.token_stride + h * a.cache.head_stride;
}

// Whether some value of the keys [k0, k1) is not finite, by a warp.
template <int D, bool FP8>
__device__ __forceinline__ bool any_not_finite(const AttnArgs& a, int r, int h, int k0, int k1) {
  constexpr int el = FP8 ? 1 : 2, chunks = D * el / 16;    // 16 bytes each
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int i = lane; i < (k1 - k0) * chunks; i += 32) {
    const int key = k0 + i / chunks;
    const int64_t at = place_of(a, r, h, key);
    if (at < 0) continue;
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.cache.v) +
                                                    at * el + i % chunks * 16);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (FP8)                                             // NaN: 0x7F and a sign
        bad = bad || (w[k] & 0x7Fu) == 0x7Fu || (w[k] & 0x7F00u) == 0x7F00u ||
              (w[k] & 0x7F0000u) == 0x7F0000u || (w[k] & 0x7F000000u) == 0x7F000000u;
      else
        bad = bad || (w[k] & 0x7F80u) == 0x7F80u || (w[k] & 0x7F800000u) == 0x7F800000u;
    }
  }
  return __any_sync(0xFFFFFFFFu, bad);
}

// Query row `row` (of the request's rows for key head h) once more, by one warp
// and from the cache, if an element of it has come out infinite or NaN that is so at
// a hidden key: its sums over the keys of [k0, k1), of which it sees a part.  To the
// output, or to the piece's row `po` relative to the piece's maximum po_ml->x.
template <int D, bool FP8>
__device__ __noinline__ void mend_row(const AttnArgs& a, int r, int h, int row, int k0, int k1,
                                      float* po, const float2* po_ml) {
  constexpr int kPer = D / 32;                             // a lane's elements
  const int lane = threadIdx.x & 31;
  const Request rq = load_request(a.batch, a.cache.page_shift, r, a.status);
  const int tok = a.group(row), pos = rq.pos0 + tok;
  const int head = h * static_cast<int>(a.group.d) + row - tok * static_cast<int>(a.group.d);
  const int lo = min(k1, max(k0, first_key(pos, a.window)));
  const int hi = max(lo, min(k1, pos + 1));
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) +
                       (rq.first + tok) * a.out.token_stride + head * a.out.head_stride +
                       lane * kPer;
  if (po != nullptr) po += lane * kPer;
  uint32_t open = 0;                                       // bits: to be explained
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (!isfinite(po != nullptr ? po[i] : __bfloat162float(out[i]))) open |= 1u << i;
  if (!__any_sync(0xFFFFFFFFu, open != 0)) return;
  // those with a hidden value that is not finite (few keys are hidden: rows of a block
  // lie within 128 positions) ...
  const auto scan = [&](int from, int to, bool nan_only) {
    uint32_t found = 0;
#pragma unroll 4
    for (int key = from; key < to; ++key) {
      float x[kPer];
      load_part<D, FP8>(a.cache.v, place_of(a, r, h, key), x);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (nan_only ? isnan(x[i]) : !isfinite(x[i])) found |= 1u << i;
    }
    return found;
  };
  open &= scan(k0, lo, false) | scan(hi, k1, false);
  if (!__any_sync(0xFFFFFFFFu, open != 0)) return;
  // ... and no NaN at a key that the row does see: that one stays, whatever its weight
  // (looked for where NaN stand side by side, next to the hidden ones)
  open &= ~(scan(lo, min(hi, lo + kAttnTileKeys), true) |
            scan(max(lo, hi - kAttnTileKeys), hi, true));
  if (!__any_sync(0xFFFFFFFFu, open != 0)) return;

  float c = a.scale * 1.4426950408889634f, v_scale = 1.0f;
  if (FP8 && a.cache.k_scale != nullptr) c *= a.cache.k_scale[h];
  if (FP8 && a.cache.v_scale != nullptr) v_scale = a.cache.v_scale[h];
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q.data) +
                           (rq.first + tok) * a.q.token_stride + head * a.q.head_stride;
  float o[kPer] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll 1
  for (int key0 = lo; key0 < hi; key0 += 32) {
    // a lane's key: its place and its weight
    const bool mine = lane < hi - key0;
    const int64_t at = mine ? place_of(a, r, h, key0 + lane) : -1;
    float s = at >= 0 ? dot_of<D, FP8>(q, a.cache.k, at) : 0.0f;
    s = mine ? s * c : -INFINITY;
    float mn = fmaxf(m, s);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, k));
    const float use = mn == -INFINITY ? 0.0f : mn, f = exp2_approx(m - use);
    const float w = exp2_approx(s - use);
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] *= f;
    // the lanes' dimensions
    for (int k = 0; k < 32; k += 8) {
      float wk[8], x[8][kPer];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        wk[j] = __shfl_sync(0xFFFFFFFFu, w, k + j);
        load_part<D, FP8>(a.cache.v, __shfl_sync(0xFFFFFFFFu, at, k + j), x[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = fmaf(wk[j], x[j][i], o[i]);
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, k);
  const float y = po != nullptr ? (m == -INFINITY ? 0.0f : exp2_approx(m - po_ml->x))
                                : (l == 0.0f ? 0.0f : v_scale / l);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (po != nullptr) po[i] = o[i] * y;
    else out[i] = __float2bfloat16_rn(o[i] * y);
  }
}

// The rows [row0, row0 + rows) of a segment, of which some sum may not be finite: one
// of `warps` warps (this one is `warp`).  [kbeg, kend): keys that any of them sees;
// [t0, t1): the tiles that have been taken.  po, po_ml: the piece's first row, or po null.
template <int D, bool FP8>
__device__ __noinline__ void mend_rows(const AttnArgs& a, int r, int h, int row0, int rows,
                                       int kbeg, int kend, int t0, int t1, float* po,
                                       const float2* po_ml, int warp, int warps) {
  const int k0 = max(t0 * kAttnTileKeys, kbeg), k1 = min(t1 * kAttnTileKeys, kend);
  if (rows <= 0 || k1 <= k0) return;
  // keys that one of the rows does not see: before the last row's window, after the
  // first row's position
  const Request rq = load_request(a.batch, a.cache.page_shift, r, a.status);
  const int first = rq.pos0 + a.group(row0), last = rq.pos0 + a.group(row0 + rows - 1);
  const int lo = min(k1, max(k0, first_key(last, a.window)));
  const int hi = min(k1, max(k0, first + 1));
  if (!any_not_finite<D, FP8>(a, r, h, k0, lo) && !any_not_finite<D, FP8>(a, r, h, hi, k1)) return;
  for (int row = warp; row < rows; row += warps)
    mend_row<D, FP8>(a, r, h, row0 + row, k0, k1,
                     po != nullptr ? po + static_cast<int64_t>(row) * D : nullptr, po_ml + row);
}

}  // namespace nvmoe
