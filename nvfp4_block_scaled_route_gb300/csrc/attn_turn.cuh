// Norm and rotation of head rows, shared by the kernels that write them densely or
// into a cache with a scale per head (attn_rope.cu) and into pages with scales of
// their own (attn_append.cu).
#pragma once

#include "attn.cuh"

namespace nvmoe {

struct RopeArgs {
  HeadRows q, k, v;           // v.heads = 0: no cache
  HeadRows q_out, k_out;
  KvCacheView cache;
  BatchView batch;
  HeadTransform tr;
  const int32_t* positions;
  int64_t T;
  int q_chunks, kv_chunks;    // chunks of HEADS heads: q's, k's (and as many of v)
  int chunks;                 // of a token
  int* status;
};

// The last i of [0, n) with below(i), which holds up to there and not after (0 if it
// holds nowhere), by the lanes of `mask`: LANES neighbours, of which this is number `sub`,
// probe at a time (each round is a load that the next one waits for).
template <int LANES, typename F>
__device__ __forceinline__ int last_below(int n, int sub, uint32_t mask, F below) {
  int lo = 0;
  while (n > 1) {
    const int step = (n + LANES - 1) / LANES, at = sub * step;
    const uint32_t yes = (__ballot_sync(mask, at < n && below(lo + at)) & mask) >> (__ffs(mask) - 1);
    const int skip = (31 - __clz(yes | 1u)) * step;
    n = min(step, n - skip);
    lo += skip;
  }
  return lo;
}

// The request that holds row t: the last r with q_start[r] <= t (so empty
// requests are passed over); -1 for a row of no request.
template <int LANES>
__device__ __forceinline__ int request_of(const BatchView& b, uint32_t row, int sub,
                                          uint32_t mask) {
  const int64_t t = row;
  const int first = b.q_start[0], end = b.q_start[b.batch];
  const int r = last_below<LANES>(b.batch, sub, mask, [&](int i) { return b.q_start[i] <= t; });
  return t >= end || t < first ? -1 : r;
}

// Four bf16 (8 bytes) as two pairs of floats.
__device__ __forceinline__ void bf16x4_to_f32x2(const uint2& u, uint64_t (&x)[2]) {
  x[0] = f32x2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u));
  x[1] = f32x2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ uint2 f32x2_to_bf16x4(const uint64_t (&x)[2]) {
  float a, b, c, d;
  f32x2_split(x[0], a, b);
  f32x2_split(x[1], c, d);
  return make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

// A lane's part of the norm and rotation: eight elements of a head of D, with the
// products of weights, cosines and sines of one token.  Halves: x_0 = elements
// i0 .. i0+3, x_1 = elements i1 .. i1+3 are the a and b of four pairs,
// y_0 = x_0 P_0 + x_1 Q_0, y_1 = x_1 P_1 + x_0 Q_1.  Neighbours (PAIRS):
// y = x P + x' Q with x' the elements exchanged within their pairs.
template <int D, bool PAIRS>
struct HeadTurn {
  static constexpr int kLanes = D / 8;                  // of a group
  uint64_t P[2][2], Q[2][2];

  // The elements that lane `sub` of a group holds.
  static __device__ __forceinline__ void places(int sub, int rotary_dim, int& i0, int& i1) {
    const bool inside = sub * 8 < rotary_dim;           // of the rotated part
    i0 = !PAIRS && inside ? sub * 4 : sub * 8;
    i1 = !PAIRS && inside ? rotary_dim / 2 + sub * 4 : sub * 8 + 4;
  }

  // The weights of this lane's elements, ones without.
  static __device__ __forceinline__ void weights(const __nv_bfloat16* weight, int i0, int i1,
                                                 uint64_t (&w)[2][2]) {
    w[0][0] = w[0][1] = w[1][0] = w[1][1] = f32x2(1.0f, 1.0f);
    if (weight != nullptr) {
      bf16x4_to_f32x2(*reinterpret_cast<const uint2*>(weight + i0), w[0]);
      bf16x4_to_f32x2(*reinterpret_cast<const uint2*>(weight + i1), w[1]);
    }
  }

  // turned: these elements belong to the rotated part (of rows that do not stay as they are).
  __device__ __forceinline__ void load(const HeadTransform& tr, const uint64_t (&w)[2][2],
                                       bool turned, int sub, int64_t pos) {
    const int half = tr.rotary_dim / 2;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        P[s][j] = w[s][j];
        Q[s][j] = 0;
      }
    if (turned) {
      const float* row = tr.rope + pos * tr.rotary_dim + sub * 4;
      const float4 c = *reinterpret_cast<const float4*>(row);
      const float4 s = *reinterpret_cast<const float4*>(row + half);
      if (PAIRS) {
        const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float w0, w1;
          f32x2_split(w[k >> 1][k & 1], w0, w1);
          P[k >> 1][k & 1] = f32x2(w0 * cv[k], w1 * cv[k]);
          Q[k >> 1][k & 1] = f32x2(-w1 * sv[k], w0 * sv[k]);
        }
      } else {
        const uint64_t cc[2] = {f32x2(c.x, c.y), f32x2(c.z, c.w)};
        const uint64_t ss[2] = {f32x2(s.x, s.y), f32x2(s.z, s.w)};
        const uint64_t minus = f32x2(-1.0f, -1.0f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          P[0][j] = mul_f32x2(w[0][j], cc[j]);
          P[1][j] = mul_f32x2(w[1][j], cc[j]);
          Q[0][j] = mul_f32x2(mul_f32x2(w[1][j], ss[j]), minus);
          Q[1][j] = mul_f32x2(w[0][j], ss[j]);
        }
      }
    }
  }

  // x to its transform; `mask`: the lanes of the group.
  __device__ __forceinline__ void apply(uint64_t (&x)[2][2], bool turned, bool normed, float eps,
                                        uint32_t mask) const {
    uint64_t y[2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        y[s][j] = mul_f32x2(x[s][j], P[s][j]);
        // (not turned: no product with a partner, which may be infinite)
        if (turned) {
          uint64_t partner = x[s ^ 1][j];
          if (PAIRS) {
            float x0, x1;
            f32x2_split(x[s][j], x0, x1);
            partner = f32x2(x1, x0);
          }
          y[s][j] = fma_f32x2(partner, Q[s][j], y[s][j]);
        }
      }
    if (normed) {
      uint64_t sq = mul_f32x2(x[0][0], x[0][0]);
      sq = fma_f32x2(x[0][1], x[0][1], sq);
      sq = fma_f32x2(x[1][0], x[1][0], sq);
      sq = fma_f32x2(x[1][1], x[1][1], sq);
      float s0, s1;
      f32x2_split(sq, s0, s1);
      float sum = s0 + s1;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
      const float rstd = rsqrtf(fmaf(sum, 1.0f / D, eps));
      const uint64_t r2 = f32x2(rstd, rstd);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j) y[s][j] = mul_f32x2(y[s][j], r2);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j) x[s][j] = y[s][j];
  }
};

// Up to HEADS heads of q, of k or of v of one token by a group of D / 8 lanes.
// APPEND: k and v go to the cache (KV: if they are among the items at all).  PAIRS:
// neighbours form the pairs.
template <int D, int HEADS, bool APPEND, bool PAIRS, bool KV = true>
__device__ __forceinline__ void transform_heads(const RopeArgs& a, uint32_t item) {
  constexpr int kLanes = D / 8;                       // lanes of a group
  const int sub = threadIdx.x & (kLanes - 1);
  const uint32_t mask = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
  const uint32_t t = item / static_cast<uint32_t>(a.chunks);
  if (t >= a.T) return;
  int chunk = static_cast<int>(item - t * a.chunks);
  int kind = 0;                                       // 0: q, 1: k, 2: v
  if (KV && chunk >= a.q_chunks) {
    chunk -= a.q_chunks;
    kind = 1;
    if (APPEND && chunk >= a.kv_chunks) {
      chunk -= a.kv_chunks;
      kind = 2;
    }
  }
  const HeadRows& src = kind == 0 ? a.q : (APPEND && kind == 2 ? a.v : a.k);
  const int h0 = chunk * HEADS;
  const int heads = min(HEADS, src.heads - h0);
  // this lane's elements: i0 .. i0+3 and i1 .. i1+3
  int i0, i1;
  HeadTurn<D, PAIRS>::places(sub, a.tr.rotary_dim, i0, i1);

  // the rows first: their loads do not depend on the position
  uint2 raw[HEADS][2];
  {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(src.data) +
                             t * src.token_stride + h0 * src.head_stride;
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      if (i < heads) {
        raw[i][0] = *reinterpret_cast<const uint2*>(p + i0);
        raw[i][1] = *reinterpret_cast<const uint2*>(p + i1);
      }
      p += src.head_stride;
    }
  }

  int64_t pos = 0;
  int64_t slot = 0;                                   // element offset of (page, offset)
  if (APPEND) {
    const int r = request_of<kLanes>(a.batch, t, sub, mask);
    if (r < 0) return;
    pos = static_cast<int64_t>(a.batch.kv_len[r]) - a.batch.q_start[r + 1] + t;
    const int64_t page_i = pos >> a.cache.page_shift;
    bool ok = pos >= 0 && page_i < a.batch.max_pages &&
              (a.tr.rope == nullptr || pos < a.tr.rope_positions);
    if (ok) {
      const int64_t page = a.batch.page_table[r * a.batch.max_pages + page_i];
      ok = page >= 0 && page < a.cache.num_pages;
      slot = page * a.cache.page_stride +
             (pos & ((int64_t{1} << a.cache.page_shift) - 1)) * a.cache.token_stride;
    }
    if (!ok) {
      record_status(a.status, kErrBadIndex);
      return;
    }
  } else if (a.tr.rope != nullptr) {
    pos = a.positions[t];
    if (pos < 0 || pos >= a.tr.rope_positions) {
      record_status(a.status, kErrBadIndex);
      return;
    }
  }

  const __nv_bfloat16* weight = kind == 0 ? a.tr.q_weight : a.tr.k_weight;
  const bool plain = APPEND && kind == 2;
  // (Whether this lane's elements are turned: known before the weights are asked for into a
  // cache, else behind them.  The compiler orders loads and spills by it: prompts of 16384
  // tokens into a bf16 cache 126 us, the other way 131; 4096 tokens to dense outputs 27.4,
  // the other way 28.1.)
  bool turned = APPEND && !plain && sub * 8 < a.tr.rotary_dim;   // (0 without rope)
  HeadTurn<D, PAIRS> turn;
  uint64_t w[2][2];
  HeadTurn<D, PAIRS>::weights(plain ? nullptr : weight, i0, i1, w);
  if (!APPEND) turned = sub * 8 < a.tr.rotary_dim;
  turn.load(a.tr, w, turned, sub, pos);

#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    if (i >= heads) break;
    const int h = h0 + i;
    uint64_t x[2][2];
    bf16x4_to_f32x2(raw[i][0], x[0]);
    bf16x4_to_f32x2(raw[i][1], x[1]);
    if (!plain) turn.apply(x, turned, weight != nullptr, a.tr.eps, mask);
    if (APPEND && KV && kind != 0) {
      const int64_t at = slot + h * a.cache.head_stride;
      void* dst = plain ? a.cache.v : a.cache.k;
      if (a.cache.fp8) {
        const float* sc = plain ? a.cache.v_scale : a.cache.k_scale;
        // (the quotient, not a product with the reciprocal: that one rounds to the
        // other side at some ties, and is infinite for a scale below 2^-128)
        const float by = sc != nullptr ? sc[h] : 1.0f;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float z[4];
          f32x2_split(x[s][0], z[0], z[1]);
          f32x2_split(x[s][1], z[2], z[3]);
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(dst) + at + (s == 0 ? i0 : i1)) =
              pack_e4m3x2(z[0] / by, z[1] / by) | (pack_e4m3x2(z[2] / by, z[3] / by) << 16);
        }
      } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(dst) + at;
        *reinterpret_cast<uint2*>(o + i0) = plain ? raw[i][0] : f32x2_to_bf16x4(x[0]);
        *reinterpret_cast<uint2*>(o + i1) = plain ? raw[i][1] : f32x2_to_bf16x4(x[1]);
      }
    } else {
      const HeadRows& dst = kind == 0 ? a.q_out : a.k_out;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(dst.data) + t * dst.token_stride +
                         h * dst.head_stride;
      *reinterpret_cast<uint2*>(o + i0) = f32x2_to_bf16x4(x[0]);
      *reinterpret_cast<uint2*>(o + i1) = f32x2_to_bf16x4(x[1]);
    }
  }
}

}  // namespace nvmoe
