// Per-head RMS norm with the rotary embedding, to dense outputs or into a
// paged key / value cache.
//
// Both are one pass over the data: x is read once, its transform written
// once, so the bound is HBM (for few tokens, the launch and two dependent
// round trips to memory).  With rstd = rsqrt(mean x^2 + eps) a pair (a, b) of
// a head turns into
//   a' = rstd * (a * (w_a cos) - b * (w_b sin)),
//   b' = rstd * (b * (w_b cos) + a * (w_a sin)),
// and the four products in brackets depend only on the token and on q or k.  A
// group of head_dim / 8 lanes keeps them in registers and runs over up to
// HEADS heads of q, of k or of v of one token, whose loads are all in flight
// at once.  A lane holds whole pairs, so nothing passes between lanes but the
// sum of squares: four elements of each half of the rotated part (8-byte
// loads), or eight neighbours where pairs are neighbours or nothing is turned.
#include "attn.cuh"

namespace nvmoe {
namespace {

constexpr int kThreads = 128;
// Many rows: eight heads a group and 64 registers a thread; into the cache
// four and 48, which hides the longer chain of loads (request, length, page,
// rotation) before a row can be stored.  Measured, 4096 tokens of 56 + 8 heads
// of 128 and 21 k tokens into an E4M3 cache: 8 heads of 64 registers 29.8 us
// and 188 us, 4 of 48 32.4 and 162, 8 of 90 registers 31.3 and 264.
// (With its start over the end of the kernel before, a launch takes 27.4 and 176:
// 5.0 and 4.3 TB/s; 160 of the latter without the divisions by the scales.  Into the
// cache instructions bound it (76 % of the issue slots): each group finds its request,
// page and rotation anew, and at 48 registers a thread spills 120 to 148 bytes and
// reads 244 to 256 back.  Groups that keep what they have found for 8 or 16 heads in
// rounds of 4 took 187 to 190 us, before the divisions.)
// Below kWideRows head rows two heads a group spread few tokens wider (into the cache
// at the same 48 registers, with 52 to 80 bytes of spills).
constexpr int64_t kWideRows = 16384;
template <bool APPEND>
constexpr int kWideHeads = APPEND ? 4 : 8;
template <bool APPEND>
constexpr int kMinBlocks = APPEND ? 10 : 8;

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

// The request that holds row t: the last r with q_start[r] <= t (so empty
// requests are passed over); -1 for a row of no request.
__device__ __forceinline__ int request_of(const BatchView& b, uint32_t row) {
  const int64_t t = row;
  if (t >= b.q_start[b.batch] || t < b.q_start[0]) return -1;
  int lo = 0, hi = b.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.q_start[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
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

// APPEND: k and v go to the cache.  PAIRS: neighbours form the pairs.
template <int D, int HEADS, bool APPEND, bool PAIRS>
__global__ void __launch_bounds__(kThreads, kMinBlocks<APPEND>)
head_transform_kernel(const RopeArgs a) {
  pdl_wait();                                         // for what came before
  constexpr int kLanes = D / 8;                       // lanes of a group
  const int sub = threadIdx.x & (kLanes - 1);
  const uint32_t mask = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
  const uint32_t item = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const uint32_t t = item / static_cast<uint32_t>(a.chunks);
  if (t >= a.T) return;
  int chunk = static_cast<int>(item - t * a.chunks);
  int kind = 0;                                       // 0: q, 1: k, 2: v
  if (chunk >= a.q_chunks) {
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
  const int half = a.tr.rotary_dim / 2;
  const bool inside = sub * 8 < a.tr.rotary_dim;      // of the rotated part
  const int i0 = !PAIRS && inside ? sub * 4 : sub * 8;
  const int i1 = !PAIRS && inside ? half + sub * 4 : sub * 8 + 4;

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
    const int r = request_of(a.batch, t);
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

  // The products of weights, cosines and sines.  Halves: x_0 = elements i0.. ,
  // x_1 = elements i1.. are the a and b of four pairs, y_0 = x_0 P_0 + x_1 Q_0,
  // y_1 = x_1 P_1 + x_0 Q_1.  Neighbours: y = x P + x' Q with x' the elements
  // exchanged within their pairs.
  const __nv_bfloat16* weight = kind == 0 ? a.tr.q_weight : a.tr.k_weight;
  const bool plain = APPEND && kind == 2;
  const bool turned = !plain && inside;               // (rotary_dim is 0 without rope)
  uint64_t P[2][2], Q[2][2];
  {
    const uint64_t one = f32x2(1.0f, 1.0f);
    uint64_t w[2][2] = {{one, one}, {one, one}};
    if (!plain && weight != nullptr) {
      bf16x4_to_f32x2(*reinterpret_cast<const uint2*>(weight + i0), w[0]);
      bf16x4_to_f32x2(*reinterpret_cast<const uint2*>(weight + i1), w[1]);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        P[s][j] = w[s][j];
        Q[s][j] = 0;
      }
    if (turned) {
      const float* row = a.tr.rope + pos * a.tr.rotary_dim + sub * 4;
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

#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    if (i >= heads) break;
    const int h = h0 + i;
    uint64_t x[2][2];
    bf16x4_to_f32x2(raw[i][0], x[0]);
    bf16x4_to_f32x2(raw[i][1], x[1]);
    if (!plain) {
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
      if (weight != nullptr) {
        uint64_t sq = mul_f32x2(x[0][0], x[0][0]);
        sq = fma_f32x2(x[0][1], x[0][1], sq);
        sq = fma_f32x2(x[1][0], x[1][0], sq);
        sq = fma_f32x2(x[1][1], x[1][1], sq);
        float s0, s1;
        f32x2_split(sq, s0, s1);
        float sum = s0 + s1;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
        const float rstd = rsqrtf(fmaf(sum, 1.0f / D, a.tr.eps));
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
    if (APPEND && kind != 0) {
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

template <int D, bool APPEND, bool PAIRS>
cudaError_t launch_d(RopeArgs a, cudaStream_t stream) {
  constexpr int kGroups = kThreads / (D / 8);
  const auto go = [&](auto kernel, int per) {
    a.q_chunks = static_cast<int>(ceil_div(a.q.heads, per));
    a.kv_chunks = static_cast<int>(ceil_div(a.k.heads, per));
    a.chunks = a.q_chunks + (APPEND ? 2 : 1) * a.kv_chunks;
    const int64_t blocks = ceil_div(a.T * a.chunks, kGroups);
    // its start overlaps the end of the kernel before
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
  };
  const int64_t heads = a.q.heads + a.k.heads + a.v.heads;
  constexpr int kWide = kWideHeads<APPEND>;
  return a.T * heads >= kWideRows ? go(head_transform_kernel<D, kWide, APPEND, PAIRS>, kWide)
                                  : go(head_transform_kernel<D, 2, APPEND, PAIRS>, 2);
}

template <bool APPEND>
cudaError_t launch(const RopeArgs& a, int head_dim, cudaStream_t stream) {
  if (a.tr.interleaved)
    return head_dim == 128 ? launch_d<128, APPEND, true>(a, stream)
                           : launch_d<64, APPEND, true>(a, stream);
  return head_dim == 128 ? launch_d<128, APPEND, false>(a, stream)
                         : launch_d<64, APPEND, false>(a, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const HeadRows& q, const HeadRows& k, int64_t T, int head_dim,
                                const int32_t* positions, const HeadTransform& tr,
                                const HeadRows& q_out, const HeadRows& k_out, int* status,
                                cudaStream_t stream) {
  RopeArgs a{};
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.tr = tr;
  a.positions = positions;
  a.T = T;
  a.status = status;
  return launch<false>(a, head_dim, stream);
}

cudaError_t launch_kv_append(const HeadRows& q, const HeadRows& k, const HeadRows& v,
                             const KvCacheView& cache, const BatchView& batch,
                             const HeadTransform& tr, const HeadRows& q_out, int* status,
                             cudaStream_t stream) {
  RopeArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.cache = cache;
  a.batch = batch;
  a.tr = tr;
  a.T = batch.tokens;
  a.status = status;
  return launch<true>(a, cache.head_dim, stream);
}

}  // namespace nvmoe
