// Per-head RMS norm with the rotary embedding, to dense outputs or into a
// paged key / value cache.
//
// Both are one pass over the data: x is read once, its transform written
// once, so the bound is HBM (for few tokens, the launch and two dependent
// round trips to memory).  With rstd = rsqrt(mean x^2 + eps) the transform of
// element i with rotation partner j is
//   out_i = rstd * (x_i * A_i + x_j * B_i),  A_i = w_i cos, B_i = -+ w_j sin
// (A_i = w_i, B_i = 0 past rotary_dim), and A and B depend only on the token
// and on q or k.  A group of head_dim / 8 lanes (16-byte loads) therefore
// keeps A and B in registers and runs over several heads of one token; the
// partner's eight elements come from another lane of the group by four
// shuffles of the packed bf16 words, or from the same lane (interleaved).
#include "attn.cuh"

namespace nvmoe {
namespace {

constexpr int kThreads = 256;

struct RopeArgs {
  HeadRows q, k, v;           // v.heads = 0: no cache
  HeadRows q_out, k_out;
  KvCacheView cache;
  BatchView batch;
  HeadTransform tr;
  const int32_t* positions;
  int64_t T;
  int chunks;                 // head chunks per token
  int* status;
};

// The request that holds row t: the last r with q_start[r] <= t (so empty
// requests are passed over); -1 for a row of no request.
__device__ __forceinline__ int request_of(const BatchView& b, int64_t t) {
  if (t >= b.q_start[b.batch] || t < b.q_start[0]) return -1;
  int lo = 0, hi = b.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.q_start[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0];
  const float4 b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// HEADS heads of one token per group, loaded together.  APPEND: k and v go to
// the cache.
template <int D, int HEADS, bool APPEND>
__global__ void __launch_bounds__(kThreads) head_transform_kernel(const RopeArgs a) {
  constexpr int kLanes = D / 8;                       // lanes of a group
  const int sub = threadIdx.x & (kLanes - 1);
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / kLanes) +
                       threadIdx.x / kLanes;
  const int heads = a.q.heads + a.k.heads + (APPEND ? a.v.heads : 0);
  int64_t t = item / a.chunks;
  const int h0 = static_cast<int>(item - t * a.chunks) * HEADS;
  // lanes of groups past the end stay for the shuffles of their warp
  bool live = t < a.T && h0 < heads;
  if (!live) t = 0;

  // the rows first: their loads do not depend on the position
  uint4 raw[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = h0 + i;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (live && h < heads) {
      const HeadRows& src = h < a.q.heads ? a.q : (h < a.q.heads + a.k.heads ? a.k : a.v);
      const int hs = h < a.q.heads ? h
                     : (h < a.q.heads + a.k.heads ? h - a.q.heads : h - a.q.heads - a.k.heads);
      raw[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(src.data) +
                                               t * src.token_stride + hs * src.head_stride +
                                               sub * 8);
    }
  }

  int64_t pos = 0;
  int64_t slot = 0;                                   // element offset of (page, offset)
  if (live) {
    if (APPEND) {
      const int r = request_of(a.batch, t);
      bool ok = false;
      if (r >= 0) {
        pos = static_cast<int64_t>(a.batch.kv_len[r]) - a.batch.q_start[r + 1] + t;
        const int64_t page_i = pos >> a.cache.page_shift;
        if (pos >= 0 && page_i < a.batch.max_pages) {
          const int64_t page = a.batch.page_table[r * a.batch.max_pages + page_i];
          ok = page >= 0 && page < a.cache.num_pages;
          slot = page * a.cache.page_stride +
                 (pos & ((int64_t{1} << a.cache.page_shift) - 1)) * a.cache.token_stride;
        }
        if (a.tr.rope != nullptr && pos >= a.tr.rope_positions) ok = false;
        if (!ok) record_status(a.status, kErrBadIndex);
      }
      live = ok;
    } else if (a.tr.rope != nullptr) {
      pos = a.positions[t];
      if (pos < 0 || pos >= a.tr.rope_positions) {
        record_status(a.status, kErrBadIndex);
        live = false;
      }
    }
  }
  if (!live) pos = 0;

  // cosines and sines of this lane's elements; `from`: the lane of the group
  // that holds the partners
  const int e0 = sub * 8;
  const int half = a.tr.rotary_dim / 2;
  const bool turned = a.tr.rope != nullptr && e0 < a.tr.rotary_dim;
  int from = sub;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
  }
  if (turned) {
    const float* row = a.tr.rope + pos * a.tr.rotary_dim;
    if (a.tr.interleaved) {
      const float4 cc = *reinterpret_cast<const float4*>(row + e0 / 2);
      const float4 ss = *reinterpret_cast<const float4*>(row + half + e0 / 2);
      const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = cv[i / 2];
        s[i] = (i & 1) ? sv[i / 2] : -sv[i / 2];
      }
    } else {
      const bool second = e0 >= half;
      const int f = second ? e0 - half : e0;
      from = second ? sub - half / 8 : sub + half / 8;
      load8(row + f, c);
      load8(row + half + f, s);
      if (!second)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = -s[i];
    }
  }
  const int from_lane = (threadIdx.x & 31 & ~(kLanes - 1)) + from;

  float A[8], B[8];
  int kind = -1;                                      // 0: q, 1: k
  const __nv_bfloat16* weight = nullptr;
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = h0 + i;
    const bool is_v = APPEND && h >= a.q.heads + a.k.heads;
    const int want = h < a.q.heads ? 0 : 1;
    if (want != kind) {
      kind = want;
      weight = kind == 0 ? a.tr.q_weight : a.tr.k_weight;
      float w[8], wp[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = wp[j] = 1.0f;
      if (weight != nullptr) {
        bf16x8_to_float(*reinterpret_cast<const uint4*>(weight + e0), w);
        bf16x8_to_float(*reinterpret_cast<const uint4*>(weight + from * 8), wp);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        A[j] = w[j] * c[j];
        B[j] = (a.tr.interleaved ? wp[j ^ 1] : wp[j]) * s[j];
      }
    }
    float x[8], xp[8];
    bf16x8_to_float(raw[i], x);
    uint4 other;
    other.x = __shfl_sync(0xFFFFFFFFu, raw[i].x, from_lane);
    other.y = __shfl_sync(0xFFFFFFFFu, raw[i].y, from_lane);
    other.z = __shfl_sync(0xFFFFFFFFu, raw[i].z, from_lane);
    other.w = __shfl_sync(0xFFFFFFFFu, raw[i].w, from_lane);
    bf16x8_to_float(other, xp);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (!live || h >= heads) continue;
    float y[8];
    if (is_v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = x[j];
    } else {
      const float rstd = weight != nullptr ? rsqrtf(sum * (1.0f / D) + a.tr.eps) : 1.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // (not turned: no product with the partner, which may be infinite)
        const float p = a.tr.interleaved ? xp[j ^ 1] : xp[j];
        y[j] = rstd * (turned ? fmaf(p, B[j], x[j] * A[j]) : x[j] * A[j]);
      }
    }
    if (APPEND && h >= a.q.heads) {
      const int hk = is_v ? h - a.q.heads - a.k.heads : h - a.q.heads;
      const int64_t at = slot + hk * a.cache.head_stride + e0;
      void* dst = is_v ? a.cache.v : a.cache.k;
      if (a.cache.fp8) {
        const float* sc = is_v ? a.cache.v_scale : a.cache.k_scale;
        const float d = sc != nullptr ? sc[hk] : 1.0f;
        uint2 o;
        o.x = pack_e4m3x2(y[0] / d, y[1] / d) | (pack_e4m3x2(y[2] / d, y[3] / d) << 16);
        o.y = pack_e4m3x2(y[4] / d, y[5] / d) | (pack_e4m3x2(y[6] / d, y[7] / d) << 16);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(dst) + at) = o;
      } else {
        uint4 o = raw[i];
        if (!is_v)
          o = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                         pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst) + at) = o;
      }
    } else {
      const HeadRows& dst = h < a.q.heads ? a.q_out : a.k_out;
      const int hd = h < a.q.heads ? h : h - a.q.heads;
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst.data) + t * dst.token_stride +
                                hd * dst.head_stride + e0) =
          make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                     pack_bf16x2(y[6], y[7]));
    }
  }
}

template <int D, bool APPEND>
cudaError_t launch_d(RopeArgs a, cudaStream_t stream) {
  const int heads = a.q.heads + a.k.heads + a.v.heads;
  constexpr int kGroups = kThreads / (D / 8);
  const auto go = [&](auto kernel, int per) {
    a.chunks = static_cast<int>(ceil_div(heads, per));
    const int64_t blocks = ceil_div(a.T * a.chunks, kGroups);
    kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  };
  return go(head_transform_kernel<D, 4, APPEND>, 4);
}

template <bool APPEND>
cudaError_t launch(const RopeArgs& a, int head_dim, cudaStream_t stream) {
  return head_dim == 128 ? launch_d<128, APPEND>(a, stream) : launch_d<64, APPEND>(a, stream);
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
