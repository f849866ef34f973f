// Attention of each request's new tokens over its paged cache.
//
// One warp per (token, query head): the keys one after the other, the dot
// product over the lanes, and the running maximum m and sum l of the softmax
//   m' = max(m, s),  l' = l e^(m - m') + e^(s - m'),  o' = o e^(m - m') + e^(s - m') v.
#include "attn.cuh"

namespace nvmoe {
namespace {

constexpr int kThreads = 128;

template <int D, bool FP8>
__device__ __forceinline__ void load_row(const void* base, int64_t at, int lane,
                                         float (&x)[D / 32]) {
  constexpr int N = D / 32;
  if (FP8) {
    const uint8_t* p = static_cast<const uint8_t*>(base) + at + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = e4m3_to_float(p[i]);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) attention_kernel(const AttnArgs a) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int hq = a.q.heads;
  const int64_t t = w / hq;
  const int h = static_cast<int>(w - t * hq);
  if (t >= a.batch.tokens) return;
  const int32_t* qs = a.batch.q_start;
  if (t < qs[0] || t >= qs[a.batch.batch]) return;
  int lo = 0, hi = a.batch.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (qs[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const Request rq = load_request(a.batch, a.cache.page_shift, lo, a.status);
  const int i = static_cast<int>(t - rq.first);
  if (i >= rq.n) return;
  const int pos = rq.pos0 + i;
  const int end = min(pos + 1, rq.len);
  const int begin = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const int hk = h / (hq / a.cache.heads);

  float q[N], o[N];
  load_row<D, false>(a.q.data, t * a.q.token_stride + h * a.q.head_stride, lane, q);
  float scale = a.scale;
  if (FP8 && a.cache.k_scale != nullptr) scale *= a.cache.k_scale[hk];
#pragma unroll
  for (int j = 0; j < N; ++j) o[j] = 0.0f;
  float m = -INFINITY, l = 0.0f;
  for (int k = begin; k < end; ++k) {
    const int64_t page = a.batch.page_table[lo * a.batch.max_pages + (k >> a.cache.page_shift)];
    const bool ok = page >= 0 && page < a.cache.num_pages;
    if (!ok) record_status(a.status, kErrBadIndex);
    const int64_t at = page * a.cache.page_stride +
                       (k & ((1 << a.cache.page_shift) - 1)) * a.cache.token_stride +
                       hk * a.cache.head_stride;
    float x[N], v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = v[j] = 0.0f;
    if (ok) {
      load_row<D, FP8>(a.cache.k, at, lane, x);
      load_row<D, FP8>(a.cache.v, at, lane, v);
    }
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) s = fmaf(q[j], x[j], s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= scale;
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.0f : expf(m - mn), p = expf(s - mn);
    m = mn;
    l = fmaf(l, f, p);
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = fmaf(o[j], f, p * v[j]);
  }
  float inv = l > 0.0f ? 1.0f / l : 0.0f;
  if (FP8 && a.cache.v_scale != nullptr) inv *= a.cache.v_scale[hk];
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) + t * a.out.token_stride +
                       h * a.out.head_stride + lane * N;
#pragma unroll
  for (int j = 0; j < N; ++j) out[j] = __float2bfloat16_rn(o[j] * inv);
  if (a.lse != nullptr && lane == 0) a.lse[t * hq + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

// Joins the pieces of the segments that were cut between CTAs: block x takes
// the segment that CTA x begins, a thread four dimensions of a row.  With the
// largest maximum M, o = sum_c 2^(m_c - M) o_c and l likewise, in the order of
// the CTAs, so results do not depend on timing.
template <int D>
__global__ void __launch_bounds__(256) attn_combine_kernel(const AttnArgs a) {
  pdl_wait();
  const AttnPiece p = a.pieces[blockIdx.x];
  const int item = blockIdx.y * 256 + threadIdx.x;
  const int row = item / (D / 4), d = (item % (D / 4)) * 4;
  if (row >= p.rows) return;
  const int G = gridDim.x;
  float top = -INFINITY;
  const auto slot_of = [&](int c) { return 2 * static_cast<int64_t>(c) + (c == blockIdx.x); };
  const auto has = [&](int c) { return p.total * c / G < p.total * (c + 1) / G; };
  for (int c = blockIdx.x; c <= p.last; ++c)
    if (has(c)) top = fmaxf(top, a.piece_ml[slot_of(c) * a.piece_rows + row].x);
  const float use = top == -INFINITY ? 0.0f : top;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float sum = 0.0f;
#pragma unroll 4
  for (int c = blockIdx.x; c <= p.last; ++c) {
    if (!has(c)) continue;
    const int64_t at = slot_of(c) * a.piece_rows + row;
    const float2 ml = a.piece_ml[at];
    const float4 x = *reinterpret_cast<const float4*>(a.piece_o + at * D + d);
    const float f = exp2_approx(ml.x - use);
    sum = fmaf(f, ml.y, sum);
    o.x = fmaf(f, x.x, o.x);
    o.y = fmaf(f, x.y, o.y);
    o.z = fmaf(f, x.z, o.z);
    o.w = fmaf(f, x.w, o.w);
  }
  const int group = a.q.heads / a.cache.heads;
  const int tok = (p.row0 + row) / group;
  const int64_t t = p.first + tok;
  const int head = p.head * group + p.row0 + row - tok * group;
  float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (a.cache.v_scale != nullptr) inv *= a.cache.v_scale[p.head];
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out.data) + t * a.out.token_stride +
                            head * a.out.head_stride + d) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (d == 0 && a.lse != nullptr) a.lse[t * a.q.heads + head] = lse_of(top, sum);
}

}  // namespace

cudaError_t launch_paged_attention(const AttnArgs& a, cudaStream_t stream) {
  const unsigned blocks =
      static_cast<unsigned>(ceil_div(a.batch.tokens * a.q.heads, kThreads / 32));
  const bool wide = a.cache.head_dim == 128;
  if (a.cache.fp8) {
    if (wide) attention_kernel<128, true><<<blocks, kThreads, 0, stream>>>(a);
    else attention_kernel<64, true><<<blocks, kThreads, 0, stream>>>(a);
  } else {
    if (wide) attention_kernel<128, false><<<blocks, kThreads, 0, stream>>>(a);
    else attention_kernel<64, false><<<blocks, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_attn_combine(const AttnArgs& a, int grid, cudaStream_t stream) {
  // launched while the attention kernel runs; it waits for that kernel's end
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, static_cast<unsigned>(
                               ceil_div(int64_t{a.piece_rows} * a.cache.head_dim / 4, 256)));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.cache.head_dim == 128 ? cudaLaunchKernelEx(&cfg, attn_combine_kernel<128>, a)
                                 : cudaLaunchKernelEx(&cfg, attn_combine_kernel<64>, a);
}

}  // namespace nvmoe
