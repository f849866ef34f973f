// Joining the pieces of paged attention (attn_rows.cu, attn_keys.cu, attn_chunk.cu).
#include "attn.cuh"

namespace nvmoe {
namespace {

// Joins the pieces of the segments that were cut between CTAs: block x takes
// the segment that CTA x begins, a thread four dimensions of a row.  With the
// largest maximum M, o = sum_c 2^(m_c - M) o_c and l likewise, in the order of
// the CTAs, so results do not depend on timing.  Its data fit the L2; it is bound
// by latency (2 us of the 8 of one request of 1000 keys, whose launch overlaps
// the pieces' kernel).
template <int D>
__global__ void __launch_bounds__(256) attn_combine_kernel(const AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  const AttnPiece p = a.pieces[blockIdx.x];
  const int item = blockIdx.y * 256 + threadIdx.x;
  const int row = item / (D / 4), d = (item % (D / 4)) * 4;
  if (row >= p.rows) return;
  // piece i: the CTA that begins the segment holds it in its slot 1, the
  // others in their slot 0
  const int n = p.last - static_cast<int>(blockIdx.x) + 1;
  const auto at = [&](int i) {
    return (2 * (static_cast<int64_t>(blockIdx.x) + i) + (i == 0)) * a.piece_rows + row;
  };
  // What bounds this kernel is the latency of its loads: a lane of the row's takes the
  // maximum and sum of a piece, and kBatch pieces' rows are on their way meanwhile.
  constexpr int kLanes = D / 4, kBatch = 8;
  const int sub = threadIdx.x & (kLanes - 1);
  const uint32_t lanes = (kLanes == 32 ? 0xFFFFFFFFu : (1u << (kLanes & 31)) - 1u)
                         << (threadIdx.x & 31 & ~(kLanes - 1));
  const auto load_ml = [&](int i) {
    return i < n ? a.piece_ml[at(i)] : make_float2(-INFINITY, 0.0f);
  };
  const auto load_o = [&](int i) {
    return i < n ? *reinterpret_cast<const float4*>(a.piece_o + at(i) * D + d)
                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  float2 ml = load_ml(sub);
  float4 x[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) x[i] = load_o(i);
  float top = ml.x;
  for (int i = sub + kLanes; i < n; i += kLanes) top = fmaxf(top, load_ml(i).x);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(lanes, top, o));
  const float use = top == -INFINITY ? 0.0f : top;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float sum = 0.0f, f = 0.0f;
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    if (i0 % kLanes == 0) {
      if (i0 > 0) ml = load_ml(i0 + sub);
      f = exp2_approx(ml.x - use);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int from = (i0 + i) & (kLanes - 1);
      const float fi = __shfl_sync(lanes, f, from, kLanes);
      sum = fmaf(fi, __shfl_sync(lanes, ml.y, from, kLanes), sum);
      o.x = fmaf(fi, x[i].x, o.x);
      o.y = fmaf(fi, x[i].y, o.y);
      o.z = fmaf(fi, x[i].z, o.z);
      o.w = fmaf(fi, x[i].w, o.w);
      x[i] = load_o(i0 + kBatch + i);
    }
  }
  const int group = static_cast<int>(a.group.d);
  const int tok = a.group(p.row0 + row);
  const int64_t t = p.first + tok;
  const int head = p.head * group + p.row0 + row - tok * group;
  float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (a.cache.v_scale != nullptr && !a.cache.paged) inv *= a.cache.v_scale[p.head];
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out.data) + t * a.out.token_stride +
                            head * a.out.head_stride + d) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (d == 0 && a.lse != nullptr) a.lse[t * a.q.heads + head] = lse_of(top, sum);
}

}  // namespace

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
