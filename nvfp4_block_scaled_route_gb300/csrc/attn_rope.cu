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
#include "attn_turn.cuh"

namespace nvmoe {
namespace {

constexpr int kThreads = 128;
// Many rows: eight heads a group and 64 registers a thread; into the cache
// four and 48, which hides the longer chain of loads (request, length, page,
// rotation) before a row can be stored.  Measured, 4096 tokens of 56 + 8 heads
// of 128 and 21 k tokens into an E4M3 cache: 8 heads of 64 registers 29.8 us
// and 188 us, 4 of 48 32.4 and 162, 8 of 90 registers 31.3 and 264.
// (With its start over the end of the kernel before, a launch takes 27.4 and 173:
// 5.0 and 4.4 TB/s; 160 of the latter without the divisions by the scales.  Into the
// cache instructions bound it (76 % of the issue slots): each group finds its request,
// page and rotation anew, and at 48 registers a thread spills 104 to 112 bytes and
// reads 204 to 252 back.  Groups that keep what they have found for 8 or 16 heads in
// rounds of 4 took 187 to 190 us, before the divisions.)
// Below kWideRows head rows two heads a group spread few tokens wider (into the cache
// at the same 48 registers, with 52 to 60 bytes of spills).
constexpr int64_t kWideRows = 16384;
template <bool APPEND>
constexpr int kWideHeads = APPEND ? 4 : 8;
template <bool APPEND>
constexpr int kMinBlocks = APPEND ? 10 : 8;

template <int D, int HEADS, bool APPEND, bool PAIRS>
__global__ void __launch_bounds__(kThreads, kMinBlocks<APPEND>)
head_transform_kernel(const RopeArgs a) {
  pdl_wait();                                         // for what came before
  constexpr int kLanes = D / 8;
  transform_heads<D, HEADS, APPEND, PAIRS>(
      a, blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes);
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
