// Appending keys and values to E4M3 pages that have one scale for each page and head.
//
// A block takes the new tokens of one page and head, of k or of v: norm and rotation
// in fp32, the largest |x| of them, the scale, the E4M3 values.  So x is read once and
// its 8 bits are written once, and the bound is HBM as without scales (single tokens:
// the launch and a chain of dependent loads).
//
// The scale is the smallest power of two s with max |x| <= 448 s, within
// kScaleLow .. kScaleHigh; a page that holds tokens already keeps its own if that is
// larger.  If it has to grow, the block also takes the page's old values times
// old / new.  E4M3 is a floating-point format: between powers of two nothing is lost
// but the last bits of values below 2^-6 of the new scale, however often a page grows,
// where scales of amax / 448 would round every value anew each time.
#include <algorithm>

#include "attn_turn.cuh"

namespace nvmoe {
namespace {

// Which blocks append: `blocks` of them, two (k and v) for each head and unit.  A unit
// is a page of new tokens, found from the unit's number: request r owns those from
// q_start[r] / page_size + 2 r on, which are enough for its pages (a run of n tokens
// touches at most n / page_size + 2).  Where there are fewer tokens than that (single
// and drafted tokens), a unit is a token, and the first one in a page takes the page.
struct PageUnits {
  uint32_t blocks;
  uint64_t share;                                       // blocks / all, in 2^-32, rounded up
};

// A thread takes R tokens' eight elements: values stay in registers as they came, turned
// keys go to shared memory as fp32 until the scale is known.  (64 registers a thread, as
// the queries' rows take, which are most of the bytes in the same launch.  Keys turned a
// second time instead: 165 us where this then took 152, 148 by now, three prompts of 8192
// tokens at most, 56 + 8 + 8 heads of 128.)
constexpr int kR = 4;
constexpr int kHeldBytes = kR * 8 * 4;                  // a thread

template <int D, int THREADS, int HEADS, bool TOKENS, bool PAIRS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
page_append_kernel(const RopeArgs a, const PageUnits units) {
  constexpr int R = kR, kLanes = D / 8, kGroups = THREADS / kLanes, kRound = kGroups * R;
  __shared__ float warp_max[THREADS / 32];
  extern __shared__ float4 smem[];
  pdl_wait();                                           // for what came before
  pdl_trigger();
  // Single tokens: appending blocks first.  Else they are spread evenly over the others,
  // which wait for bytes where these compute (152 -> 148 us; the division that single
  // tokens do without is 0.3-0.9 us of a launch of 4.8).
  uint32_t mine = blockIdx.x, others = blockIdx.x - units.blocks;
  bool append = mine < units.blocks;
  if (!TOKENS) {
    mine = static_cast<uint32_t>(blockIdx.x * units.share >> 32);
    append = static_cast<uint32_t>((blockIdx.x + uint64_t{1}) * units.share >> 32) != mine;
    others = blockIdx.x - mine;
  }
  if (!append) {
    transform_heads<D, HEADS, true, PAIRS, false>(a, others * kGroups + threadIdx.x / kLanes);
    return;
  }
  const bool value = mine & 1;
  const uint32_t unit = (mine >> 1) / static_cast<uint32_t>(a.cache.heads);
  const int head = static_cast<int>((mine >> 1) - unit * a.cache.heads);
  const HeadRows& src = value ? a.v : a.k;
  const int ps = a.cache.page_shift;

  if (TOKENS && threadIdx.x < kLanes) {
    // the row's way in starts before its request is known
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(src.data) +
                             unit * src.token_stride + head * src.head_stride + threadIdx.x * 8;
    asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
  }
  // ---- the page: request r, whose row t has position t + to_pos ----
  int r;
  if (TOKENS) {
    r = request_of<32>(a.batch, unit, threadIdx.x & 31, 0xFFFFFFFFu);
    if (r < 0) return;
  } else {
    r = last_below<32>(a.batch.batch, threadIdx.x & 31, 0xFFFFFFFFu, [&](int i) {
      return (max(0, a.batch.q_start[i]) >> ps) + 2ll * i <= unit;
    });
  }
  const int64_t begin = a.batch.q_start[r], end = a.batch.q_start[r + 1];
  const int64_t row0 = max(begin, int64_t{0}), row1 = min(end, a.batch.tokens);
  if (row1 <= row0) return;
  const int64_t to_pos = static_cast<int64_t>(a.batch.kv_len[r]) - end;
  int64_t page_i;                                       // of the request
  if (TOKENS) {
    const int64_t pos = unit + to_pos;
    if (pos < 0) {
      record_status(a.status, kErrBadIndex);
      return;
    }
    if ((pos & ((int64_t{1} << ps) - 1)) != 0 && unit != row0) return;
    page_i = pos >> ps;
  } else {
    const int64_t i = unit - ((max(int64_t{0}, begin) >> ps) + 2ll * r);
    if (i < 0) return;
    if (i == 0 && row0 + to_pos < 0) record_status(a.status, kErrBadIndex);
    page_i = (max(row0 + to_pos, int64_t{0}) >> ps) + i;
  }
  // new positions [p0, p1) of the page
  const int64_t first = page_i << ps;
  const int64_t p0 = max(first, row0 + to_pos);
  int64_t p1 = min(first + (int64_t{1} << ps), row1 + to_pos);
  if (p1 <= p0) return;
  bool ok = page_i < a.batch.max_pages;
  int64_t page = 0;
  if (ok) {
    page = a.batch.page_table[r * a.batch.max_pages + page_i];
    ok = page >= 0 && page < a.cache.num_pages;
  }
  if (a.tr.rope != nullptr && p1 > a.tr.rope_positions) {
    p1 = a.tr.rope_positions;
    if (threadIdx.x == 0) record_status(a.status, kErrBadIndex);
  }
  if (!ok && threadIdx.x == 0) record_status(a.status, kErrBadIndex);
  if (!ok || p1 <= p0) return;

  float* scale = (value ? a.cache.v_scale : a.cache.k_scale) + page * a.cache.heads + head;
  const bool grown = p0 > first;                        // holds tokens already
  const float had = grown ? page_scale(*scale) : 0.0f;
  uint8_t* out = static_cast<uint8_t*>(value ? a.cache.v : a.cache.k) + page * a.cache.page_stride +
                 head * a.cache.head_stride;
  const int old = static_cast<int>(p0 - first), count = static_cast<int>(p1 - p0);
  const int sub = threadIdx.x & (kLanes - 1), group = threadIdx.x / kLanes;
  const uint32_t mask = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
  int i0 = sub * 8, i1 = sub * 8 + 4;                   // this lane's elements
  if (!value) HeadTurn<D, PAIRS>::places(sub, a.tr.rotary_dim, i0, i1);
  const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(src.data) +
                            (p0 - to_pos) * src.token_stride + head * src.head_stride;

  // Up to kRound tokens are read once; more (pages of D * page_size > 512 * 8 * R) twice.
  const int rounds = (count + kRound - 1) / kRound;
  const int steps = rounds == 1 ? 1 : 2 * rounds;
  float most = 0.0f, by = 1.0f, inv = 1.0f;
  bool exact = true;
  uint2 raw[R][2];
  float4* held = smem + threadIdx.x;                    // [R][2][THREADS]
  uint64_t w[2][2];
  HeadTurn<D, PAIRS>::weights(value ? nullptr : a.tr.k_weight, i0, i1, w);
  const int64_t step_in = kGroups * src.token_stride, step_out = kGroups * a.cache.token_stride;
  // eight values in the page's scale, to their place
  const auto put = [&](uint8_t* p, const uint64_t (&x)[2][2]) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float z[4];
      f32x2_split(x[s][0], z[0], z[1]);
      f32x2_split(x[s][1], z[2], z[3]);
      if (exact) {
        const uint64_t by2 = f32x2(inv, inv);
        f32x2_split(mul_f32x2(x[s][0], by2), z[0], z[1]);
        f32x2_split(mul_f32x2(x[s][1], by2), z[2], z[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] /= by;
      }
      *reinterpret_cast<uint32_t*>(p + (s == 0 ? i0 : i1)) =
          pack_e4m3x2(z[0], z[1]) | (pack_e4m3x2(z[2], z[3]) << 16);
    }
  };
#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    const int base = (step < rounds ? step : step - rounds) * kRound + group;
    const __nv_bfloat16* p = in + base * src.token_stride;
#pragma unroll
    for (int i = 0; i < R; ++i, p += step_in) {
      if (base + i * kGroups < count) {
        raw[i][0] = *reinterpret_cast<const uint2*>(p + i0);
        raw[i][1] = *reinterpret_cast<const uint2*>(p + i1);
      }
    }
    uint8_t* to = out + (old + base) * a.cache.token_stride;
#pragma unroll
    for (int i = 0; i < R; ++i, to += step_out) {
      const int j = base + i * kGroups;
      if (j >= count) break;
      uint64_t x[2][2];
      bf16x4_to_f32x2(raw[i][0], x[0]);
      bf16x4_to_f32x2(raw[i][1], x[1]);
      if (!value) {
        HeadTurn<D, PAIRS> turn;
        const bool turned = sub * 8 < a.tr.rotary_dim;
        turn.load(a.tr, w, turned, sub, p0 + j);
        turn.apply(x, turned, a.tr.k_weight != nullptr, a.tr.eps, mask);
        if (rounds == 1) {
          held[(2 * i) * THREADS] = reinterpret_cast<const float4&>(x[0]);
          held[(2 * i + 1) * THREADS] = reinterpret_cast<const float4&>(x[1]);
        }
      }
      if (step < rounds) {
        // Infinities saturate and NaN stays NaN: neither counts for the scale.  (x * 0 + x
        // is x or, of those, NaN, which the maximum leaves out.)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float u, v;
          f32x2_split(fma_f32x2(x[k >> 1][k & 1], 0, x[k >> 1][k & 1]), u, v);
          most = fmaxf(most, fmaxf(fabsf(u), fabsf(v)));
        }
      } else {
        put(to, x);
      }
    }
    if (step == rounds - 1) {
      // ---- the scale ----
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
      if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = most;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) most = fmaxf(most, warp_max[w]);
      // most = m 2^e with 1 <= m < 2, 448 = 1.75 * 2^8
      const uint32_t bits = __float_as_uint(most);
      const int e = static_cast<int>(bits >> 23) - ((bits & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
      by = page_scale(__uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23));
      if (grown && by > had) {
        // ---- the values that the page holds already, in the new scale ----
        const float f = had / by;
        constexpr int kChunks = D / 16;
        for (int i = threadIdx.x; i < old * kChunks; i += THREADS) {
          uint4* p = reinterpret_cast<uint4*>(out + i / kChunks * a.cache.token_stride +
                                              i % kChunks * 16);
          const uint4 u = *p;
          uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t y = 0;
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              const uint32_t h = e4m3x2_to_f16x2(w[k] >> (16 * d));
              const float2 z = __half22float2(reinterpret_cast<const __half2&>(h));
              y |= pack_e4m3x2(z.x * f, z.y * f) << (16 * d);
            }
            w[k] = y;
          }
          *p = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      by = fmaxf(by, had);
      if (threadIdx.x == 0) *scale = by;
      // (a product with the reciprocal of a power of two is the quotient; scales that
      // came with the cache may be others)
      exact = (__float_as_uint(by) & 0x7FFFFFu) == 0;
      inv = 1.0f / by;
    }
    if (rounds == 1) {
      uint8_t* to = out + (old + base) * a.cache.token_stride;
#pragma unroll
      for (int i = 0; i < R; ++i, to += step_out) {
        if (base + i * kGroups >= count) break;
        uint64_t x[2][2];
        if (value) {
          bf16x4_to_f32x2(raw[i][0], x[0]);
          bf16x4_to_f32x2(raw[i][1], x[1]);
        } else {
          reinterpret_cast<float4&>(x[0]) = held[(2 * i) * THREADS];
          reinterpret_cast<float4&>(x[1]) = held[(2 * i + 1) * THREADS];
        }
        put(to, x);
      }
    }
  }
}

// units: pages, or tokens where there are fewer.
template <int D, int THREADS, int HEADS, bool TOKENS, bool PAIRS>
cudaError_t launch_with(RopeArgs a, int64_t units, cudaStream_t stream) {
  const auto kernel = page_append_kernel<D, THREADS, HEADS, TOKENS, PAIRS>;
  static PerDeviceOnce once;
  const cudaError_t e = set_smem_attr_once(once, reinterpret_cast<const void*>(kernel),
                                           kHeldBytes * THREADS);
  if (e != cudaSuccess) return e;
  // (tokens * (q heads + 2 key heads) < 2^31, and a page has 16 tokens at least)
  const int64_t kv = units * a.cache.heads * 2;
  a.q_chunks = static_cast<int>(ceil_div(a.q.heads, HEADS));
  a.kv_chunks = 0;
  a.chunks = a.q_chunks;
  const int64_t blocks = kv + ceil_div(a.T * a.chunks, THREADS / (D / 8));
  // (blocks < 2^32: the last block's number times this is below kv + 1)
  const uint64_t share = ((static_cast<uint64_t>(kv) << 32) + blocks - 1) / blocks;
  // its start overlaps the end of the kernel before
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = kHeldBytes * THREADS;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a,
                            PageUnits{static_cast<uint32_t>(kv), share});
}

template <int D, bool PAIRS>
cudaError_t launch_d(const RopeArgs& a, cudaStream_t stream) {
  const int64_t page = int64_t{1} << a.cache.page_shift;
  const int64_t by_page = a.T / page + 2 * int64_t{a.batch.batch};
  // threads so that a page's new tokens are held
  if (a.T <= by_page) return launch_with<D, 128, 2, true, PAIRS>(a, a.T, stream);
  const int64_t elements = page * D;
  if (elements <= 128 * 8 * kR) return launch_with<D, 128, 8, false, PAIRS>(a, by_page, stream);
  if (elements <= 256 * 8 * kR) return launch_with<D, 256, 8, false, PAIRS>(a, by_page, stream);
  return launch_with<D, 512, 8, false, PAIRS>(a, by_page, stream);
}

}  // namespace

cudaError_t launch_page_append(const HeadRows& q, const HeadRows& k, const HeadRows& v,
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
  if (a.tr.interleaved)
    return cache.head_dim == 128 ? launch_d<128, true>(a, stream) : launch_d<64, true>(a, stream);
  return cache.head_dim == 128 ? launch_d<128, false>(a, stream) : launch_d<64, false>(a, stream);
}

}  // namespace nvmoe
