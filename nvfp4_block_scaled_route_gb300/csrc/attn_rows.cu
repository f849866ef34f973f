// Paged attention for few query rows per key head (single tokens, drafted
// tokens): rows = new tokens * (query heads / key heads) <= 16.
//
// Every key and value is read once and used by all the rows of its head, so
// the bound is HBM: 2 * 2 * D bytes of a bf16 key and value against 4 * rows *
// D flops.  The work is the flat list of 128-key tiles of all (request, key
// head) segments; CTA c of G takes the tiles [c n / G, (c + 1) n / G), so
// uneven requests and one long request load the SMs alike.  A segment cut by
// such a border leaves pieces (unscaled sums, maxima, weight sums) that
// attn_combine_kernel joins.
//
// One producer warp keeps a ring of key and value tiles in flight by TMA (one
// box per page; the 128-byte swizzle makes the ldmatrix reads conflict-free).
// Eight compute warps share each tile: for the scores a warp takes 16 of the
// 128 keys; the warps exchange row maxima and the 16-bit weights through
// shared memory, and for the weighted sum a warp takes D / 8 of the
// dimensions over all keys.  So a warp holds few accumulators (no partial sums
// of whole rows to join per tile), and both products run on mma.sync
// m16n8k16: with one tile of rows the tensor pipe is far from its limit even so.
// 64 requests of up to 16384 tokens (56 query, 8 key heads of 128, bf16) take
// 226 us, 6.0 TB/s.
//
// E4M3 caches: two groups of eight warps take the tiles in
// turn, each with its own sums and maxima and a ring of its own (so that it
// waits for every phase of its barriers), and the second hands its part of a
// segment to the first.  A tile's chain of products, exchanges and products
// takes 1900 cycles of latency, an E4M3 tile's bytes 1400 of HBM: two requests
// of up to 131072 tokens 72 -> 65 us.  (Its 17 warps leave a thread 96 registers, of
// which 72 to 132 bytes spill.)  A bf16 tile takes 2800 anyway, and there
// the second group costs (64 requests 228 -> 240 us).
//
// E4M3 caches: keys and values are exact in fp16, so the products run in fp16.
// A query row is scaled by a power of two to a maximum in [1, 2), which keeps
// every element above 2^-16 of it exact, and the factor goes back in with the
// softmax scale.  Weights are taken relative to 2^-15 of the running maximum, so
// that they are at most 2^15 and have all 11 bits of fp16 down to 2^-29 of the largest.
// Values arrive as pairs of neighbouring dimensions (ldmatrix
// moves 16-bit units), so one accumulator tile holds the even dimensions and
// one the odd.
#include "attn.cuh"

namespace nvmoe {
namespace {

constexpr int kKeys = kAttnTileKeys;
constexpr int kRows = kAttnFewRows;               // an m16 tile
static_assert(kRows == 16, "rows of a product");
constexpr int kComputeWarps = 8;                  // of a group
constexpr int kComputeThreads = kComputeWarps * 32;
template <bool FP8>
constexpr int kGroups = FP8 ? 2 : 1;
template <bool FP8>
constexpr int kThreads = kGroups<FP8> * kComputeThreads + 32;
constexpr int kMaxBufs = 16;
// Powers of two by which a row's reference stands below its running maximum.
template <bool FP8>
constexpr float kLift = FP8 ? 15.0f : 0.0f;

template <int D, bool FP8>
struct Tile {
  static constexpr int kRingBytes = 192 * 1024;
  static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
  static constexpr int kLine = kRowBytes < 128 ? kRowBytes : 128;   // bytes of a TMA box row
  static constexpr int kHalves = kRowBytes / kLine;
  static constexpr int kBytes = kKeys * kRowBytes;
  static constexpr int kBufs = kRingBytes / kBytes < kMaxBufs ? kRingBytes / kBytes : kMaxBufs;
  // Byte offset of 16-byte chunk c of key row r.
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    if (kLine == 128)
      return (c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  }
};

// Byte offset of chunk c of row r of a row-major 16-bit matrix of ROW bytes a
// row (128 or 256), chunks permuted within each 128 bytes.
template <int ROW>
__device__ __forceinline__ uint32_t mat_at(int r, int c) {
  return r * ROW + ((c ^ (r & 7)) << 4);
}

struct Bars {
  uint64_t full[kMaxBufs];
  uint64_t empty[kMaxBufs];
  int abort;
  int spoilt;                         // some sum is not finite
  // where the CTA starts: request, tile within it
  Request rq;
  int r;
  long long tile;
};

template <int D, bool FP8>
constexpr int smem_bytes() {
  constexpr int rows = kRows, groups = kGroups<FP8>;
  return 1024 + Tile<D, FP8>::kBufs * Tile<D, FP8>::kBytes + rows * D * 2 +
         groups * (rows * kKeys * 2 + rows * kComputeWarps * 4) + rows * 4 +
         (groups - 1) * (rows * D * 4 + rows * 8) + static_cast<int>(sizeof(Bars));
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <bool HALF>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (HALF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The warps of one group; those of all.
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kComputeThreads) : "memory");
}
template <int GROUPS>
__device__ __forceinline__ void all_sync() {
  asm volatile("bar.sync 3, %0;" ::"n"(GROUPS * kComputeThreads) : "memory");
}

// 128-key tiles of a request: [t0, t1), empty without new tokens.  A request
// whose rows see nothing still gets one tile, so that its rows are written.
struct Span {
  int t0, t1;
};
__device__ __forceinline__ Span tiles_of(const Request& q, int window) {
  if (q.n == 0) return {0, 0};
  const int end = min(q.len, q.pos0 + q.n);
  const int begin = first_key(q.pos0, window);
  if (end <= begin) return {0, 1};
  return {begin / kKeys, (end + kKeys - 1) / kKeys};
}

// A CTA's walk over its tiles: request r, key head h, tile t of [t0, t1).
struct Walk {
  int r, h;
  Request rq;
  Span sp;
  __device__ __forceinline__ void load(const AttnArgs& a, int request) {
    r = request;
    rq = load_request(a.batch, a.cache.page_shift, r, a.status);
    sp = tiles_of(rq, a.window);
  }
  // (only called while tiles are left; false if the batch ends all the same)
  __device__ __forceinline__ bool next_segment(const AttnArgs& a) {
    if (++h < a.cache.heads) return true;
    h = 0;
    do {
      if (r + 1 >= a.batch.batch) return false;
      load(a, r + 1);
    } while (sp.t1 == sp.t0);
    return true;
  }
};

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads<FP8>, 1)
attention_rows_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v) {
  using T = Tile<D, FP8>;
  constexpr int kQRow = D * 2, kPRow = kKeys * 2;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* ring = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  uint8_t* sq = ring + T::kBufs * T::kBytes;
  uint8_t* sp_ = sq + kRows * kQRow;
  constexpr int kG = kGroups<FP8>, kWarps = kThreads<FP8> / 32;
  constexpr int kPer = T::kBufs / kG;                               // buffers of a group
  float* smax = reinterpret_cast<float*>(sp_ + kG * kRows * kPRow);      // [group][kRows][8]
  float* sfac = smax + kG * kRows * kComputeWarps;                       // [kRows]
  float* join_o = sfac + kRows;                       // second group's sums, by thread
  float2* join_ml = reinterpret_cast<float2*>(join_o + (kG - 1) * kRows * D);  // [kRows]
  Bars* bars = reinterpret_cast<Bars*>(join_ml + (kG - 1) * kRows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();                                       // for what came before

  // ---- this CTA's share of the tiles ----
  long long* scan = reinterpret_cast<long long*>(smax);           // [kWarps] warp sums
  const int per = (a.batch.batch + kThreads<FP8> - 1) / kThreads<FP8>;
  const int r_begin = min(a.batch.batch, static_cast<int>(threadIdx.x) * per);
  const int r_end = min(a.batch.batch, r_begin + per);
  long long mine = 0;
  for (int r = r_begin; r < r_end; ++r) {
    const Span s = tiles_of(load_request(a.batch, a.cache.page_shift, r, a.status), a.window);
    mine += static_cast<long long>(s.t1 - s.t0) * a.cache.heads;
  }
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) scan[warp] = upto;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kG * kPer; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->empty[i], kComputeWarps);
    }
    bars->abort = 0;
    bars->spoilt = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
  }
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const int takers = share_takers(total, gridDim.x);
  AttnPiece* piece = a.pieces + blockIdx.x;
  if (static_cast<int>(blockIdx.x) >= takers) {
    if (threadIdx.x == 0) piece->rows = 0;
    return;
  }
  const long long lo = share_begin(total, blockIdx.x, takers);
  const long long hi = share_begin(total, blockIdx.x + 1, takers);
  long long first = before + upto - mine;
  if (lo >= first && lo < first + mine) {
    int r = r_begin;
    Request rq;
    while (true) {
      rq = load_request(a.batch, a.cache.page_shift, r, a.status);
      const Span s = tiles_of(rq, a.window);
      const long long c = static_cast<long long>(s.t1 - s.t0) * a.cache.heads;
      if (lo < first + c || r + 1 >= r_end) break;
      first += c;
      ++r;
    }
    bars->rq = rq;
    bars->r = r;
    bars->tile = lo - first;
  }
  __syncthreads();
  Walk wk;
  wk.r = bars->r;
  wk.rq = bars->rq;
  wk.sp = tiles_of(wk.rq, a.window);
  const int span0 = max(1, wk.sp.t1 - wk.sp.t0);
  const long long tile = bars->tile;
  wk.h = tile < (1ll << 32) ? static_cast<uint32_t>(tile) / static_cast<uint32_t>(span0)
                            : static_cast<int>(tile / span0);
  int t = wk.sp.t0 + static_cast<int>(tile - static_cast<long long>(wk.h) * span0);
  long long left = hi - lo;
  volatile int* abort = &bars->abort;

  if (warp == kG * kComputeWarps) {
    // ---- producer: lane = box of the tile (page part, half row) ----
    const int box = min(kKeys, 1 << a.cache.page_shift);
    const int boxes = kKeys / box;
    const int b = lane & 7, half = lane >> 3;
    const uint64_t policy = policy_evict_first();
    int buf[kG] = {}, side = 0;
    uint32_t phase[kG] = {};
    bool ok = true;
    while (left > 0 && ok) {
      const int kbeg = first_key(wk.rq.pos0, a.window);
      const int kend = min(wk.rq.len, wk.rq.pos0 + wk.rq.n);
      const int stop = static_cast<int>(min(static_cast<long long>(wk.sp.t1), t + left));
      left -= stop - t;
      for (; t < stop && ok; ++t) {
        const int key = t * kKeys + b * box;
        const bool take = b < boxes && half < T::kHalves && key < kend && key + box > kbeg;
        int page = 0;
        if (take) {
          page = a.batch.page_table[wk.r * a.batch.max_pages + (key >> a.cache.page_shift)];
          if (page < 0 || page >= a.cache.num_pages) {
            record_status(a.status, kErrBadIndex);
            page = static_cast<int>(a.cache.num_pages);     // past the map: zeros
          }
        }
        const int loads = T::kHalves * boxes_of(t * kKeys, box, kbeg, kend);
        const int in_page = key & ((1 << a.cache.page_shift) - 1);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int n = side * kPer + buf[side];
          // (nothing here joins the lanes again: in a failing CTA some may go on)
          ok = ok && mbar_wait(&bars->empty[n], phase[side] ^ 1u, a.status, abort);
          if (!ok) break;
          if (lane == 0)
            mbar_arrive_expect_tx(&bars->full[n], static_cast<uint32_t>(loads * box * T::kLine));
          if (take)
            tma_load_4d(ring + n * T::kBytes + half * kKeys * T::kLine + b * box * T::kLine,
                        kv == 0 ? &map_k : &map_v, half * (T::kLine / (FP8 ? 1 : 2)), in_page,
                        wk.h, page, &bars->full[n], policy);
          if (++buf[side] == kPer) {
            buf[side] = 0;
            phase[side] ^= 1u;
          }
        }
        if (kG == 2) side ^= 1;                         // the groups take turns
      }
      if (left > 0) {
        if (!wk.next_segment(a)) break;
        t = wk.sp.t0;
      }
    }
    __syncthreads();
    drain_after_abort(abort);
    return;
  }

  // ---- compute warps: group `side`, warp `w` of it ----
  const int side = kG == 2 ? warp >> 3 : 0, w = warp & 7;
  const int thread = threadIdx.x & (kComputeThreads - 1);
  const int group = a.q.heads / a.cache.heads;
  sp_ += side * kRows * kPRow;
  smax += side * kRows * kComputeWarps;
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  constexpr int kN = (D == 128) ? 2 : 1;            // 8-wide accumulator tiles of a warp
  const uint32_t sq_u = smem_u32(sq), sp_u = smem_u32(sp_);
  ring += side * kPer * T::kBytes;
  const uint32_t ring_u = smem_u32(ring);
  uint64_t* full = bars->full + side * kPer;
  uint64_t* empty = bars->empty + side * kPer;
  int buf = 0;
  uint32_t phase = 0, seq = 0;
  const auto next_buffer = [&] {
    if (++buf == kPer) {
      buf = 0;
      phase ^= 1u;
    }
  };
  int slot1_rows = 0;
  while (left > 0) {
    const int rows = wk.rq.n * group;               // <= kRows, checked on the host
    const int stop = static_cast<int>(min(static_cast<long long>(wk.sp.t1), t + left));
    const bool whole = t == wk.sp.t0 && stop == wk.sp.t1;
    const int slot = t == wk.sp.t0 ? 1 : 0;         // a cut segment: begun here, or before
    left -= stop - t;
    float c = a.scale * 1.4426950408889634f;        // scores in powers of two
    if (FP8 && a.cache.k_scale != nullptr) c *= a.cache.k_scale[wk.h];

    // queries to shared memory
    constexpr int kLanes = D / 8;
    for (int row = threadIdx.x / kLanes; row < kRows; row += kG * kComputeThreads / kLanes) {
      const int ch = threadIdx.x & (kLanes - 1);
      uint4 u = make_uint4(0, 0, 0, 0);
      if (row < rows) {
        const int i = row / group;
        u = *reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(a.q.data) + (wk.rq.first + i) * a.q.token_stride +
            (wk.h * group + row - i * group) * a.q.head_stride + ch * 8);
      }
      if (!FP8) {
        *reinterpret_cast<uint4*>(sq + mat_at<kQRow>(row, ch)) = u;
      } else {
        float x[8], most = 0.0f;
        bf16x8_to_float(u, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(x[j]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
          most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
        // 2^(127 - e) and 2^(e - 127); rows of zeros or infinities stay as they are
        int e = static_cast<int>(__float_as_uint(most) >> 23);
        e = e == 0 || e == 255 ? 127 : min(e, 253);
        const float up = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        if (ch == 0) sfac[row] = __uint_as_float(static_cast<uint32_t>(e) << 23);
        // a 4-byte word of an E4M3 key row holds dimensions 4i .. 4i+3 of its 16:
        // the first two are the product's k = 2i, 2i+1, the others its 2i+8, 2i+9
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int pair = (ch & 1) * 4 + j;        // of the 8 pairs of 16 dimensions
          const int k = (pair & 1) * 4 + (pair >> 1);
          *reinterpret_cast<uint32_t*>(sq + mat_at<kQRow>(row, (ch & ~1) + (k >> 2)) +
                                       (k & 3) * 4) =
              pack_f16x2(x[2 * j] * up, x[2 * j + 1] * up);
        }
      }
    }
    all_sync<kG>();

    float o[kN][4], m[2], l[2], cr[2];
    int vis_hi[2], vis_lo[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = e * 8 + g;
      const int pos = wk.rq.pos0 + row / group;
      vis_hi[e] = min(pos + 1, wk.rq.len);
      vis_lo[e] = first_key(pos, a.window);
      m[e] = -INFINITY;
      l[e] = 0.0f;
      cr[e] = FP8 ? c * sfac[row] : c;
#pragma unroll
      for (int n = 0; n < kN; ++n) o[n][2 * e] = o[n][2 * e + 1] = 0.0f;
    }
    // keys that every row sees
    const int all_hi = min(wk.rq.pos0 + 1, wk.rq.len);
    const int all_lo = first_key(wk.rq.pos0 + wk.rq.n - 1, a.window);
    // keys that any row sees
    const int kend = min(wk.rq.len, wk.rq.pos0 + wk.rq.n);
    const int kbeg = first_key(wk.rq.pos0, a.window);

    for (; t < stop; ++t, ++seq) {
      if (kG == 2 && static_cast<int>(seq & 1u) != side) continue;
      const int key0 = t * kKeys;
      // scores of this warp's 16 keys
      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
      mbar_wait(&full[buf], phase, a.status, abort);
      {
        const uint32_t kb = ring_u + buf * T::kBytes;
        const int krow = w * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
        for (int ks = 0; ks < D / (FP8 ? 32 : 16); ++ks) {
          uint32_t kf[4];
          ldsm4(kb + T::at(krow, 2 * ks + ((lane >> 3) & 1)), kf);
          if (!FP8) {
            uint32_t qf[4];
            ldsm4(sq_u + mat_at<kQRow>(lane & 15, 2 * ks + (lane >> 4)), qf);
            mma16816<false>(s[0], qf, kf[0], kf[1]);
            mma16816<false>(s[1], qf, kf[2], kf[3]);
          } else {
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
              uint32_t qf[4];
              ldsm4(sq_u + mat_at<kQRow>(lane & 15, 4 * ks + 2 * k2 + (lane >> 4)),
                    qf);
              mma16816<true>(s[0], qf, e4m3x2_to_f16x2(kf[k2]),
                             e4m3x2_to_f16x2(kf[k2] >> 16));
              mma16816<true>(s[1], qf, e4m3x2_to_f16x2(kf[2 + k2]),
                             e4m3x2_to_f16x2(kf[2 + k2] >> 16));
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[buf]);
      next_buffer();

      const bool masked = key0 + kKeys > all_hi || key0 < all_lo;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float& x = s[n][2 * e + j];
            x *= cr[e];
            if (masked) {
              const int key = key0 + w * 16 + n * 8 + c2 + j;
              if (key >= vis_hi[e] || key < vis_lo[e]) x = -INFINITY;
            }
            top = fmaxf(top, x);
          }
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        if ((lane & 3) == 0) smax[(e * 8 + g) * kComputeWarps + w] = top;
      }
      group_sync(side);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = e * 8 + g;
        const float4* mx = reinterpret_cast<const float4*>(smax + row * kComputeWarps);
        const float4 u = mx[0], v = mx[1];
        const float mn =
            fmaxf(fmaxf(fmaxf(fmaxf(u.x, u.y), fmaxf(u.z, u.w)),
                        fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w))) - kLift<FP8>, m[e]);
        const float use = mn == -INFINITY ? 0.0f : mn;   // a row without keys so far
        const float f = exp2_approx(m[e] - use);
        m[e] = mn;
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = exp2_approx(s[n][2 * e] - use);
          const float p1 = exp2_approx(s[n][2 * e + 1] - use);
          sum += p0 + p1;
          *reinterpret_cast<uint32_t*>(sp_ + mat_at<kPRow>(row, w * 2 + n) + c2 * 2) =
              FP8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
        }
        l[e] = fmaf(l[e], f, sum);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          o[n][2 * e] *= f;
          o[n][2 * e + 1] *= f;
        }
      }
      mbar_wait(&full[buf], phase, a.status, abort);
      const bool cut = key0 < kbeg || key0 + kKeys > kend;
      if (cut) {
        // values that no row sees may hold anything: make them zeros
        for (int i = thread; i < kKeys * (T::kRowBytes / 16); i += kComputeThreads) {
          const int row = i / (T::kRowBytes / 16), ch = i % (T::kRowBytes / 16);
          if (key0 + row < kbeg || key0 + row >= kend)
            *reinterpret_cast<uint4*>(ring + buf * T::kBytes + T::at(row, ch)) =
                make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();                   // before the next TMA into this buffer
      }
      group_sync(side);
      // weighted sum over the 128 keys of this warp's dimensions
      const uint32_t vb = ring_u + buf * T::kBytes;
#pragma unroll
      for (int k2 = 0; k2 < kKeys / 32; ++k2) {
        uint32_t b0[2][kN], b1[2][kN];              // k16 step, accumulator tile
        if (FP8) {
          uint32_t v[4];
          ldsm4_t(vb + T::at(k2 * 32 + lane, D == 128 ? w : w >> 1), v);
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            uint32_t h[4];
            h[0] = e4m3x2_to_f16x2(v[2 * st]);              // (key, dims d and d + 1)
            h[1] = e4m3x2_to_f16x2(v[2 * st] >> 16);        // (key + 1, ...)
            h[2] = e4m3x2_to_f16x2(v[2 * st + 1]);
            h[3] = e4m3x2_to_f16x2(v[2 * st + 1] >> 16);
            if (D == 128) {
#pragma unroll
              for (int n = 0; n < kN; ++n) {
                b0[st][n] = __byte_perm(h[0], h[1], n == 0 ? 0x5410 : 0x7632);
                b1[st][n] = __byte_perm(h[2], h[3], n == 0 ? 0x5410 : 0x7632);
              }
            } else {
              const uint32_t sel = (w & 1) == 0 ? 0x5410 : 0x7632;
              b0[st][0] = __byte_perm(h[0], h[1], sel);
              b1[st][0] = __byte_perm(h[2], h[3], sel);
            }
          }
        } else if (D == 128) {
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            uint32_t v[4];
            ldsm4_t(vb + T::at(k2 * 32 + st * 16 + (lane & 15), w * 2 + (lane >> 4)), v);
            b0[st][0] = v[0];
            b1[st][0] = v[1];
            b0[st][kN - 1] = v[2];
            b1[st][kN - 1] = v[3];
          }
        } else {
          uint32_t v[4];
          ldsm4_t(vb + T::at(k2 * 32 + lane, w), v);
          b0[0][0] = v[0];
          b1[0][0] = v[1];
          b0[1][0] = v[2];
          b1[1][0] = v[3];
        }
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          uint32_t pf[4];
          ldsm4(sp_u + mat_at<kPRow>(lane & 15, (k2 * 2 + st) * 2 + (lane >> 4)), pf);
#pragma unroll
          for (int n = 0; n < kN; ++n) mma16816<FP8>(o[n], pf, b0[st][n], b1[st][n]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[buf]);
      next_buffer();
    }

    // ---- weight sums over the warps, then the rows out ----
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[e];
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
      if ((lane & 3) == 0) smax[(e * 8 + g) * kComputeWarps + w] = x;
    }
    group_sync(side);
    float lsum[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float4* sm =
          reinterpret_cast<const float4*>(smax + (e * 8 + g) * kComputeWarps);
      const float4 u = sm[0], v = sm[1];
      lsum[e] = ((u.x + u.y) + (u.z + u.w)) + ((v.x + v.y) + (v.z + v.w));
    }
    if (kG == 2) {
      // the second group's part to the first
      if (side == 1) {
#pragma unroll
        for (int k = 0; k < kN * 4; ++k) join_o[k * kComputeThreads + thread] = o[k >> 2][k & 3];
        if (w == 0 && (lane & 3) == 0)
#pragma unroll
          for (int e = 0; e < 2; ++e) join_ml[e * 8 + g] = make_float2(m[e], lsum[e]);
      }
      all_sync<kG>();
      if (side == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 ml = join_ml[e * 8 + g];
          const float mn = fmaxf(m[e], ml.x), use = mn == -INFINITY ? 0.0f : mn;
          const float f0 = exp2_approx(m[e] - use), f1 = exp2_approx(ml.x - use);
          m[e] = mn;
          lsum[e] = lsum[e] * f0 + ml.y * f1;
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int k = n * 4 + 2 * e + j;
              o[n][2 * e + j] =
                  o[n][2 * e + j] * f0 + join_o[k * kComputeThreads + thread] * f1;
            }
        }
      }
    }
    const float v_scale = FP8 && a.cache.v_scale != nullptr ? a.cache.v_scale[wk.h] : 1.0f;
    const int64_t pc = 2 * static_cast<int64_t>(blockIdx.x) + slot;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = e * 8 + g;
      if (row >= rows || side != 0) continue;
      const float sum = lsum[e];
      const int tok = row / group;
      const int64_t tk = wk.rq.first + tok;
      const int head = wk.h * group + row - tok * group;
      const float inv = sum == 0.0f ? 0.0f : v_scale / sum;
      float probe = 0.0f;                         // NaN if some sum is not finite
#pragma unroll
      for (int n = 0; n < kN; ++n)
        probe = fmaf(o[n][2 * e], 0.0f, fmaf(o[n][2 * e + 1], 0.0f, probe));
      if (probe != 0.0f) bars->spoilt = 1;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) +
                           tk * a.out.token_stride + head * a.out.head_stride;
      float* po = a.piece_o + (pc * a.piece_rows + row) * D;
      // the dimensions of this thread's accumulators
      if (FP8 && D == 128) {
        const int d = w * 16 + c2 * 2;
        const float y[4] = {o[0][2 * e], o[kN - 1][2 * e], o[0][2 * e + 1],
                            o[kN - 1][2 * e + 1]};
        if (whole)
          *reinterpret_cast<uint2*>(out + d) =
              make_uint2(pack_bf16x2(y[0] * inv, y[1] * inv),
                         pack_bf16x2(y[2] * inv, y[3] * inv));
        else
          *reinterpret_cast<float4*>(po + d) = make_float4(y[0], y[1], y[2], y[3]);
      } else if (FP8) {
        const int d = (w >> 1) * 16 + c2 * 2 + (w & 1);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (whole) out[d + 2 * j] = __float2bfloat16_rn(o[0][2 * e + j] * inv);
          else po[d + 2 * j] = o[0][2 * e + j];
        }
      } else {
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          const int d = (w * kN + n) * 8 + c2;
          const float y0 = o[n][2 * e], y1 = o[n][2 * e + 1];
          if (whole)
            *reinterpret_cast<uint32_t*>(out + d) = pack_bf16x2(y0 * inv, y1 * inv);
          else
            *reinterpret_cast<float2*>(po + d) = make_float2(y0, y1);
        }
      }
      if (w == 0 && (lane & 3) == 0) {
        if (whole) {
          if (a.lse != nullptr) a.lse[tk * a.q.heads + head] = lse_of(m[e], sum);
        } else {
          a.piece_ml[pc * a.piece_rows + row] = make_float2(m[e], sum);
        }
      }
    }
    if (threadIdx.x == 0 && !whole && slot == 1) {
      // this CTA begins a cut segment: where its pieces end, for the join
      long long end = hi + (wk.sp.t1 - stop);
      int last = blockIdx.x + 1;
      while (last + 1 < takers && share_begin(total, last + 1, takers) < end) ++last;
      AttnPiece p;
      p.rows = rows;
      p.head = wk.h;
      p.first = wk.rq.first;
      p.row0 = 0;
      p.last = last;
      *piece = p;
      slot1_rows = rows;
    }
    if (left > 0) {
      if (!wk.next_segment(a)) break;
      t = wk.sp.t0;
    }
  }
  if (threadIdx.x == 0 && slot1_rows == 0) piece->rows = 0;
  __syncthreads();
  drain_after_abort(abort);
  if (bars->spoilt == 0) return;
  // ---- rows that hidden keys may have spoilt: the same walk again ----
  wk.load(a, bars->r);
  wk.h = static_cast<int>(bars->tile / max(1, wk.sp.t1 - wk.sp.t0));
  t = wk.sp.t0 + static_cast<int>(bars->tile % max(1, wk.sp.t1 - wk.sp.t0));
  for (left = hi - lo; left > 0; t = wk.sp.t0) {
    const int stop = static_cast<int>(min(static_cast<long long>(wk.sp.t1), t + left));
    const bool whole = t == wk.sp.t0 && stop == wk.sp.t1;
    left -= stop - t;
    const int kbeg = first_key(wk.rq.pos0, a.window);
    const int kend = min(wk.rq.len, wk.rq.pos0 + wk.rq.n);
    const int64_t at =
        (2 * static_cast<int64_t>(blockIdx.x) + (t == wk.sp.t0 ? 1 : 0)) * a.piece_rows;
    mend_rows<D, FP8>(a, wk.r, wk.h, 0, wk.rq.n * group, kbeg, kend, t, stop,
              whole ? nullptr : a.piece_o + at * D, a.piece_ml + at, warp, kG * kComputeWarps);
    if (left > 0 && !wk.next_segment(a)) break;
  }
}

template <int D, bool FP8>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int grid,
                   cudaStream_t stream) {
  static PerDeviceOnce once;
  constexpr int bytes = smem_bytes<D, FP8>();
  static_assert(bytes <= 232448, "shared memory");
  auto kernel = attention_rows_kernel<D, FP8>;
  cudaError_t e = set_smem_attr_once(once, reinterpret_cast<const void*>(kernel), bytes);
  if (e != cudaSuccess) return e;
  // its start overlaps the end of the kernel before
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads<FP8>);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, mk, mv);
}

}  // namespace

cudaError_t launch_attention_rows(const AttnArgs& a, const CUtensorMap& map_k,
                                  const CUtensorMap& map_v, int grid, cudaStream_t stream) {
  if (a.cache.fp8)
    return a.cache.head_dim == 128 ? launch<128, true>(a, map_k, map_v, grid, stream)
                                   : launch<64, true>(a, map_k, map_v, grid, stream);
  return a.cache.head_dim == 128 ? launch<128, false>(a, map_k, map_v, grid, stream)
                                 : launch<64, false>(a, map_k, map_v, grid, stream);
}

}  // namespace nvmoe
