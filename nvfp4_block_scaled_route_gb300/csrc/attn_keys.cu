// Paged attention of up to 16 query rows per key head (single tokens, drafted tokens)
// over E4M3 pages with scales of their own, 128-wide heads: keys in the rows of the
// tcgen05 tiles.
//
// Every key and value is read once for all rows of its head, so the bound is HBM: 2 * D
// bytes for a key and value against 4 * rows * D flops.  What has to stay off the way
// is the conversion of the values to 16 bits, which the products with the queries in the
// tiles' rows need.  Here the cache's bytes are the tensor cores' first operand as they
// lie in shared memory, both times, and the few rows are the second:
//
//   S^T = K Q^T     keys x rows: K is the tile of keys; Q twice, as Qhi + Qlo
//   O^T += V^T P^T  dims x rows: V is the tile of values, read across (MN-major)
//
// A query is the sum of two E4M3 numbers (8 bits of its elements down to 2^-9 of its
// row's largest, to within 2^-17 of that below).  A weight is the sum of four, the
// later ones 2^8, 2^16 and 2^24 times what is left, each with columns of its own in O^T:
// the products are exact, and of weights, fp16 numbers of 11 bits, nothing is lost down to
// 2^-17 of their reference; they are right to within 2^-8 down to 2^-22 of the row's
// largest and to within 2^-31 of that below, where the last numbers are E4M3's small ones.
// (In the sum they go with the scale of their value's page, as a power of two in the
// exponent; without it, in the row's weight sum.)
//
// A thread holds one key and half of the rows, so the scales of pages are one number for
// it, and a row's maximum would have to be looked for across threads.  It is not: m is a
// reference as in the chunk kernel, and only when some thread finds a weight above 2^2
// (a barrier with a vote) is the maximum exchanged and O^T rescaled.
//
// The chain of a tile (scores to registers, vote, exponentials, four conversions, weights
// to shared memory) takes 1300 cycles of latency and its bytes 1080 of HBM, and between
// two segments the queries' way in and the rows' way out take some 4000, so an SM runs
// two CTAs, with half of the shared memory each (at a time when two took 126 us, one took
// 138, and one with two tiles in the work at a time 142).  64 tokens on up to 16384 keys,
// 56 query and 8 key heads, pages of 16: 122 us, 5.6 TB/s (117 with heads first);
// attention_rows_kernel, which turns the values to 16 bits, took 200.  Up to 1000 keys: 28
// us.  Of a request with one tile (7.6 us) 6.5 are this kernel, most of them the fetching
// of code that runs once and six loads on one another, so values of rows are joined over
// the threads in halves (32 -> 29 us for 1000 keys; 2 tokens, 14 rows: 48 -> 42).
//
// The work is the flat list of 128-key tiles of all (request, key head) segments in equal
// shares, as in attention_rows_kernel; attn_combine_kernel joins what is cut.
//
// Roles: warps 0-3 and 4-7 hold the softmax, each the 128 keys of a tile for half of the
// rows; warps 8 and 9 load keys (with the scales) and values by TMA, a box per page;
// warps 10 and 11 issue the products.
#include "attn.cuh"

namespace nvmoe {
namespace {

constexpr int kKeys = kAttnTileKeys, kD = 128;
constexpr int kThreads = 384, kSoftmaxThreads = 256;
constexpr int kLoadK = 8, kLoadV = 9, kIssueS = 10;    // and 11: the sums
constexpr int kLevels = 4;                             // E4M3 numbers of a weight
constexpr int kTileBytes = kKeys * kD;
constexpr int kScaleSlots = 8, kTileScales = 8;       // scales of 16 keys each
constexpr uint32_t kTmemColumns = 128;
// Powers of two by which a row's maximum may stand above its reference, the maximum when
// it was set.  No number of a weight may pass 448, where E4M3 ends: it would be cut.  A
// number between 2^e and 2^(e+1) leaves 2^(e-4) at most, the next one is at most 2^(e+4).
// Below 2^2 the first leaves 2^-3, the second is at most 2^5 and leaves 1, the third at
// most 2^8; of the fp16 weight's 11 bits that is one, which it holds.  (Below 2^4, half of
// the weights above 2^3 lose up to 2^-9.9 of themselves in the third and fourth.)
constexpr float kSlack = 2.0f;

// RG: rows of a softmax group; both have as many.
template <int RG>
struct Cfg {
  static_assert(2 * RG <= kAttnFewRows, "rows");
  static constexpr int kRows = 2 * RG;
  // columns of the two products: a row's Qhi and, kRows on, its Qlo; a weight's levels
  static constexpr int kN1 = 2 * kRows, kN2 = kLevels * kRows;
  static_assert(kN1 % 16 == 0 && kN2 % 16 == 0 && kN2 <= 256, "columns of a product");
  static constexpr uint32_t kTmemO = 2 * kN1;          // S: columns 0 and kN1
  static_assert(kTmemO + kN2 <= kTmemColumns, "TMEM");
  static constexpr int kQAt = 0, kQBytes = kRows * kD;  // Qhi, Qlo
  static constexpr int kPAt = 2 * kQBytes, kPBytes = kN2 * kKeys;
  static constexpr int kRingAt = kPAt + 2 * kPBytes;
  // buffers of keys and of values
  static constexpr int kK = 3, kV = RG > 4 ? 2 : 3;
  static constexpr int kWordsAt = kRingAt + (kK + kV) * kTileBytes;
  static constexpr int kScaleBytes = kScaleSlots * 3 * kTileScales * 4;
  static_assert(kK + 3 <= kScaleSlots, "slots");
  // of a row, [segment parity]: its factor, its first and last key + 1
  static constexpr int kRowBytes = 2 * kRows * 12;
  static constexpr int kJoinBytes = 2 * 5 * RG * 4;    // words of rows: of each warp, of all
  static constexpr int kSmem = kWordsAt + 512 + kScaleBytes + kRowBytes + kJoinBytes;
  static_assert(kSmem <= 115712, "shared memory of two CTAs an SM");
  static constexpr uint32_t kIdescS = idesc_e4m3_f32(kKeys, kN1);
  static constexpr uint32_t kIdescO = idesc_e4m3_f32(kD, kN2) | (1u << 15);   // A is MN-major
};

struct Bars {
  uint64_t full[6], empty[6];                          // tiles: keys, then values
  // by parity of the CTA's tile counter, whose next bit is then the phase
  uint64_t s_full[2], s_free[2], p_ready[2], pv_done[2];
  uint64_t q_ready, done[2];
  uint32_t tmem;
  int abort;
  int spoilt;                                          // some sum is not finite
  int r;                                               // where the CTA starts
  long long tile;
  Request rq;
};
static_assert(sizeof(Bars) <= 512, "barriers");

// 128-key tiles of a request: [t0, t1), empty without new tokens.  A request whose rows
// see nothing still gets one tile, so that its rows are written.
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

// A CTA's walk over its segments: request r, key head h, keys that any row sees.
struct Walk {
  int r, h;
  Request rq;
  Span sp;
  int kbeg, kend;
  __device__ __forceinline__ void load(const AttnArgs& a, int request) {
    r = request;
    set(a, load_request(a.batch, a.cache.page_shift, r, a.status));
  }
  __device__ __forceinline__ void set(const AttnArgs& a, const Request& request) {
    rq = request;
    sp = tiles_of(rq, a.window);
    kbeg = first_key(rq.pos0, a.window);
    kend = min(rq.len, rq.pos0 + rq.n);
  }
  // (only called while tiles are left; false if the batch ends all the same)
  __device__ __forceinline__ bool next(const AttnArgs& a, int step) {
    if ((h += step) < a.cache.heads) return true;
    h %= step;
    do {
      if (r + 1 >= a.batch.batch) return false;
      load(a, r + 1);
    } while (sp.t1 == sp.t0);
    return true;
  }
};

// Byte offset of byte c of row r of a tile of 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return r * 128 + (((c >> 4) ^ (r & 7)) << 4) + (c & 15);
}

__device__ __forceinline__ void tmem_ld_x4(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x4(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};"
               ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
// N columns (a multiple of 4) from taddr on; nothing uses them before they are there.
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) tmem_ld_x4(taddr + i, r + i);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Barrier of a group's 128 threads; whether any of them says yes.
__device__ __forceinline__ bool group_any(int group, bool yes) {
  int any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 q, %1, 0;\n\t"
      "bar.red.or.pred p, %2, 128, q;\n\t"
      "selp.s32 %0, 1, 0, p;\n\t}"
      : "=r"(any) : "r"(static_cast<int>(yes)), "r"(1 + group) : "memory");
  return any != 0;
}
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}

// RG values of each lane joined over the warp: the result of row lane / (32 / RG) in each.
// (Lanes exchange halves of what they hold: RG + 4 - log2 RG exchanges, and as many fewer
// instructions to fetch, where each value by itself takes 5 RG.)
template <int RG, typename Op>
__device__ __forceinline__ float join_rows(const float (&x)[RG], Op op) {
  const int lane = threadIdx.x & 31;
  float v[RG];
#pragma unroll
  for (int r = 0; r < RG; ++r) v[r] = x[r];
#pragma unroll
  for (int h = RG / 2, o = 16; o > 0; h /= 2, o /= 2) {
    if (h > 0) {
      const bool upper = (lane & o) != 0;
#pragma unroll
      for (int r = 0; r < h; ++r) {
        const float keep = upper ? v[r + h] : v[r], send = upper ? v[r] : v[r + h];
        v[r] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, send, o));
      }
    } else {
      v[0] = op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], o));
    }
  }
  return v[0];
}

// Two fp16 as E4M3 (satfinite, nearest even), the lower one in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2_f16x2(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}

template <int RG>
__global__ void __launch_bounds__(kThreads, 2)
attention_keys_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<RG>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {                 // the swizzle goes by the address
    record_status(a.status, kErrBounds);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kWordsAt);
  float* scales = reinterpret_cast<float*>(smem + C::kWordsAt + 512);   // [slot][3][kTileScales]
  float* row_factor = scales + kScaleSlots * 3 * kTileScales;           // [parity][kRows]
  int* row_lo = reinterpret_cast<int*>(row_factor + 2 * C::kRows);
  int* row_hi = row_lo + 2 * C::kRows;
  float* join = reinterpret_cast<float*>(row_hi + 2 * C::kRows);        // [group][5][RG]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == kThreads - 32) {                  // (a warp that has no request as a rule)
    for (int i = 0; i < C::kK + C::kV; ++i) {
      // (and the loader's lanes that bring scales)
      mbar_init(&bars->full[i], i < C::kK ? 1 + 2 * kTileScales : 1);
      mbar_init(&bars->empty[i], 1);
    }
    mbar_init(&bars->q_ready, kSoftmaxThreads);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 2);                  // (and the scales made ready)
      mbar_init(&bars->s_free[i], kSoftmaxThreads);
      mbar_init(&bars->p_ready[i], kSoftmaxThreads);
      mbar_init(&bars->pv_done[i], 1);
      mbar_init(&bars->done[i], 1);
    }
    bars->abort = 0;
    bars->spoilt = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
  }
  pdl_trigger();
  pdl_wait();                                          // for what came before

  // ---- this CTA's share of the tiles: of the even or of the odd heads, if there are as
  // many of both (two CTAs that start together then read the halves of the same 256 bytes
  // of a tokens-first cache), which the CTAs `me` of [0, ctas) and of [ctas, 2 ctas) take
  const int step = a.cache.heads % 2 == 0 ? 2 : 1, ctas = static_cast<int>(gridDim.x) / step;
  const int side = step == 2 ? static_cast<int>(blockIdx.x & 1u) : 0;
  const int share = static_cast<int>(blockIdx.x) / step, me = share + side * ctas;
  long long* scan = reinterpret_cast<long long*>(smem);           // [kThreads / 32] warp sums
  const int per = (a.batch.batch + kThreads - 1) / kThreads;
  const int r_begin = min(a.batch.batch, static_cast<int>(threadIdx.x) * per);
  const int r_end = min(a.batch.batch, r_begin + per);
  long long mine = 0;
  Request rq;                                          // of this thread, where it has one
  for (int r = r_begin; r < r_end; ++r) {
    rq = load_request(a.batch, a.cache.page_shift, r, a.status);
    const Span s = tiles_of(rq, a.window);
    mine += static_cast<long long>(s.t1 - s.t0) * (a.cache.heads / step);
  }
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const int takers = share_takers(total, ctas);
  AttnPiece* piece = a.pieces + me;
  if (share >= takers) {
    if (threadIdx.x == 0) piece->rows = 0;
    return;
  }
  const long long lo = share_begin(total, share, takers);
  const long long hi = share_begin(total, share + 1, takers);
  long long first = before + upto - mine;
  if (lo >= first && lo < first + mine) {
    int r = r_begin;
    while (true) {
      if (per > 1) rq = load_request(a.batch, a.cache.page_shift, r, a.status);
      const Span s = tiles_of(rq, a.window);
      const long long c = static_cast<long long>(s.t1 - s.t0) * (a.cache.heads / step);
      if (lo < first + c || r + 1 >= r_end) break;
      first += c;
      ++r;
    }
    bars->rq = rq;
    bars->r = r;
    bars->tile = lo - first;
  }
  if (warp == kIssueS) {
    tmem_alloc(&bars->tmem, kTmemColumns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  volatile int* abort = &bars->abort;
  const int group = static_cast<int>(a.group.d);
  Walk wk;
  const auto start = [&] {                             // the first tile
    wk.r = bars->r;
    wk.set(a, bars->rq);
    const int span = max(1, wk.sp.t1 - wk.sp.t0);
    const long long tile = bars->tile;
    const int k = tile >> 32 == 0 ? static_cast<int>(static_cast<uint32_t>(tile) / static_cast<uint32_t>(span))
                                  : static_cast<int>(tile / span);
    wk.h = k * step + side;
    return wk.sp.t0 + static_cast<int>(tile - static_cast<long long>(k) * span);
  };
  int t = start();
  long long left = hi - lo;

  if (warp == kLoadK || warp == kLoadV) {
    // ---- key or value tiles: lane = box (page part) ----
    const bool keys = warp == kLoadK;
    const CUtensorMap* map = keys ? &map_k : &map_v;
    uint64_t* full = bars->full + (keys ? 0 : C::kK);
    uint64_t* empty = bars->empty + (keys ? 0 : C::kK);
    uint8_t* base = smem + C::kRingAt + (keys ? 0 : C::kK * kTileBytes);
    const int box = min(kKeys, 1 << a.cache.page_shift);
    const uint64_t policy = policy_evict_first();
    // Scales: lanes 8-15 bring those of keys, 16-23 those of values, of 16 keys each,
    // without waiting for them.  (Brought through registers, one tile ahead, a tile took
    // the time of a load from HBM: 192 us instead of 141, 64 tokens on up to 16384 keys.)
    const bool brings = keys && lane >= 8 && lane < 24;
    const int off = brings ? (lane & 7) * 16 : lane * box, span = brings ? 16 : box;
    const float* side = lane < 16 ? a.cache.k_scale : a.cache.v_scale;
    // Page numbers: 32 at a time, a lane each, the next ones while these are used.
    const int box_shift = min(7, a.cache.page_shift);
    const auto pages_from = [&](int chunk) {
      const int64_t i = int64_t{chunk} * 32 + lane;
      return i << a.cache.page_shift < wk.kend ? a.batch.page_table[wk.r * a.batch.max_pages + i] : -1;
    };
    const int bufs = keys ? C::kK : C::kV;
    int buf = 0;
    uint32_t phase = 0, tiles = 0;
    bool ok = true;
    while (left > 0 && ok) {
      const int stop = static_cast<int>(min(static_cast<long long>(wk.sp.t1), t + left));
      left -= stop - t;
      int chunk = t * kKeys >> a.cache.page_shift >> 5;
      int ids = pages_from(chunk), more_ids = pages_from(chunk + 1);
      for (; t < stop; ++t, ++tiles) {
        const int key0 = t * kKeys, key = key0 + off;
        if (key0 >> a.cache.page_shift >> 5 != chunk) {
          ids = more_ids;
          more_ids = pages_from(++chunk + 1);
        }
        const int page = __shfl_sync(0xFFFFFFFFu, ids, key >> a.cache.page_shift & 31);
        const bool take = off < kKeys && key < wk.kend && key + span > wk.kbeg;
        const bool there = page >= 0 && page < a.cache.num_pages;
        const int loads = max(0, (min(kKeys, max(0, wk.kend - key0)) + box - 1 >> box_shift) -
                                     (max(0, wk.kbeg - key0) >> box_shift));
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&empty[buf], phase ^ 1u, a.status, abort));
        if (!ok) break;
        if (lane == 0)
          mbar_arrive_expect_tx(&full[buf], static_cast<uint32_t>(loads * box * kD));
        if (brings) {
          const int64_t from = take && there ? page * int64_t{a.cache.heads} + wk.h : 0;
          cp_async_4(scales + tiles % kScaleSlots * (3 * kTileScales) + lane - 8, side + from,
                     take && there);
          cp_async_arrive(&full[buf]);
        } else if (take) {
          if (!there) record_status(a.status, kErrBadIndex);
          tma_load_4d(base + buf * kTileBytes + off * kD, map, 0,
                      key & ((1 << a.cache.page_shift) - 1), wk.h,
                      there ? page : static_cast<int>(a.cache.num_pages),   // past the map: zeros
                      &full[buf], policy);
        }
        if (++buf == bufs) {
          buf = 0;
          phase ^= 1u;
        }
      }
      if (left > 0) {
        if (!wk.next(a, step)) break;
        t = wk.sp.t0;
      }
    }
    if (keys) cp_async_wait_all();
  } else if (warp >= kIssueS) {
    // ---- products ----
    const bool keys = warp == kIssueS;
    uint64_t* full = bars->full + (keys ? 0 : C::kK);
    uint64_t* empty = bars->empty + (keys ? 0 : C::kK);
    const uint64_t tile_desc =
        smem_desc(smem_u32(smem + C::kRingAt + (keys ? 0 : C::kK * kTileBytes)), 16, 1024, 2);
    const uint64_t row_desc = smem_desc(smem_u32(smem + (keys ? C::kQAt : C::kPAt)), 16, 1024, 2);
    const int bufs = keys ? C::kK : C::kV;
    int buf = 0;
    uint32_t phase = 0, q_phase = 0, n = 0;
    while (left > 0) {
      const int stop = static_cast<int>(min(static_cast<long long>(wk.sp.t1), t + left));
      left -= stop - t;
      const int j0 = t;
      if (keys) {
        mbar_wait(&bars->q_ready, q_phase, a.status, abort);
        q_phase ^= 1u;
      }
      for (; t < stop; ++t, ++n) {
        const uint32_t sb = n & 1u, parity = (n >> 1) & 1u;
        const uint64_t desc = tile_desc + static_cast<uint32_t>(buf) * (kTileBytes >> 4);
        mbar_wait(&full[buf], phase, a.status, abort);
        if (keys) {
          mbar_wait(&bars->s_free[sb], parity ^ 1u, a.status, abort);   // S (n - 2) is in registers
          tc_fence_after();
          if (lane == 0) {
#pragma unroll
            for (int ks = 0; ks < kD / 32; ++ks)
              mma_f8(tmem + sb * C::kN1, desc + (ks * 32 >> 4), row_desc + (ks * 32 >> 4),
                     C::kIdescS, ks != 0);
            tc_commit(&bars->s_full[sb]);
          }
          // while they run: the keys' scales, and the values' as logarithms and inverted
          float* sc = scales + n % kScaleSlots * (3 * kTileScales) + (lane & 7);
          if (lane < 8) {
            sc[0] = page_scale(sc[0]);
          } else if (lane < 16) {
            const float log_scale = __log2f(page_scale(sc[kTileScales]));
            sc[kTileScales] = log_scale;
            sc[2 * kTileScales] = exp2_approx(-log_scale);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->s_full[sb]);
        } else {
          mbar_wait(&bars->p_ready[sb], parity, a.status, abort);
          tc_fence_after();
          if (lane == 0) {
#pragma unroll
            for (int ks = 0; ks < kKeys / 32; ++ks)
              mma_f8(tmem + C::kTmemO, desc + ks * (32 * kD >> 4),
                     row_desc + ((sb * C::kPBytes + ks * 32) >> 4), C::kIdescO,
                     t != j0 || ks != 0);
            tc_commit(&bars->pv_done[sb]);
          }
        }
        if (lane == 0) tc_commit(&empty[buf]);
        if (++buf == bufs) {
          buf = 0;
          phase ^= 1u;
        }
      }
      if (left > 0) {
        if (!wk.next(a, step)) break;
        t = wk.sp.t0;
      }
    }
    // every arrival that the tensor cores still owe the barriers
    if (lane == 0) tc_commit(&bars->done[keys]);
    mbar_wait(&bars->done[keys], 0, a.status, abort);
  } else {
    // ---- softmax: group g has the rows g * RG .., a thread a key (and a dimension) ----
    const int g = warp >> 2, key = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float* my_join = join + g * 5 * RG;                // a word of each warp and row
    float* inverse = my_join + 4 * RG;                 // of the rows' weight sums
    constexpr int kRowLanes = 32 / RG;                 // that join_rows leaves a row
    bool begun = false;
    uint32_t n = 0;                                    // tiles so far
    int seg = 0;                                       // parity of the segment
    int stop = 0, rows = 0, slot = 0;
    bool whole = false;
    // the segment: queries to shared memory, D / 8 lanes a row (the last S with the
    // previous ones has landed)
    const auto open = [&] {
      stop = static_cast<int>(min(static_cast<long long>(wk.sp.t1), t + left));
      whole = t == wk.sp.t0 && stop == wk.sp.t1;
      slot = t == wk.sp.t0 ? 1 : 0;                    // a cut segment: begun here, or before
      left -= stop - t;
      rows = wk.rq.n * group;                          // <= kRows, checked on the host
      if (threadIdx.x == 0 && !whole && slot == 1) {
        // this CTA begins a cut segment: where its pieces end, for the join
        const long long end = hi + (wk.sp.t1 - stop);
        int last = share + 1;
        while (last + 1 < takers && share_begin(total, last + 1, takers) < end) ++last;
        AttnPiece p;
        p.rows = rows;
        p.head = wk.h;
        p.first = wk.rq.first;
        p.row0 = 0;
        p.last = last + side * ctas;
        *piece = p;
        begun = true;
      }
      seg ^= 1;
      // scores in powers of two, 2^-7 of a row's factor
      const float c = a.scale * 1.4426950408889634f * 0.0078125f;
      constexpr int kLanes = kD / 8, kStep = kSoftmaxThreads / kLanes;
      const int ch = threadIdx.x & (kLanes - 1);
      static_assert(C::kRows <= kStep, "a row for each group of lanes");
      const int row = threadIdx.x / kLanes;
      if (row < C::kRows) {
        const int tok = a.group(row);
        uint4 u = make_uint4(0, 0, 0, 0);
        if (row < rows)
          u = *reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(a.q.data) + (wk.rq.first + tok) * a.q.token_stride +
              (wk.h * group + row - tok * group) * a.q.head_stride + ch * 8);
        float x[8], most = 0.0f;
        bf16x8_to_float(u, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) most = fmaxf(most, fabsf(x[k]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
          most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
        // 2^(134 - e), and 2^(e - 127) * 2^-7 to undo it; rows of zeros stay as they are,
        // infinities become NaN
        int e = static_cast<int>(__float_as_uint(most) >> 23);
        const bool finite = e != 255;
        e = e == 0 || e == 255 ? 127 : min(max(e, 8), 253);
        const float up = __uint_as_float(static_cast<uint32_t>(261 - e) << 23);
        uint32_t hi8[2], lo8[2];
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
          float y[4], z[4];
#pragma unroll
          for (int d = 0; d < 4; ++d) y[d] = finite ? x[k + d] * up : x[k + d] - x[k + d];
          hi8[k >> 2] = pack_e4m3x2(y[0], y[1]) | pack_e4m3x2(y[2], y[3]) << 16;
#pragma unroll
          for (int d = 0; d < 4; d += 2) {
            const uint32_t h = e4m3x2_to_f16x2(hi8[k >> 2] >> (d * 8));
            const float2 f = __half22float2(reinterpret_cast<const __half2&>(h));
            z[d] = y[d] - f.x;
            z[d + 1] = y[d + 1] - f.y;
          }
          lo8[k >> 2] = pack_e4m3x2(z[0], z[1]) | pack_e4m3x2(z[2], z[3]) << 16;
        }
        uint8_t* to = smem + C::kQAt + tile_at(row, ch * 8);
        *reinterpret_cast<uint2*>(to) = make_uint2(hi8[0], hi8[1]);
        *reinterpret_cast<uint2*>(to + C::kQBytes) = make_uint2(lo8[0], lo8[1]);
        if (ch == 0) {
          // (finite and not 0 once the scale of a page comes in)
          const int at = seg * C::kRows + row, pos = wk.rq.pos0 + tok;
          row_factor[at] = fminf(
              fmaxf(c * __uint_as_float(static_cast<uint32_t>(e) << 23), 0x1p-86f), 0x1p86f);
          row_lo[at] = first_key(pos, a.window);
          row_hi[at] = min(pos + 1, wk.rq.len);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars->q_ready);
    };
    bool more = true;
    open();
    while (more) {
      float m[RG], l[RG];                              // m: 0 until a key has been seen
      float above[RG];                                 // where the reference has to move
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        m[r] = l[r] = 0.0f;
        above[r] = -3.0e38f;
      }
      const int words = seg * C::kRows + g * RG;       // this group's, of the segment
      // keys that every row sees
      const int all_hi = min(wk.rq.pos0 + 1, wk.rq.len);
      const int all_lo = first_key(wk.rq.pos0 + wk.rq.n - 1, a.window);
      const int j0 = t;
      for (; t < stop; ++t, ++n) {
        const uint32_t sb = n & 1u, parity = (n >> 1) & 1u;
        const int at = t * kKeys + key;                // this thread's key
        mbar_wait(&bars->s_full[sb], parity, a.status, abort);
        __syncwarp();
        tc_fence_after();
        uint32_t s[RG], s_lo[RG];
#pragma unroll
        for (int i = 0; i < RG; i += 4) tmem_ld_x4(tmem + sb * C::kN1 + g * RG + i + lanes, s + i);
        tmem_ld_n<RG>(tmem + sb * C::kN1 + C::kRows + g * RG + lanes, s_lo);
#pragma unroll
        for (int r = 0; r < RG; ++r) asm volatile("" : "+r"(s[r]));
        tc_fence_before();
        mbar_arrive(&bars->s_free[sb]);
        const float* sc = scales + n % kScaleSlots * (3 * kTileScales) + (key >> 4);
        const float ks = sc[0], lift = sc[kTileScales], inv_scale = sc[2 * kTileScales];
        // (S follows the arrivals of all that wrote the queries and the rows' words)
        float y[RG];
        bool over = false;
#pragma unroll
        for (int r = 0; r < RG; ++r)
          y[r] = fmaf(__uint_as_float(s[r]) + __uint_as_float(s_lo[r]), row_factor[words + r] * ks, lift);
        if (t * kKeys + kKeys > all_hi || t * kKeys < all_lo) {
#pragma unroll
          for (int r = 0; r < RG; ++r)
            if (at >= row_hi[words + r] || at < row_lo[words + r]) y[r] = -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < RG; ++r) over = over || y[r] > above[r];
        if (group_any(g, over)) {
          // ---- new references: the rows' maxima over the tile ----
          const float warp_top = join_rows<RG>(y, [](float a, float b) { return fmaxf(a, b); });
          if (lane % kRowLanes == 0) my_join[(warp & 3) * RG + lane / kRowLanes] = warp_top;
          group_sync(g);
          float f[RG];
#pragma unroll
          for (int r = 0; r < RG; ++r) {
            const float top = fmaxf(fmaxf(my_join[r], my_join[RG + r]),
                                    fmaxf(my_join[2 * RG + r], my_join[3 * RG + r]));
            f[r] = 1.0f;
            if (top > above[r]) {
              const float mn = top;
              f[r] = above[r] == -3.0e38f ? 0.0f : exp2_approx(m[r] - mn);
              m[r] = mn;
              above[r] = mn + kSlack;
              l[r] *= f[r];
            }
          }
          if (t > j0) {                                // O^T holds tiles up to t - 1
            if (n > 1) mbar_wait(&bars->pv_done[sb], parity ^ 1u, a.status, abort);
            mbar_wait(&bars->pv_done[sb ^ 1u], ((n - 1) >> 1) & 1u, a.status, abort);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int level = 0; level < kLevels; ++level) {
              const uint32_t to = tmem + C::kTmemO + level * C::kRows + g * RG + lanes;
              uint32_t o[RG];
              tmem_ld_n<RG>(to, o);
#pragma unroll
              for (int r = 0; r < RG; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * f[r]);
#pragma unroll
              for (int r = 0; r < RG; r += 4) tmem_st_x4(to + r, o + r);
            }
            tmem_st_wait();
          }
          group_sync(g);                               // before the words are written again
        }
        float p[RG];
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          p[r] = exp2_approx(y[r] - m[r]);
          l[r] = fmaf(p[r], inv_scale, l[r]);
        }
        // P V (n - 2) has read its weights
        if (n > 1) mbar_wait(&bars->pv_done[sb], parity ^ 1u, a.status, abort);
        uint8_t* to = smem + C::kPAt + sb * C::kPBytes;
#pragma unroll
        for (int r = 0; r < RG; r += 2) {
          // 2^11 p of two rows as fp16; what a number leaves of it is exact
          const uint32_t w = pack_f16x2(p[r] * 2048.0f, p[r + 1] * 2048.0f);
          __half2 x = reinterpret_cast<const __half2&>(w);
          const int row = g * RG + r;
          const uint32_t at0 = tile_at(row, key), at1 = tile_at(row + 1, key);
#pragma unroll
          for (int level = 0; level < kLevels; ++level) {
            const float up = level == 0 ? 0x1p-11f : (level == 1 ? 0x1p-3f : (level == 2 ? 0x1p5f : 0x1p13f));
            const __half2 y = __hmul2(x, __float2half2_rn(up));
            const uint32_t e = pack_e4m3x2_f16x2(reinterpret_cast<const uint32_t&>(y));
            to[level * C::kRows * 128 + at0] = static_cast<uint8_t>(e);
            to[level * C::kRows * 128 + at1] = static_cast<uint8_t>(e >> 8);
            const uint32_t back = e4m3x2_to_f16x2(e);
            x = __hfma2(reinterpret_cast<const __half2&>(back), __float2half2_rn(-1.0f / up), x);
          }
        }
        if (g == 0 && (t * kKeys < wk.kbeg || (t + 1) * kKeys > wk.kend)) {
          // values that no row sees may hold anything: make them zeros
          mbar_wait(&bars->full[C::kK + n % C::kV], (n / C::kV) & 1u, a.status, abort);
          if (at < wk.kbeg || at >= wk.kend) {
            uint8_t* v = smem + C::kRingAt + (C::kK + n % C::kV) * kTileBytes + key * kD;
#pragma unroll
            for (int i = 0; i < kD; i += 16) *reinterpret_cast<uint4*>(v + i) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&bars->p_ready[sb]);
      }
      // ---- weight sums over the threads, a thread's for its row ----
      const int64_t po = (2 * static_cast<int64_t>(me) + slot) * a.piece_rows;
      {
        const float warp_sum = join_rows<RG>(l, [](float a, float b) { return a + b; });
        if (lane % kRowLanes == 0) my_join[(warp & 3) * RG + lane / kRowLanes] = warp_sum;
        group_sync(g);
        const int row = g * RG + key;
        if (key < RG && row < rows) {
          const float sum = (my_join[key] + my_join[RG + key]) + (my_join[2 * RG + key] + my_join[3 * RG + key]);
          float mr = -INFINITY;                        // no key seen, as where pieces are joined
#pragma unroll
          for (int r = 0; r < RG; ++r)
            if (r == key && above[r] != -3.0e38f) mr = m[r];
          inverse[key] = sum == 0.0f ? 0.0f : 1.0f / sum;
          if (!whole) {
            a.piece_ml[po + row] = make_float2(mr, sum);
          } else if (a.lse != nullptr) {
            const int tok = a.group(row);
            a.lse[(wk.rq.first + tok) * a.q.heads + wk.h * group + row - tok * group] = lse_of(mr, sum);
          }
        }
        group_sync(g);
      }
      // ---- the next segment's queries, then this one's rows ----
      const Walk out_wk = wk;
      const int out_rows = rows;
      const bool to_out = whole;
      const uint32_t last = n - 1;
      more = left > 0 && wk.next(a, step);
      if (more) {
        t = wk.sp.t0;
        open();
      }
      mbar_wait(&bars->pv_done[last & 1u], (last >> 1) & 1u, a.status, abort);
      __syncwarp();
      tc_fence_after();
      float o[RG];
#pragma unroll
      for (int level = kLevels - 1; level >= 0; --level) {
        uint32_t x[RG];
        tmem_ld_n<RG>(tmem + C::kTmemO + level * C::kRows + g * RG + lanes, x);
#pragma unroll
        for (int r = 0; r < RG; ++r)
          o[r] = level == kLevels - 1 ? __uint_as_float(x[r])
                                      : fmaf(o[r], 0.00390625f, __uint_as_float(x[r]));
      }
      tc_fence_before();
      float probe = 0.0f;                              // NaN if some sum is not finite
      const int tok0 = a.group(g * RG);
      int of_group = g * RG - tok0 * group;            // the row's query head, of the key head's
      __nv_bfloat16* to_row = static_cast<__nv_bfloat16*>(a.out.data) +
                              (out_wk.rq.first + tok0) * a.out.token_stride +
                              (out_wk.h * group + of_group) * a.out.head_stride + key;
      float* to_piece = a.piece_o + (po + g * RG) * kD + key;
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        if (g * RG + r >= out_rows) break;
        probe = fmaf(o[r], 0.0f, probe);
        if (to_out)
          *to_row = __float2bfloat16_rn(o[r] * inverse[r]);
        else
          to_piece[r * kD] = o[r];
        to_row += a.out.head_stride;
        if (++of_group == group) {
          of_group = 0;
          to_row += a.out.token_stride - group * a.out.head_stride;
        }
      }
      if (probe != 0.0f) bars->spoilt = 1;
    }
    if (threadIdx.x == 0 && !begun) piece->rows = 0;
    asm volatile("bar.sync 3, %0;" ::"n"(kSoftmaxThreads) : "memory");
    if (bars->spoilt != 0) {
      // ---- rows that hidden keys may have spoilt: the same walk again ----
      t = start();
      for (left = hi - lo; left > 0; t = wk.sp.t0) {
        const int end = static_cast<int>(min(static_cast<long long>(wk.sp.t1), t + left));
        const bool all = t == wk.sp.t0 && end == wk.sp.t1;
        left -= end - t;
        const int64_t at =
            (2 * static_cast<int64_t>(me) + (t == wk.sp.t0 ? 1 : 0)) * a.piece_rows;
        mend_rows<kD, true, true>(a, wk.r, wk.h, 0, wk.rq.n * group, wk.kbeg, wk.kend, t, end,
                                  all ? nullptr : a.piece_o + at * kD, a.piece_ml + at, warp,
                                  kSoftmaxThreads / 32);
        if (left > 0 && !wk.next(a, step)) break;
      }
    }
  }
  __syncthreads();
  drain_after_abort(abort);
  if (warp == kIssueS) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemColumns);
  }
}

template <int RG>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int grid,
                   cudaStream_t stream) {
  static PerDeviceOnce once;
  using C = Cfg<RG>;
  auto kernel = attention_keys_kernel<RG>;
  cudaError_t e = set_smem_attr_once(once, reinterpret_cast<const void*>(kernel), C::kSmem);
  if (e != cudaSuccess) return e;
  // its start overlaps the end of the kernel before
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, mk, mv);
}

}  // namespace

cudaError_t launch_attention_keys(const AttnArgs& a, const CUtensorMap& map_k,
                                  const CUtensorMap& map_v, int grid, cudaStream_t stream) {
  if (a.piece_rows <= Cfg<4>::kRows) return launch<4>(a, map_k, map_v, grid, stream);
  return launch<8>(a, map_k, map_v, grid, stream);
}

}  // namespace nvmoe
