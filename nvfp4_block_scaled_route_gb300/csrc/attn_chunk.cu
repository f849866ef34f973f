// Paged attention of chunks of new tokens on the tcgen05 tensor cores.
//
// The rows of a request and key head -- new tokens x query heads of the key
// head, token-major -- are taken in blocks of 128 by a CTA.  (Clusters of two CTAs
// that share each key and value tile by multicast took 6 of 629 us off 2048 new
// tokens of 16384 and 9 of 90 off 16 requests of 280 rows, and cost 3 of 217 on 4 x
// 512 on an E4M3 cache; but loads of that kind stay out of a library that processes
// on several GPUs load.)
//
// Per 128 keys a CTA runs two products of 128 x 128 x D and 128 x 128
// exponentials (4 * rows * keys * D flops in all).  The softmax is the bound: its
// chain takes a warp 1750 cycles a tile, the products 1024 of the tensor pipe, which
// is two thirds busy.  2048 new tokens over 16384 keys, 56 query and 8 key heads of
// 128: 668 us, 1.35 PFLOP/s (up to 680 by box).
//
//   S = Q K^T       both from shared memory (K-major), into TMEM
//   P = 2^(cS - m)  TMEM -> registers -> 16 bits -> TMEM
//   O += P V        P from TMEM, V from shared memory (MN-major)
//
// TMEM holds S and P twice: while the softmax of tile j is computed, the tensor
// cores run P V (j - 1) and S (j + 1).  (Two query tiles of 128-wide heads in one CTA
// would fill TMEM with one S, P in its place, and one O each, and the pipe would wait
// for every softmax.)  The next segment's queries go in before a segment's rows go out,
// so that its first scores are computed meanwhile.
//
// Roles: warps 0-7 hold the softmax, a row's keys 0-63 and 64-127 in two
// threads that exchange maxima through shared memory; warps 8 and 9 load key
// and value tiles by TMA (one box per page) into a ring each; warps 10 and 11
// issue the MMAs of S and of P V.  (One warp for both did not keep the pipe
// fed: an MMA of 128 x 128 x 16 takes 64 cycles and few are queued, while a
// tile's four commits and three waits take some 600.)
//
// E4M3 caches: the keys go to the tensor cores as they are, and a query as the
// sum of two E4M3 numbers, S = Qhi K^T + Qlo K^T, at twice the rate of 16-bit
// products.  A query row is scaled by a power of two to a maximum in [128, 256),
// and the factor goes back in with the softmax scale; the two hold the 8 bits of
// its elements exactly down to 2^-9 of the maximum, smaller ones to within
// 2^-17 of it.  The values are turned into fp16 (exact) by four warps on their
// way from a ring of raw tiles to a ring of operand tiles, for weights in fp16.
// (Keys converted likewise, by two of the four warps: 248.6 us where this takes
// 233.5 us, 4 requests of up to 512 new tokens.)
//
// m is a reference, not always the maximum: O is rescaled only when a row's
// maximum has grown by more than 2^8 over its reference (any reference gives
// the same quotient; weights stay below 2^8, sums are fp32).  E4M3 caches, whose
// weights are fp16: the reference is 2^10 below the maximum and moves when the maximum
// has grown by more than 2^5, so that weights stay below 2^15 and have all their bits
// down to 2^-24 of the largest, those of bf16 down to 2^-27.  (With the reference at
// the maximum, weights would lose bits below 2^-14 of it and be 0 below 2^-25, which
// all the others' are beside one key 18 nats above them.  4 x 512 new tokens on up to
// 9000 keys, growth of 2 / 3 / 4 / 5 / 6 / 8: 260 / 247 / 230 / 219.5 / 217 / 216.5 us.)
//
// The work is the flat list of 128-key tiles of all (request, key head, row
// block) segments, causal limits taken off; CTA c of G takes a run of it of
// equal cost, and attn_combine_kernel joins the segments cut by a border.  Where
// the runs start is found by each CTA itself for up to kAttnPlanHere requests and
// row blocks (16 requests of 35 rows 30.2 us, 34.0 with a launch for it), else by
// attn_plan_kernel.
#include "attn.cuh"

namespace nvmoe {
namespace {

constexpr int kKeys = kAttnTileKeys;
constexpr int kTile = kAttnTileRows;         // query rows of a tile
constexpr int kLoadK = 8, kLoadV = 9, kIssueS = 10;   // and 11: P V
constexpr int kConvert = 12;                 // warps 12-15: values to fp16 (E4M3)
constexpr int kSoftmaxThreads = 256;
constexpr int kConvertThreads = 128;
// E4M3: registers of a thread; the launch gives each 128 (the most for 512
// threads), the softmax warps take what the others leave.  (168 and 88: the
// others' loops spill, 252 us instead of 233.5.)
constexpr int kRegsSoftmax = 152, kRegsOther = 104;
static_assert(256 * kRegsSoftmax + 256 * kRegsOther <= 128 * 512, "registers");
// Powers of two by which a row's reference stands below its maximum when it is set,
// and by which the maximum may grow over that before the reference moves.
template <bool FP8>
constexpr float kLift = FP8 ? 10.0f : 0.0f;
template <bool FP8>
constexpr float kSlack = FP8 ? 5.0f : 8.0f;
constexpr int kPlanThreads = 1024;
// What a segment costs beside its tiles (its queries in, a first tile without
// anything to overlap, its rows out), in tiles, when the work is shared out.
// Measured, 0 / 2 / 4 / 6 tiles: 4 requests of 512 new tokens on an E4M3 cache
// 234.6 / 225.5 / 216.8 / 214.7 us, 6 windowed prompts of 64-wide heads
// 91.7 / 88.4 / 89.9 / 89.7, 16 requests of 5 drafted tokens
// 32.9 / 30.1 / 30.3 / 30.8, 2048 new tokens of 16384 678 / 680 / 678 / 682.
constexpr int kSegmentTiles = 4;
static_assert(kMaxGrid < kPlanThreads && kMaxGrid < 384, "a thread for each start");

// Rows [row0, row0 + rows) of a request and the key tiles that they see.
struct Block {
  int row0, rows;
  int t0, t1;                                // tiles of the segment (at least one)
  int kbeg, kend;                            // keys that any row sees; none if kend is 0
};
__device__ __forceinline__ Block block_of(const Request& q, const FastDiv& group, int window,
                                          int p) {
  Block b;
  b.row0 = p * kTile;
  b.rows = min(kTile, q.n * static_cast<int>(group.d) - b.row0);
  b.t0 = b.kbeg = b.kend = 0;
  b.t1 = 1;                                  // nothing seen: a tile all the same, rows get zeros
  const int first = q.pos0 + group(b.row0);
  const int last = q.pos0 + group(b.row0 + b.rows - 1);
  const int end = min(q.len, last + 1);
  const int beg = first_key(first, window);
  if (end > beg) {
    b.t0 = beg / kKeys;
    b.t1 = (end + kKeys - 1) / kKeys;
    b.kbeg = beg;
    b.kend = end;
  }
  return b;
}
__device__ __forceinline__ int blocks_of(const Request& q, int group) {
  return static_cast<int>((static_cast<int64_t>(q.n) * group + kTile - 1) / kTile);
}

// Sum of the values of the threads before this one; *total: of all.
template <int THREADS>
__device__ __forceinline__ long long block_scan(long long v, long long* sums, long long* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long s = lane < THREADS / 32 ? sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  *total = sums[31];
  return x - v + (warp > 0 ? sums[warp - 1] : 0);
}

// The largest i in [lo, hi) with f(i) <= x, f ascending, f(lo) <= x.
template <typename F>
__device__ __forceinline__ int last_le(int lo, int hi, long long x, F f) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (f(mid) <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Prefix sums of the blocks of the requests (block0) and of the cost of the
// blocks in tiles (cost0, one key head), then where each of the G CTAs of the
// attention kernel starts.  Called by all THREADS > G threads of a
// CTA; thread c returns the start of c.
struct PlanShared {
  long long sums[32];
  long long tile_of[kMaxGrid + 1];           // of all tiles, a CTA's first
  long long cut_end[kMaxGrid + 1];           // ... the end of the segment that it is inside of
};
template <int THREADS>
__device__ __forceinline__ AttnStart plan(const AttnArgs& a, int G, PlanShared* sh, int* block0,
                                          long long* cost0) {
  const int B = a.batch.batch, group = static_cast<int>(a.group.d);
  long long total = 0, blocks = 0;
  for (int r0 = 0; r0 < B; r0 += THREADS) {
    const int r = r0 + threadIdx.x;
    int n = 0;
    if (r < B) n = blocks_of(load_request(a.batch, a.cache.page_shift, r, a.status), group);
    const long long at = blocks + block_scan<THREADS>(n, sh->sums, &total);
    if (r < B) block0[r] = static_cast<int>(min(at, static_cast<long long>(a.max_blocks)));
    blocks += total;
  }
  blocks = min(blocks, static_cast<long long>(a.max_blocks));
  if (threadIdx.x == 0) block0[B] = static_cast<int>(blocks);
  __syncthreads();
  long long units = 0;
  for (int i0 = 0; i0 < blocks; i0 += THREADS) {
    const int i = i0 + threadIdx.x;
    int n = 0;
    if (i < blocks) {
      const int r = last_le(0, B, i, [&](int k) { return block0[k]; });
      const Request rq = load_request(a.batch, a.cache.page_shift, r, a.status);
      const Block b = block_of(rq, a.group, a.window, i - block0[r]);
      n = b.t1 - b.t0 + kSegmentTiles;
    }
    const long long at = units + block_scan<THREADS>(n, sh->sums, &total);
    if (i < blocks) cost0[i] = at;
    units += total;
  }
  if (threadIdx.x == 0) cost0[blocks] = units;
  __syncthreads();
  const long long total_units = units * a.cache.heads;
  const long long total_tiles = total_units - kSegmentTiles * blocks * a.cache.heads;
  const int takers = share_takers(total_units, G);
  AttnStart s = {};
  const int c = threadIdx.x;
  if (c <= G) {
    const long long x = c < takers ? share_begin(total_units, c, takers) : total_units;
    long long first = total_tiles, end = total_tiles;
    if (x < total_units) {
      const auto base = [&](int k) { return cost0[block0[k]] * a.cache.heads; };
      const int r = last_le(0, B, x, base);            // (the last of equals has blocks)
      const int b0 = block0[r], b1 = block0[r + 1];
      const long long u0 = cost0[b0], per = cost0[b1] - u0;
      const long long y = x - u0 * a.cache.heads;
      if (per > 0 && y >= 0 && y / per < a.cache.heads) {    // (not if q_start descends)
        s.request = r;
        s.head = static_cast<int>(y / per);
        const long long z = y - s.head * per + u0;
        const int b = last_le(b0, b1, z, [&](int k) { return cost0[k]; });
        const long long ub = cost0[b];
        s.block = b - b0;
        s.tile = max(0, static_cast<int>(z - ub) - kSegmentTiles);
        const long long segments =
            static_cast<long long>(b0) * a.cache.heads + s.head * (b1 - b0) + s.block;
        first = u0 * a.cache.heads + s.head * per + ub - u0 - kSegmentTiles * segments;
        end = first + (s.tile > 0 ? cost0[b + 1] - ub - kSegmentTiles : 0);
        first += s.tile;
      }
    }
    sh->tile_of[c] = first;
    sh->cut_end[c] = end;
  }
  __syncthreads();
  if (c < G) {
    s.left = sh->tile_of[c + 1] - sh->tile_of[c];
    s.last = c + 1;
    while (s.last + 1 < G && sh->tile_of[s.last + 1] < sh->cut_end[c + 1]) ++s.last;
  }
  return s;
}

__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const AttnArgs a, int G) {
  __shared__ PlanShared sh;
  pdl_trigger();
  const AttnStart s = plan<kPlanThreads>(a, G, &sh, a.plan_block0, a.plan_cost0);
  if (static_cast<int>(threadIdx.x) < G) a.starts[threadIdx.x] = s;
}

// A CTA's walk over its segments.
struct Walk {
  int r, h, p, blocks;
  Request rq;
  Block b;
  __device__ __forceinline__ void load(const AttnArgs& a, int group, int request) {
    r = request;
    rq = load_request(a.batch, a.cache.page_shift, r, a.status);
    blocks = blocks_of(rq, group);
  }
  // (only called while tiles are left; false if the batch ends all the same)
  __device__ __forceinline__ bool next(const AttnArgs& a, int group) {
    if (++p >= blocks) {
      p = 0;
      if (++h >= a.cache.heads) {
        h = 0;
        do {
          if (r + 1 >= a.batch.batch) return false;
          load(a, group, r + 1);
        } while (blocks == 0);
      }
    }
    b = block_of(rq, a.group, a.window, p);
    return true;
  }
};

template <int D, bool FP8>
struct Cfg {
  static constexpr int kThreads = FP8 ? 512 : 384;
  static constexpr int kBytes = kKeys * D * 2;         // an operand tile
  static constexpr int kLoadBytes = FP8 ? kKeys * D : kBytes;   // a tile as loaded
  static constexpr int kRow = D * (FP8 ? 1 : 2);
  static constexpr int kLine = kRow < 128 ? kRow : 128;   // bytes of a box row
  static constexpr int kHalves = kRow / kLine;         // column blocks
  // tiles of keys (as loaded), operand tiles of values (bf16: as loaded), raw
  // tiles of E4M3 values
  static constexpr int kK = (FP8 ? 4 : 3) * (D == 128 ? 1 : 2), kV = 3 * (D == 128 ? 1 : 2);
  static constexpr int kRaw = FP8 ? (D == 128 ? 2 : 5) : 0;
  static constexpr int kVAt = kBytes;                  // after the queries: values, keys, raw
  static constexpr int kKAt = kVAt + kV * kBytes, kRawAt = kKAt + kK * kLoadBytes;
  static constexpr int kRing = kRawAt + kRaw * kLoadBytes;
  static constexpr int kSmem = kRing + 512 + 5 * kTile * 4;
  static_assert(kSmem <= 232448, "shared memory");
  static constexpr uint32_t kTmemO = 256, kTmemP = 384;   // S: columns 0 and 128
  // instruction descriptors: fp16 operands are format 0, bf16 format 1; V is MN-major
  static constexpr uint32_t kFormats = FP8 ? (1u << 7) | (1u << 10) : 0u;
  static constexpr uint32_t kIdescS =
      FP8 ? idesc_e4m3_f32(kTile, kKeys) : idesc_bf16_f32(kTile, kKeys);
  static constexpr uint32_t kIdescO = (idesc_bf16_f32(kTile, D) ^ kFormats) | (1u << 16);
};

struct Bars {
  uint64_t full[14], empty[14];                        // loaded tiles: keys, then values
  uint64_t op_full[6], op_empty[6];                    // E4M3: operand tiles of values
  // by parity of the CTA's tile counter, whose next bit is then the phase
  uint64_t s_full[2], s_free[2], p_ready[2], pv_done[2];
  uint64_t q_ready, done[2];
  uint32_t tmem;
  int abort;
  int spoilt;                                          // some sum is not finite
  AttnStart start;
};
static_assert(sizeof(Bars) <= 512, "barriers");

// D[tmem] (+)= A[tmem] x B[smem], 16-bit operands.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Byte offset of 16-byte chunk c of row r of a tile: 128-byte lines, 128-byte
// swizzle, column blocks of 64 elements one after the other.
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return (c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Likewise in an E4M3 tile (K-major for the tensor cores, as TMA writes it: the
// swizzle of 128 bytes, or of 64 where a row has no more).
template <int D>
__device__ __forceinline__ uint32_t raw_at(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::kThreads, 1)
attention_chunk_kernel(const __grid_constant__ AttnArgs a,
                       const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D, FP8>;
  // the swizzle goes by the address: tiles start at multiples of 1024 bytes,
  // and there is no room to round up to one
  extern __shared__ __align__(1024) uint8_t sq[];       // queries, operand tiles, raw tiles
  if ((smem_u32(sq) & 1023u) != 0) {
    record_status(a.status, kErrBounds);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(sq + C::kRing);
  float* swap = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + 512);
  // E4M3: each query row's power of two, [segment parity][row] (a thread may be
  // a segment ahead of another)
  uint8_t* q_exp = reinterpret_cast<uint8_t*>(swap + 4 * kTile);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kK + (FP8 ? C::kRaw : C::kV); ++i) {
      mbar_init(&bars->full[i], 1);
      // the readers: an issuer, or four converting warps
      mbar_init(&bars->empty[i], FP8 && i >= C::kK ? 4 : 1);
    }
    for (int i = 0; FP8 && i < C::kV; ++i) {
      mbar_init(&bars->op_full[i], kConvertThreads);
      mbar_init(&bars->op_empty[i], 1);
    }
    mbar_init(&bars->q_ready, kSoftmaxThreads);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
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
  if (warp == kIssueS) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  volatile int* abort = &bars->abort;
  pdl_trigger();
  pdl_wait();                                          // the plan, or what came before

  if (a.plan_here) {
    PlanShared* sh = reinterpret_cast<PlanShared*>(sq);  // where the queries will be
    long long* cost0 = reinterpret_cast<long long*>(sh + 1);
    int* block0 = reinterpret_cast<int*>(cost0 + kAttnPlanHere + 1);
    static_assert(sizeof(PlanShared) + (kAttnPlanHere + 1) * 12 <= C::kBytes, "room");
    const AttnStart s = plan<C::kThreads>(a, static_cast<int>(gridDim.x), sh, block0, cost0);
    if (threadIdx.x == blockIdx.x) bars->start = s;
    __syncthreads();
  }
  const AttnStart st = a.plan_here ? bars->start : a.starts[blockIdx.x];
  long long left = st.left;
  const int group = static_cast<int>(a.group.d);
  Walk wk;
  int t = 0;
  if (left > 0) {
    wk.load(a, group, st.request);
    wk.h = st.head;
    wk.p = st.block;
    wk.b = block_of(wk.rq, a.group, a.window, wk.p);
    t = wk.b.t0 + st.tile;
  }

  if (warp >= kLoadK) {
    if (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
  if (warp == kLoadK || warp == kLoadV) {
    // ---- key or value tiles: lane = box (page part, column block) ----
    const bool keys = warp == kLoadK;
    const CUtensorMap* map = keys ? &map_k : &map_v;
    const int bufs = keys ? C::kK : (FP8 ? C::kRaw : C::kV);
    const int buf0 = keys ? 0 : C::kK;                  // barriers
    uint8_t* base = sq + (keys ? C::kKAt : (FP8 ? C::kRawAt : C::kVAt));
    const int box = min(kKeys, 1 << a.cache.page_shift);
    const int b = lane & 7, half = lane >> 3;
    const uint64_t policy = policy_evict_normal();
    int buf = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (left > 0 && ok) {
      const int stop = static_cast<int>(min(static_cast<long long>(wk.b.t1), t + left));
      left -= stop - t;
      // the segment's queries to L2, ahead of the softmax warps' loads
      if (keys)
        for (int i = lane; i < wk.b.rows; i += 32) {
          const int r = wk.b.row0 + i, k = a.group(r);
          const __nv_bfloat16* q =
              static_cast<const __nv_bfloat16*>(a.q.data) + (wk.rq.first + k) * a.q.token_stride +
              (wk.h * group + r - k * group) * a.q.head_stride;
#pragma unroll
          for (int d = 0; d < D; d += 64)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q + d));
        }
      for (; t < stop; ++t) {
        const int key = t * kKeys + b * box;
        const bool take = b * box < kKeys && half < C::kHalves && key < wk.b.kend &&
                          key + box > wk.b.kbeg;
        int page = 0;
        if (take) {
          page = a.batch.page_table[wk.r * a.batch.max_pages + (key >> a.cache.page_shift)];
          if (page < 0 || page >= a.cache.num_pages) {
            record_status(a.status, kErrBadIndex);
            page = static_cast<int>(a.cache.num_pages);       // past the map: zeros
          }
        }
        const int loads = C::kHalves * boxes_of(t * kKeys, box, wk.b.kbeg, wk.b.kend);
        const int in_page = key & ((1 << a.cache.page_shift) - 1);
        const int n = buf0 + buf;
        // (nothing here joins the lanes again: in a failing CTA some may go on)
        ok = mbar_wait(&bars->empty[n], phase ^ 1u, a.status, abort);
        if (!ok) break;
        if (lane == 0)
          mbar_arrive_expect_tx(&bars->full[n], static_cast<uint32_t>(loads * box * C::kLine));
        if (take) {
          uint8_t* dst = base + buf * C::kLoadBytes + half * kKeys * C::kLine + b * box * C::kLine;
          const int x = half * (FP8 ? C::kLine : C::kLine / 2);
          tma_load_4d(dst, map, x, in_page, wk.h, page, &bars->full[n], policy);
        }
        if (++buf == bufs) {
          buf = 0;
          phase ^= 1u;
        }
      }
      if (left > 0) {
        if (!wk.next(a, group)) break;
        t = wk.b.t0;
      }
    }
  } else if (FP8 && warp >= kConvert) {
    // ---- E4M3 values to fp16: 16 bytes at a time, eight rows of one column side
    // by side (no bank conflicts either way) ----
    constexpr int kChunks = D / 16;                     // of a row
    constexpr int kStepRows = kConvertThreads / kChunks, kSteps = kKeys / kStepRows;
    const int thread = threadIdx.x & (kConvertThreads - 1);
    const int ch = (thread >> 3) % kChunks, row0 = (thread & 7) + (thread >> 3) / kChunks * 8;
    // (a step's rows are a multiple of 8 on: the swizzles stay)
    const uint32_t src0 = raw_at<D>(row0, ch);
    const uint32_t dst0 = tile_at(row0, 2 * ch), dst1 = tile_at(row0, 2 * ch + 1);
    int in = 0, out = 0;
    uint32_t in_phase = 0, out_phase = 0;
    while (left > 0) {
      const int stop = static_cast<int>(min(static_cast<long long>(wk.b.t1), t + left));
      left -= stop - t;
      for (; t < stop; ++t) {
        mbar_wait(&bars->full[C::kK + in], in_phase, a.status, abort);
        mbar_wait(&bars->op_empty[out], out_phase ^ 1u, a.status, abort);
        const uint8_t* src = sq + C::kRawAt + in * C::kLoadBytes + src0;
        uint8_t* dst = sq + C::kVAt + out * C::kBytes;
        // values that no row sees may hold anything: make them zeros
        const int lo = wk.b.kbeg - t * kKeys, hi = wk.b.kend - t * kKeys;
        const bool cut = lo > 0 || hi < kKeys;
        uint4 u[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          u[i] = *reinterpret_cast<const uint4*>(src + i * kStepRows * D);
        if (cut)
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            const int row = row0 + i * kStepRows;
            if (row < lo || row >= hi) u[i] = make_uint4(0, 0, 0, 0);
          }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          uint8_t* to = dst + i * kStepRows * 128;
          *reinterpret_cast<uint4*>(to + dst0) =
              make_uint4(e4m3x2_to_f16x2(u[i].x), e4m3x2_to_f16x2(u[i].x >> 16),
                         e4m3x2_to_f16x2(u[i].y), e4m3x2_to_f16x2(u[i].y >> 16));
          *reinterpret_cast<uint4*>(to + dst1) =
              make_uint4(e4m3x2_to_f16x2(u[i].z), e4m3x2_to_f16x2(u[i].z >> 16),
                         e4m3x2_to_f16x2(u[i].w), e4m3x2_to_f16x2(u[i].w >> 16));
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars->op_full[out]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->empty[C::kK + in]);   // this warp has read the raw tile
        if (++in == C::kRaw) {
          in = 0;
          in_phase ^= 1u;
        }
        if (++out == C::kV) {
          out = 0;
          out_phase ^= 1u;
        }
      }
      if (left > 0) {
        if (!wk.next(a, group)) break;
        t = wk.b.t0;
      }
    }
  } else {
    // ---- MMAs ----
    const bool keys = warp == kIssueS;
    const int bufs = keys ? C::kK : C::kV;
    const bool made = FP8 && !keys;                     // tiles of the converting warps
    uint64_t* full = made ? bars->op_full : bars->full + (keys ? 0 : C::kK);
    uint64_t* empty = made ? bars->op_empty : bars->empty + (keys ? 0 : C::kK);
    const uint32_t tile_bytes = keys ? C::kLoadBytes : C::kBytes;
    // A tile's descriptors are this one plus multiples of 16 bytes (building
    // each anew takes the issuing thread longer than the MMA does the pipe).
    // (E4M3 of 64 dimensions: rows of 64 bytes, the 64-byte swizzle)
    constexpr bool kShort = C::kRow < 128;
    const uint64_t desc0 =
        keys ? smem_desc(smem_u32(sq + C::kKAt), 16, kShort ? 512 : 1024, kShort ? 4 : 2)
             : smem_desc(smem_u32(sq + C::kVAt), kKeys * 128, 1024, 2);
    const uint64_t q_desc = smem_desc(smem_u32(sq), 16, kShort ? 512 : 1024, kShort ? 4 : 2);
    int buf = 0;
    uint32_t phase = 0, q_phase = 0;
    uint32_t n = 0;                                     // tiles so far
    while (left > 0) {
      const int stop = static_cast<int>(min(static_cast<long long>(wk.b.t1), t + left));
      left -= stop - t;
      const int j0 = t;
      const bool seen = wk.b.kend > 0;
      if (keys && seen) {
        mbar_wait(&bars->q_ready, q_phase, a.status, abort);
        q_phase ^= 1u;
      }
      for (; t < stop; ++t) {
        const uint32_t sb = n & 1u, parity = (n >> 1) & 1u;
        const uint64_t desc = desc0 + static_cast<uint32_t>(buf) * (tile_bytes >> 4);
        mbar_wait(&full[buf], phase, a.status, abort);
        if (keys) {
          if (seen) {
            // S (n - 2) is in registers
            mbar_wait(&bars->s_free[sb], parity ^ 1u, a.status, abort);
            tc_fence_after();
            if (lane == 0) {
              if (FP8) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {   // Qhi, then Qlo
                  const int part = ks / (D / 32), at = ks % (D / 32) * 32;
                  mma_f8(tmem + sb * 128, q_desc + ((part * kTile * D + at) >> 4),
                         desc + (at >> 4), C::kIdescS, ks != 0);
                }
              } else {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                  mma_f16(tmem + sb * 128,
                          q_desc + (((ks >> 2) * (kTile * 128) + (ks & 3) * 32) >> 4),
                          desc + (((ks >> 2) * (kKeys * 128) + (ks & 3) * 32) >> 4), C::kIdescS,
                          ks != 0);
              }
              tc_commit(&bars->s_full[sb]);
            }
          }
        } else {
          if (!FP8 && (t * kKeys < wk.b.kbeg || (t + 1) * kKeys > wk.b.kend)) {
            // values that no row sees may hold anything: make them zeros
            for (int i = lane; i < kKeys * (D / 8); i += 32) {
              const int row = i / (D / 8), key = t * kKeys + row;
              if (key < wk.b.kbeg || key >= wk.b.kend)
                *reinterpret_cast<uint4*>(sq + C::kVAt + buf * C::kBytes +
                                          tile_at(row, i % (D / 8))) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (seen) {
            mbar_wait(&bars->p_ready[sb], parity, a.status, abort);
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
              for (int ks = 0; ks < kKeys / 16; ++ks)
                mma_f16_ts(tmem + C::kTmemO, tmem + C::kTmemP + sb * 64 + ks * 8,
                           desc + ks * (2048 >> 4), C::kIdescO, t != j0 || ks != 0);
              tc_commit(&bars->pv_done[sb]);
            }
          }
        }
        if (lane == 0) tc_commit(&empty[buf]);
        if (seen) ++n;
        if (++buf == bufs) {
          buf = 0;
          phase ^= 1u;
        }
      }
      if (left > 0) {
        if (!wk.next(a, group)) break;
        t = wk.b.t0;
      }
    }
    // every arrival that the tensor cores still owe the barriers
    if (lane == 0) tc_commit(&bars->done[keys]);
    mbar_wait(&bars->done[keys], 0, a.status, abort);
  }
  } else {
    // ---- softmax: a row's keys 0-63 and 64-127 in two threads ----
    if (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int half = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + half * 64 + lanes;                     // this thread's scores,
    const uint32_t tp = tmem + C::kTmemP + half * 32 + lanes;         // weights,
    const uint32_t to = tmem + C::kTmemO + half * (D / 2) + lanes;    // output columns
    const int pair_bar = 1 + (warp & 3);                              // the two warps of 32 rows
    // words of a row's two threads: [tile parity][half][row].  A tile's word has
    // been read once its thread has met the other one at the next tile's.
    float* mine = swap + half * kTile + row;
    const float* other = swap + (half ^ 1) * kTile + row;
    AttnPiece* piece = a.pieces + blockIdx.x;
    bool begun = false;
    // 32-byte stores of the output rows
    const bool wide = ((reinterpret_cast<uintptr_t>(a.out.data) | a.out.token_stride * 2 |
                        a.out.head_stride * 2) & 31) == 0;
    uint32_t n = 0;                                     // tiles so far
    // the segment: its tiles in this CTA, this thread's row
    int stop = 0, j0 = 0, rows = 0, row0 = 0, tok = 0, head = 0, slot = 0;
    int64_t tk = 0;
    // sees: some row sees a key; busy: some row of this warp is real
    bool sees = false, whole = false, busy = false;
    float c = 0.0f;                                     // scores in powers of two
    int seg = 0;                                        // parity of the queries' segment
    const auto open = [&] {
      stop = static_cast<int>(min(static_cast<long long>(wk.b.t1), t + left));
      whole = t == wk.b.t0 && stop == wk.b.t1;
      slot = t == wk.b.t0 ? 1 : 0;
      left -= stop - t;
      rows = wk.b.rows;
      j0 = t;
      sees = wk.b.kend > 0;
      row0 = wk.b.row0;
      busy = (warp & 3) * 32 < rows;
      const int my = row0 + min(row, rows - 1);  // rows past the end act as the last
      tok = a.group(my);
      tk = wk.rq.first + tok;
      head = wk.h * group + my - tok * group;
      if (threadIdx.x == 0 && !whole && slot == 1) {
        // this CTA begins a cut segment: where its pieces end, for the join
        AttnPiece p;
        p.rows = wk.b.rows;
        p.head = wk.h;
        p.first = wk.rq.first;
        p.row0 = wk.b.row0;
        p.last = st.last;
        *piece = p;
        begun = true;
      }
      c = a.scale * 1.4426950408889634f;
      if (FP8) c *= 0.0078125f * (a.cache.k_scale != nullptr ? a.cache.k_scale[wk.h] : 1.0f);
      if (!sees) return;
      seg ^= 1;
      // the queries, D / 8 lanes a row (the last S with the previous ones has landed)
      constexpr int kLanes = D / 8, kStep = kSoftmaxThreads / kLanes;
      const int ch = threadIdx.x & (kLanes - 1), i0 = threadIdx.x / kLanes;
      uint4 u[kTile / kStep];
#pragma unroll
      for (int i = 0; i < kTile / kStep; ++i) {
        u[i] = make_uint4(0, 0, 0, 0);
        if (i0 + i * kStep < rows) {
          const int r = row0 + i0 + i * kStep, k = a.group(r);
          u[i] = *reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(a.q.data) + (wk.rq.first + k) * a.q.token_stride +
              (wk.h * group + r - k * group) * a.q.head_stride + ch * 8);
        }
      }
#pragma unroll
      for (int i = 0; i < kTile / kStep; ++i) {
        if (FP8) {
          float x[8], most = 0.0f;
          bf16x8_to_float(u[i], x);
#pragma unroll
          for (int k = 0; k < 8; ++k) most = fmaxf(most, fabsf(x[k]));
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1)
            most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
          // 2^(134 - e), and 2^(e - 127) * 2^-7 to undo it (2^-7 is in c); rows of
          // zeros stay as they are, infinities become NaN
          int e = static_cast<int>(__float_as_uint(most) >> 23);
          const bool finite = e != 255;
          e = e == 0 || e == 255 ? 127 : min(max(e, 8), 253);
          const float up = __uint_as_float(static_cast<uint32_t>(261 - e) << 23);
          if (ch == 0) q_exp[seg * kTile + i0 + i * kStep] = static_cast<uint8_t>(e);
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int k = 0; k < 8; k += 4) {
            float y[4], z[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) y[d] = finite ? x[k + d] * up : x[k + d] - x[k + d];
            hi[k >> 2] = pack_e4m3x2(y[0], y[1]) | pack_e4m3x2(y[2], y[3]) << 16;
#pragma unroll
            for (int d = 0; d < 4; d += 2) {
              const uint32_t h = e4m3x2_to_f16x2(hi[k >> 2] >> (d * 8));
              const float2 f = __half22float2(reinterpret_cast<const __half2&>(h));
              z[d] = y[d] - f.x;
              z[d + 1] = y[d + 1] - f.y;
            }
            lo[k >> 2] = pack_e4m3x2(z[0], z[1]) | pack_e4m3x2(z[2], z[3]) << 16;
          }
          uint8_t* to = sq + raw_at<D>(i0 + i * kStep, ch >> 1) + (ch & 1) * 8;
          *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(to + kTile * D) = make_uint2(lo[0], lo[1]);
        } else {
          *reinterpret_cast<uint4*>(sq + tile_at(i0 + i * kStep, ch)) = u[i];
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars->q_ready);
    };
    bool more = left > 0;
    if (more) open();
    while (more) {
      float m = -INFINITY, l = 0.0f;
      if (sees) {
        float cr = c;
        const int seg_now = seg;
        const int pos = wk.rq.pos0 + tok;
        const int vis_hi = min(pos + 1, wk.rq.len) - half * 64;
        const int vis_lo = first_key(pos, a.window) - half * 64;
        // keys that every row of the warp sees (rows come in order)
        const int all_hi = __shfl_sync(0xFFFFFFFFu, vis_hi, 0);
        const int all_lo = __shfl_sync(0xFFFFFFFFu, vis_lo, 31);
        for (int j = j0; j < stop; ++j, ++n) {
          const uint32_t sb = n & 1u;
          mbar_wait(&bars->s_full[sb], (n >> 1) & 1u, a.status, abort);
          // (S follows the arrivals of all that wrote the queries and their factors)
          if (FP8 && j == j0)
            // (not 0, which would make NaN of the -inf of a hidden key)
            cr = fmaxf(0x1p-126f,
                       c * __uint_as_float(static_cast<uint32_t>(q_exp[seg_now * kTile + row])
                                           << 23));
          if (!busy) {                                  // what these rows hold is not used
            mbar_arrive(&bars->s_free[sb]);
            if (n > 1) mbar_wait(&bars->pv_done[sb], ((n - 2) >> 1) & 1u, a.status, abort);
            mbar_arrive(&bars->p_ready[sb]);
            continue;
          }
          __syncwarp();
          tc_fence_after();
          uint32_t s[2][32];
          tmem_ld_32x32b_x32(ts + sb * 128, s[0]);
          tmem_ld_32x32b_x32(ts + sb * 128 + 32, s[1]);
          tmem_ld_wait();
          tc_fence_before();
          mbar_arrive(&bars->s_free[sb]);
          if (j * kKeys + 64 > all_hi) {
            const int h = vis_hi - j * kKeys;
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= h) s[i >> 5][i & 31] = 0xFF800000u;              // -inf
          }
          if (j * kKeys < all_lo) {
            const int lw = vis_lo - j * kKeys;
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i < lw) s[i >> 5][i & 31] = 0xFF800000u;
          }
          float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 64; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              t4[k] = max3(t4[k], __uint_as_float(s[i >> 5][(i & 31) + 2 * k]),
                           __uint_as_float(s[i >> 5][(i & 31) + 2 * k + 1]));
          float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
          mine[sb * 2 * kTile] = top;
          asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
          top = fmaxf(top, other[sb * 2 * kTile]) * cr;
          // a new reference where some row's maximum has left the old one behind
          if (__any_sync(0xFFFFFFFFu, top > m + (kLift<FP8> + kSlack<FP8>))) {
            const float mn = fmaxf(m, top - kLift<FP8>);
            if (j > j0) {
              // O holds P V up to tile j - 1.  (That P V (n - 2) is done says that
              // the other barrier's phase is that of tile n - 1.)
              if (n > 1) mbar_wait(&bars->pv_done[sb], ((n - 2) >> 1) & 1u, a.status, abort);
              mbar_wait(&bars->pv_done[sb ^ 1u], ((n - 1) >> 1) & 1u, a.status, abort);
              __syncwarp();
              tc_fence_after();
              const float f = exp2_approx(m - (mn == -INFINITY ? 0.0f : mn));
              l *= f;
#pragma unroll 1
              for (int i = 0; i < D / 2; i += 16) {
                uint32_t o[16];
                tmem_ld_32x32b_x16(to + i, o);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st_32x32b_x16(to + i, o);
              }
            }
            m = mn;
          }
          const float use = m == -INFINITY ? 0.0f : m;  // a row without keys so far
          uint64_t sum[2] = {0, 0};
          const uint64_t c2 = f32x2(cr, cr), use2 = f32x2(-use, -use);
          uint32_t p[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            float x, y;
            f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[k >> 4][(2 * k) & 31]),
                                        __uint_as_float(s[k >> 4][(2 * k + 1) & 31])), c2, use2),
                        x, y);
            x = exp2_approx(x);
            y = exp2_approx(y);
            sum[k & 1] = add_f32x2(sum[k & 1], f32x2(x, y));
            p[k] = FP8 ? pack_f16x2(x, y) : pack_bf16x2(x, y);
          }
          if (n > 1) {                                  // P V (n - 2) has read its weights
            mbar_wait(&bars->pv_done[sb], ((n - 2) >> 1) & 1u, a.status, abort);
            __syncwarp();
            tc_fence_after();
          }
          tmem_st_32x32b_x32(tp + sb * 64, p);
          float s0, s1;
          f32x2_split(add_f32x2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&bars->p_ready[sb]);
        }
      }
      // ---- the next segment's queries, then this one's rows ----
      const bool seen = sees, real = row < rows, live = busy, to_out = whole;
      const int64_t tk_out = tk;
      const int head_out = head;
      const int64_t at = (2 * static_cast<int64_t>(blockIdx.x) + slot) * kTile + row;
      const float v_scale =
          FP8 && a.cache.v_scale != nullptr ? a.cache.v_scale[wk.h] : 1.0f;
      const uint32_t end = n - 1;                       // the last tile
      more = left > 0;
      if (more) {
        more = wk.next(a, group);
        t = wk.b.t0;
      }
      if (more) open();
      if (!live) continue;
      if (seen) {
        mbar_wait(&bars->pv_done[end & 1u], (end >> 1) & 1u, a.status, abort);
        __syncwarp();
        tc_fence_after();
        // the row's other sum.  (All have read the words of the last tile, whose
        // P V is done; the next tile's are the others.)
        mine[((n + 1) & 1u) * 2 * kTile] = l;
        asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
        l += other[((n + 1) & 1u) * 2 * kTile];
      }
      // (a tile that saw no key here: zeros)
      const float inv = l == 0.0f ? 0.0f : v_scale / l;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) + tk_out * a.out.token_stride +
                           head_out * a.out.head_stride + half * (D / 2);
      float probe = 0.0f;                               // NaN if some sum is not finite
#pragma unroll 1
      for (int i = 0; i < D / 2; i += 32) {
        uint32_t o[32];
        __syncwarp();
        if (seen) {
          tmem_ld_32x32b_x32(to + i, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) probe = fmaf(__uint_as_float(o[k]), 0.0f, probe);
        if (real && to_out) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          if (wide) {
#pragma unroll
            for (int k = 0; k < 16; k += 8) {
              const uint32_t v[8] = {w[k],     w[k + 1], w[k + 2], w[k + 3],
                                     w[k + 4], w[k + 5], w[k + 6], w[k + 7]};
              st_global_v8_b32(out + i + 2 * k, v);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<uint4*>(out + i + 2 * k) =
                  make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
          }
        } else if (real) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            const uint32_t v[8] = {o[k],     o[k + 1], o[k + 2], o[k + 3],
                                   o[k + 4], o[k + 5], o[k + 6], o[k + 7]};
            st_global_v8_b32(a.piece_o + at * D + half * (D / 2) + i + k, v);
          }
        }
      }
      if (real && probe != 0.0f) bars->spoilt = 1;
      if (real && half == 0) {
        if (!to_out) a.piece_ml[at] = make_float2(m, l);
        else if (a.lse != nullptr) a.lse[tk_out * a.q.heads + head_out] = lse_of(m, l);
      }
      tc_fence_before();
    }
    if (threadIdx.x == 0 && !begun) piece->rows = 0;
    tc_fence_before();
    asm volatile("bar.sync 9, %0;" ::"n"(kSoftmaxThreads) : "memory");
    if (bars->spoilt != 0 && st.left > 0) {
      // ---- rows that hidden keys may have spoilt: the same walk again ----
      wk.load(a, group, st.request);
      wk.h = st.head;
      wk.p = st.block;
      wk.b = block_of(wk.rq, a.group, a.window, wk.p);
      t = wk.b.t0 + st.tile;
      for (left = st.left; left > 0; t = wk.b.t0) {
        const int stop = static_cast<int>(min(static_cast<long long>(wk.b.t1), t + left));
        const bool whole = t == wk.b.t0 && stop == wk.b.t1;
        left -= stop - t;
        const int64_t at =
            (2 * static_cast<int64_t>(blockIdx.x) + (t == wk.b.t0 ? 1 : 0)) * kTile;
        mend_rows<D, FP8>(a, wk.r, wk.h, wk.b.row0, wk.b.rows, wk.b.kbeg, wk.b.kend, t, stop,
                  whole ? nullptr : a.piece_o + at * D, a.piece_ml + at, warp,
                  kSoftmaxThreads / 32);
        if (left > 0 && !wk.next(a, group)) break;
      }
    }
  }
  __syncthreads();
  drain_after_abort(abort);
  if (warp == kIssueS) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool FP8>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int grid,
                   cudaStream_t stream) {
  static PerDeviceOnce once;
  using C = Cfg<D, FP8>;
  auto kernel = attention_chunk_kernel<D, FP8>;
  cudaError_t e = set_smem_attr_once(once, reinterpret_cast<const void*>(kernel), C::kSmem);
  if (e != cudaSuccess) return e;
  // its prologue overlaps the plan; it waits for the plan before it reads anything
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, mk, mv);
}

}  // namespace

cudaError_t launch_attn_plan(const AttnArgs& a, int grid, cudaStream_t stream) {
  attn_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, grid);
  return cudaGetLastError();
}

cudaError_t launch_attention_chunk(const AttnArgs& a, const CUtensorMap& map_k,
                                   const CUtensorMap& map_v, int grid, cudaStream_t stream) {
  if (a.cache.fp8)
    return a.cache.head_dim == 128 ? launch<128, true>(a, map_k, map_v, grid, stream)
                                   : launch<64, true>(a, map_k, map_v, grid, stream);
  return a.cache.head_dim == 128 ? launch<128, false>(a, map_k, map_v, grid, stream)
                                 : launch<64, false>(a, map_k, map_v, grid, stream);
}

}  // namespace nvmoe
