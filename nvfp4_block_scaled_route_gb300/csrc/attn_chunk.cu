// Paged attention of chunks of new tokens on the tcgen05 tensor cores.
//
// The rows of a request and key head -- new tokens x query heads of the key
// head, token-major -- are taken in blocks of 256 by a cluster of two CTAs, a
// tile of 128 rows each, which share every key and value tile: each CTA loads
// half of its pages and multicasts them to both.  Per 128 keys a CTA runs two
// products of 128 x 128 x D and 128 x 128 exponentials; the tensor pipe is the
// bound (4 * rows * keys * D flops).
//
//   S = Q K^T       Q from TMEM, K from shared memory (K-major), into TMEM
//   P = 2^(cS - m)  TMEM -> registers -> 16 bits -> TMEM, over S
//   O += P V        P from TMEM, V from shared memory (MN-major)
//
// TMEM holds S twice: while the softmax of tile j is computed, the tensor
// cores run P V (j - 1) and S (j + 1).  (Two query tiles in one CTA would fill
// TMEM with one S and O each, and the pipe would wait for every softmax.)
//
// Roles: warps 0-7 hold the softmax, a row's keys 0-63 and 64-127 in two
// threads that exchange maxima through shared memory; warps 8 and 9 load key
// and value tiles by TMA (one box per page) into a ring each; warps 10 and 11
// issue the MMAs of S and of P V.  (One warp for both did not keep the pipe
// fed: an MMA of 128 x 128 x 16 takes 64 cycles and few are queued, while a
// tile's four commits and three waits take some 600.)
//
// m is a reference, not always the maximum: O is rescaled only when a row's
// maximum has grown by more than 2^8 over its reference (any reference gives
// the same quotient; weights stay below 2^8, sums are fp32).
//
// The work is the flat list of 128-key tiles of all (request, key head, row
// block) segments, causal limits taken off; cluster c of G takes an equal run
// of it (attn_plan_kernel finds where it starts), and attn_combine_kernel
// joins the segments cut by a border.
#include "attn.cuh"

namespace nvmoe {
namespace {

constexpr int kKeys = kAttnTileKeys;
constexpr int kTile = 128;                   // query rows of a tile
constexpr int kBlock = kAttnBlockRows;       // rows of a segment
constexpr int kLoadK = 8, kLoadV = 9, kIssueS = 10, kIssueO = 11;
constexpr int kThreads = 384;
constexpr int kSoftmaxThreads = 256;
constexpr int kPlanThreads = 1024;

// Rows [row0, row0 + rows) of a request and the key tiles that they see.
struct Block {
  int row0, rows;
  int t0, t1;                                // tiles of the segment (at least one)
  int a0[2], a1[2];                          // of each query tile; empty if a1 <= a0
  int kbeg, kend;                            // keys that any row sees
};
__device__ __forceinline__ Block block_of(const Request& q, int group, int window, int p) {
  Block b;
  b.row0 = p * kBlock;
  b.rows = min(kBlock, q.n * group - b.row0);
  b.t0 = b.t1 = b.kbeg = b.kend = 0;
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    b.a0[a] = b.a1[a] = 0;
    const int rows = min(kTile, b.rows - a * kTile);
    if (rows <= 0) continue;
    const int first = q.pos0 + (b.row0 + a * kTile) / group;
    const int last = q.pos0 + (b.row0 + a * kTile + rows - 1) / group;
    const int end = min(q.len, last + 1);
    const int beg = window > 0 ? max(0, first - window + 1) : 0;
    if (end <= beg) continue;
    b.a0[a] = beg / kKeys;
    b.a1[a] = (end + kKeys - 1) / kKeys;
    if (b.t1 == 0) {
      b.t0 = b.a0[a];
      b.kbeg = beg;
    }
    b.t1 = b.a1[a];
    b.kend = end;
  }
  if (b.t1 == 0) b.t1 = 1;                   // nothing seen: a tile all the same, rows get zeros
  return b;
}
__device__ __forceinline__ int blocks_of(const Request& q, int group) {
  return static_cast<int>((static_cast<int64_t>(q.n) * group + kBlock - 1) / kBlock);
}

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
    long long s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  *total = sums[31];
  return x - v + (warp > 0 ? sums[warp - 1] : 0);      // exclusive
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

// One CTA: prefix sums of the blocks of the requests (block0) and of the key
// tiles of the blocks (tile0, one key head), then where each of the G CTAs of
// the attention kernel starts.
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(const AttnArgs a, int G) {
  __shared__ long long sums[32];
  const int B = a.batch.batch, group = a.q.heads / a.cache.heads;
  pdl_trigger();
  long long total = 0, blocks = 0;
  for (int r0 = 0; r0 < B; r0 += kPlanThreads) {
    const int r = r0 + threadIdx.x;
    int n = 0;
    if (r < B) n = blocks_of(load_request(a.batch, a.cache.page_shift, r, a.status), group);
    const long long at = blocks + block_scan(n, sums, &total);
    if (r < B) a.plan_block0[r] = static_cast<int>(min(at, static_cast<long long>(a.max_blocks)));
    blocks += total;
  }
  blocks = min(blocks, static_cast<long long>(a.max_blocks));
  if (threadIdx.x == 0) a.plan_block0[B] = static_cast<int>(blocks);
  __syncthreads();
  long long tiles = 0;
  for (int i0 = 0; i0 < blocks; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int n = 0;
    if (i < blocks) {
      const int r = last_le(0, B, i, [&](int k) { return a.plan_block0[k]; });
      const Request rq = load_request(a.batch, a.cache.page_shift, r, a.status);
      const Block b = block_of(rq, group, a.window, i - a.plan_block0[r]);
      n = b.t1 - b.t0;
    }
    const long long at = tiles + block_scan(n, sums, &total);
    if (i < blocks) a.plan_tile0[i] = at;
    tiles += total;
  }
  if (threadIdx.x == 0) a.plan_tile0[blocks] = tiles;
  __syncthreads();
  total = tiles * a.cache.heads;
  for (int c = threadIdx.x; c < G; c += kPlanThreads) {
    AttnStart s;
    const long long lo = total * c / G;
    s.total = total;
    s.left = total * (c + 1) / G - lo;
    s.request = s.head = s.block = s.tile = 0;
    if (s.left > 0) {
      const auto base = [&](int k) { return a.plan_tile0[a.plan_block0[k]] * a.cache.heads; };
      const int r = last_le(0, B, lo, base);           // (the last of equals has blocks)
      const int b0 = a.plan_block0[r], b1 = a.plan_block0[r + 1];
      const long long t0 = a.plan_tile0[b0], per = a.plan_tile0[b1] - t0;
      const long long y = lo - t0 * a.cache.heads;
      if (per <= 0 || y < 0 || y / per >= a.cache.heads) {   // q_start not ascending
        s.left = 0;
        a.starts[c] = s;
        continue;
      }
      s.request = r;
      s.head = static_cast<int>(y / per);
      const long long z = y - s.head * per + t0;
      const int b = last_le(b0, b1, z, [&](int k) { return a.plan_tile0[k]; });
      s.block = b - b0;
      s.tile = static_cast<int>(z - a.plan_tile0[b]);
    }
    a.starts[c] = s;
  }
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
    b = block_of(rq, group, a.window, p);
    return true;
  }
};

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;               // 128-byte column blocks
  static constexpr int kBytes = kKeys * D * 2;         // a key or value tile
  static constexpr int kBufs = D == 128 ? 7 : 14;
  static constexpr int kKBufs = kBufs - kBufs / 2, kVBufs = kBufs / 2;
  static constexpr int kSmem = kBufs * kBytes + 512 + 2 * kTile * 4;
  static_assert(kSmem <= 232448, "shared memory");
  static constexpr uint32_t kTmemO = 256, kTmemQ = 384;   // S: columns 0 and 128
};

struct Bars {
  uint64_t full[14], empty[14];                        // keys, then values
  // by parity of the CTA's tile counter; its next bit is the barrier's phase
  uint64_t s_full[2], p_ready[2], pv_done[2];
  uint64_t q_ready, done[2];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 512, "barriers");

// One box into the shared memory of both CTAs of the cluster, signalling the
// barrier at the same offset in each.
__device__ __forceinline__ void tma_load_4d_both(void* smem_dst, const CUtensorMap* map, int32_t x,
                                                 int32_t y, int32_t z, int32_t w, uint64_t* bar,
                                                 uint64_t cache_hint) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".multicast::cluster.L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7, %8;"
      ::"r"(smem_u32(smem_dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z),
        "r"(w), "r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3)), "l"(cache_hint)
      : "memory");
}

// tc_commit on the barrier at the same offset in both CTAs.
__device__ __forceinline__ void tc_commit_both(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;"
      ::"r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3)) : "memory");
}

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

// Pairs of fp32 in one register pair (one instruction for both).
__device__ __forceinline__ uint64_t f32x2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attention_chunk_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v) {
  using C = Cfg<D>;
  // the swizzle goes by the address: tiles start at multiples of 1024 bytes,
  // and there is no room to round up to one
  extern __shared__ __align__(1024) uint8_t ring[];
  if ((smem_u32(ring) & 1023u) != 0) {
    record_status(a.status, kErrBounds);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(ring + C::kBufs * C::kBytes);
  float* swap = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + 512);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());   // query tile of the block
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->empty[i], 2);                      // both CTAs' issuers
    }
    mbar_init(&bars->q_ready, kSoftmaxThreads);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_ready[i], kSoftmaxThreads);
      mbar_init(&bars->pv_done[i], 1);
      mbar_init(&bars->done[i], 1);
    }
    bars->abort = 0;
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
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  volatile int* abort = &bars->abort;
  pdl_trigger();
  pdl_wait();                                          // the plan

  const AttnStart st = a.starts[cluster];
  long long left = st.left;
  const int group = a.q.heads / a.cache.heads;
  Walk wk;
  int t = 0;
  if (left > 0) {
    wk.load(a, group, st.request);
    wk.h = st.head;
    wk.p = st.block;
    wk.b = block_of(wk.rq, group, a.window, wk.p);
    t = wk.b.t0 + st.tile;
  }

  if (warp == kLoadK || warp == kLoadV) {
    // ---- this CTA's half (64 keys) of the key or value tiles, to both CTAs:
    // lane = box (page part, column block) ----
    const bool keys = warp == kLoadK;
    const CUtensorMap* map = keys ? &map_k : &map_v;
    const int bufs = keys ? C::kKBufs : C::kVBufs, buf0 = keys ? 0 : C::kKBufs;
    const int box = min(kKeys / 2, 1 << a.cache.page_shift);
    const int b = lane & 7, half = lane >> 3;
    const uint64_t policy = policy_evict_normal();
    int buf = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (left > 0 && ok) {
      const int stop = static_cast<int>(min(static_cast<long long>(wk.b.t1), t + left));
      left -= stop - t;
      for (; t < stop; ++t) {
        const int key = t * kKeys + b * box;
        const bool in = b * box < kKeys && half < C::kHalves && key < wk.b.kend &&
                        key + box > wk.b.kbeg;
        const bool take = in && (b * box >= kKeys / 2) == (rank == 1);
        int page = 0;
        if (take) {
          page = a.batch.page_table[wk.r * a.batch.max_pages + (key >> a.cache.page_shift)];
          if (page < 0 || page >= a.cache.num_pages) {
            record_status(a.status, kErrBadIndex);
            page = static_cast<int>(a.cache.num_pages);       // past the map: zeros
          }
        }
        const int loads = __popc(__ballot_sync(0xFFFFFFFFu, in));
        const int in_page = key & ((1 << a.cache.page_shift) - 1);
        const int n = buf0 + buf;
        ok = mbar_wait(&bars->empty[n], phase ^ 1u, a.status, abort);
        if (!ok) break;
        if (lane == 0)
          mbar_arrive_expect_tx(&bars->full[n], static_cast<uint32_t>(loads * box * 128));
        __syncwarp();
        if (take)
          tma_load_4d_both(ring + n * C::kBytes + half * kKeys * 128 + b * box * 128, map,
                           half * 64, in_page, wk.h, page, &bars->full[n], policy);
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
  } else if (warp == kIssueS || warp == kIssueO) {
    // ---- MMAs ----
    constexpr uint32_t kIdescS = idesc_bf16_f32(kTile, kKeys);
    constexpr uint32_t kIdescO = idesc_bf16_f32(kTile, D) | (1u << 16);     // B is MN-major
    const bool keys = warp == kIssueS;
    const int bufs = keys ? C::kKBufs : C::kVBufs, buf0 = keys ? 0 : C::kKBufs;
    // A tile's descriptors are this one plus multiples of 16 bytes (building
    // each anew takes the issuing thread longer than the MMA does the pipe).
    const uint64_t desc0 = smem_desc(smem_u32(ring + buf0 * C::kBytes),
                                     keys ? 16 : kKeys * 128, 1024, 2);
    int buf = 0;
    uint32_t phase = 0, q_phase = 0;
    uint32_t n = 0;                                     // tiles so far
    while (left > 0) {
      const int stop = static_cast<int>(min(static_cast<long long>(wk.b.t1), t + left));
      left -= stop - t;
      const int j0 = max(t, rank == 0 ? wk.b.a0[0] : wk.b.a0[1]);
      const int j1 = min(stop, rank == 0 ? wk.b.a1[0] : wk.b.a1[1]);
      if (keys && j1 > j0) {
        mbar_wait(&bars->q_ready, q_phase, a.status, abort);
        q_phase ^= 1u;
      }
      for (; t < stop; ++t) {
        const bool mine = t >= j0 && t < j1;
        const uint32_t sb = n & 1u, parity = (n >> 1) & 1u;
        const uint64_t desc = desc0 + static_cast<uint32_t>(buf) * (C::kBytes >> 4);
        mbar_wait(&bars->full[buf0 + buf], phase, a.status, abort);
        if (keys) {
          if (mine) {
            // S goes where P (n - 2) was
            mbar_wait(&bars->pv_done[sb], parity ^ 1u, a.status, abort);
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks)
                mma_f16_ts(tmem + sb * 128, tmem + C::kTmemQ + ks * 8,
                           desc + (((ks >> 2) * (kKeys * 128) + (ks & 3) * 32) >> 4), kIdescS,
                           ks != 0);
              tc_commit(&bars->s_full[sb]);
            }
          }
        } else {
          if (t * kKeys < wk.b.kbeg || (t + 1) * kKeys > wk.b.kend) {
            // values that no row sees may hold anything: make them zeros
            for (int i = lane; i < kKeys * (D / 8); i += 32) {
              const int row = i / (D / 8), key = t * kKeys + row;
              if (key < wk.b.kbeg || key >= wk.b.kend)
                *reinterpret_cast<uint4*>(ring + (buf0 + buf) * C::kBytes +
                                          tile_at(row, i % (D / 8))) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (mine) {
            mbar_wait(&bars->p_ready[sb], parity, a.status, abort);
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
              for (int ks = 0; ks < kKeys / 16; ++ks)
                mma_f16_ts(tmem + C::kTmemO, tmem + sb * 128 + ks * 8,
                           desc + ks * (2048 >> 4), kIdescO, t != j0 || ks != 0);
              tc_commit(&bars->pv_done[sb]);
            }
          }
        }
        if (lane == 0) tc_commit_both(&bars->empty[buf0 + buf]);
        if (mine) ++n;
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
  } else {
    // ---- softmax: a row's keys 0-63 and 64-127 in two threads ----
    const int half = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + half * 64 + lanes;                     // this thread's scores,
    const uint32_t tp = tmem + half * 32 + lanes;                     // weights,
    const uint32_t to = tmem + C::kTmemO + half * (D / 2) + lanes;    // output columns
    const uint32_t tq = tmem + C::kTmemQ + half * (D / 4) + lanes;    // and query columns
    const int pair_bar = 1 + (warp & 3);                              // the two warps of 32 rows
    float* mine = swap + half * kTile + row;
    float* other = swap + (half ^ 1) * kTile + row;
    const long long hi = st.total * (cluster + 1) / clusters;
    uint32_t n = 0;                                     // tiles so far
    AttnPiece* piece = a.pieces + cluster;
    bool begun = false;
    const float c = a.scale * 1.4426950408889634f;      // scores in powers of two
    while (left > 0) {
      const int stop = static_cast<int>(min(static_cast<long long>(wk.b.t1), t + left));
      const bool whole = t == wk.b.t0 && stop == wk.b.t1;
      const int slot = t == wk.b.t0 ? 1 : 0;
      left -= stop - t;
      const int rows = min(kTile, wk.b.rows - rank * kTile);
      const int j0 = max(t, rank == 0 ? wk.b.a0[0] : wk.b.a0[1]);
      const int j1 = min(stop, rank == 0 ? wk.b.a1[0] : wk.b.a1[1]);
      const int row0 = wk.b.row0 + rank * kTile;
      const int my = row0 + min(row, max(rows, 1) - 1);  // rows past the end act as the last
      const int tok = my / group;
      const int64_t tk = wk.rq.first + tok;
      const int head = wk.h * group + my - tok * group;
      float m = -INFINITY, l = 0.0f;
      if (j1 > j0) {
        // this row's half of the query (the last S with the previous ones has landed)
        {
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(a.q.data) + tk * a.q.token_stride +
              head * a.q.head_stride + half * (D / 2));
          uint4 u[D / 16];
#pragma unroll
          for (int i = 0; i < D / 16; ++i) u[i] = src[i];
#pragma unroll
          for (int i = 0; i < D / 16; i += 4) {
            const uint32_t w[16] = {u[i].x, u[i].y, u[i].z, u[i].w,
                                    u[i + 1].x, u[i + 1].y, u[i + 1].z, u[i + 1].w,
                                    u[i + 2].x, u[i + 2].y, u[i + 2].z, u[i + 2].w,
                                    u[i + 3].x, u[i + 3].y, u[i + 3].z, u[i + 3].w};
            tmem_st_32x32b_x16(tq + i * 4, w);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars->q_ready);
        const int pos = wk.rq.pos0 + tok;
        const int vis_hi = min(pos + 1, wk.rq.len) - half * 64;
        const int vis_lo = (a.window > 0 ? pos - a.window + 1 : 0) - half * 64;
        // keys that every row of the tile sees
        const int all_hi = min(wk.rq.pos0 + row0 / group + 1, wk.rq.len);
        const int all_lo =
            a.window > 0 ? wk.rq.pos0 + (row0 + rows - 1) / group - a.window + 1 : 0;
        for (int j = j0; j < j1; ++j, ++n) {
          const uint32_t sb = n & 1u;
          mbar_wait(&bars->s_full[sb], (n >> 1) & 1u, a.status, abort);
          __syncwarp();
          tc_fence_after();
          uint32_t s[2][32];
          tmem_ld_32x32b_x32(ts + sb * 128, s[0]);
          tmem_ld_32x32b_x32(ts + sb * 128 + 32, s[1]);
          tmem_ld_wait();
          if ((j + 1) * kKeys > all_hi || j * kKeys < all_lo) {
            const int h = vis_hi - j * kKeys, lw = vis_lo - j * kKeys;
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= h || i < lw) s[i >> 5][i & 31] = 0xFF800000u;      // -inf
          }
          float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 64; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              t4[k] = max3(t4[k], __uint_as_float(s[i >> 5][(i & 31) + 2 * k]),
                           __uint_as_float(s[i >> 5][(i & 31) + 2 * k + 1]));
          float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
          *mine = top;
          asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
          top = fmaxf(top, *other) * c;
          // a new reference where some row's maximum has left the old one behind
          if (__any_sync(0xFFFFFFFFu, top > m + 8.0f)) {
            const float mn = fmaxf(m, top);
            if (j > j0) {
              // O holds P V up to tile j - 1
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
          const uint64_t c2 = f32x2(c, c), use2 = f32x2(-use, -use);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float x, y;
              f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[i][2 * k]),
                                          __uint_as_float(s[i][2 * k + 1])), c2, use2), x, y);
              x = exp2_approx(x);
              y = exp2_approx(y);
              sum[k & 1] = add_f32x2(sum[k & 1], f32x2(x, y));
              p[k] = pack_bf16x2(x, y);
            }
            tmem_st_32x32b_x16(tp + sb * 128 + i * 16, p);
          }
          float s0, s1;
          f32x2_split(add_f32x2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&bars->p_ready[sb]);
        }
        mbar_wait(&bars->pv_done[(n - 1) & 1u], ((n - 1) >> 1) & 1u, a.status, abort);
        __syncwarp();
        tc_fence_after();
        // the row's other sum
        *mine = l;
        asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
        l += *other;
      }
      // ---- the rows out (a tile that saw no key here: zeros) ----
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) + tk * a.out.token_stride +
                           head * a.out.head_stride + half * (D / 2);
      const int64_t at = (2 * static_cast<int64_t>(cluster) + slot) * a.piece_rows +
                         rank * kTile + row;
#pragma unroll 1
      for (int i = 0; i < D / 2; i += 32) {
        uint32_t o[32];
        __syncwarp();
        if (j1 > j0) {
          tmem_ld_32x32b_x32(to + i, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (row < rows && whole) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            uint32_t w[4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
              w[n] = pack_bf16x2(__uint_as_float(o[k + 2 * n]) * inv,
                                 __uint_as_float(o[k + 2 * n + 1]) * inv);
            *reinterpret_cast<uint4*>(out + i + k) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (row < rows) {
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            *reinterpret_cast<uint4*>(a.piece_o + at * D + half * (D / 2) + i + k) =
                make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
      }
      if (row < rows && half == 0) {
        if (!whole) a.piece_ml[at] = make_float2(m, l);
        else if (a.lse != nullptr) a.lse[tk * a.q.heads + head] = lse_of(m, l);
      }
      if (threadIdx.x == 0 && rank == 0 && !whole && slot == 1) {
        // this cluster begins a cut segment: where its pieces end, for the join
        const long long end = hi + (wk.b.t1 - stop);
        int last = cluster + 1;
        while (st.total * (last + 1) / clusters < end) ++last;
        AttnPiece p;
        p.rows = wk.b.rows;
        p.head = wk.h;
        p.first = wk.rq.first;
        p.row0 = wk.b.row0;
        p.last = last;
        p.total = st.total;
        *piece = p;
        begun = true;
      }
      t = stop;
      if (left > 0) {
        if (!wk.next(a, group)) break;
        t = wk.b.t0;
      }
    }
    if (threadIdx.x == 0 && rank == 0 && !begun) piece->rows = 0;
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync();                       // the other CTA may still write here until now
  if (warp == kIssueS) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int clusters,
                   cudaStream_t stream) {
  static PerDeviceOnce once;
  auto kernel = attention_chunk_kernel<D>;
  cudaError_t e =
      set_smem_attr_once(once, reinterpret_cast<const void*>(kernel), Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  // its prologue overlaps the plan; it waits for the plan before it reads anything
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, mk, mv);
}

}  // namespace

cudaError_t launch_attn_plan(const AttnArgs& a, int grid, cudaStream_t stream) {
  attn_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, grid);
  return cudaGetLastError();
}

cudaError_t launch_attention_chunk(const AttnArgs& a, const CUtensorMap& map_k,
                                   const CUtensorMap& map_v, int clusters, cudaStream_t stream) {
  return a.cache.head_dim == 128 ? launch<128>(a, map_k, map_v, clusters, stream)
                                 : launch<64>(a, map_k, map_v, clusters, stream);
}

}  // namespace nvmoe
