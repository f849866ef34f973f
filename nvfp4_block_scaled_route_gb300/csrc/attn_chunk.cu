// Paged attention of chunks of new tokens on the tcgen05 tensor cores.
//
// The rows of a request and key head -- new tokens x query heads of the key
// head, token-major -- are taken in blocks of 256: two tiles of 128 query
// rows that share every key and value tile in shared memory.  Per 128 keys a
// tile costs two products of 128 x 128 x D, and 128 x 128 exponentials; the
// tensor pipe is the bound (4 * rows * keys * D flops), so the two tiles take
// turns: while the tensor cores run the products of one, the other's warps
// compute its softmax.
//
// Roles: warps 0-3 and 4-7 hold the softmax of tile 0 and 1 (a thread owns a
// row, so maxima and sums need no exchange), warp 8 loads key and value tiles
// by TMA (one box per page), warp 9 issues the MMAs.
//
//   S = Q K^T       both K-major from shared memory, into TMEM
//   P = 2^(cS - m)  TMEM -> registers -> 16 bits -> TMEM, over S
//   O += P V        P from TMEM, V as the MN-major operand from shared memory
//
// m is a reference, not always the maximum: O is rescaled only when a row's
// maximum has grown by more than 2^8 over its reference (any reference gives
// the same quotient; weights stay below 2^8, sums are fp32).  S(j) of a tile
// is issued after P V (j - 1), so once it has landed O may be rescaled.
//
// The work is the flat list of 128-key tiles of all (request, key head, row
// block) segments, causal limits taken off; CTA c of G takes an equal run of
// it (attn_plan_kernel finds where it starts), and attn_combine_kernel joins
// the segments cut by a border.
#include "attn.cuh"

namespace nvmoe {
namespace {

constexpr int kKeys = kAttnTileKeys;
constexpr int kTile = 128;                   // query rows of a tile
constexpr int kBlock = kAttnBlockRows;       // rows of a segment
constexpr int kProducer = 8, kIssuer = 9;
constexpr int kThreads = 320;
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
  static constexpr int kBytes = kKeys * D * 2;         // a key or value tile, a query tile
  static constexpr int kBufs = D == 128 ? 5 : 10;
  static constexpr int kSmem = 1024 + 2 * kBytes + kBufs * kBytes + 512;
  static constexpr uint32_t kTmemO = 256;              // S: columns 0 and 128
};

struct Bars {
  uint64_t full[10], empty[10];
  uint64_t q_ready[2], s_full[2], p_ready[2], o_full[2], done;
  uint32_t tmem;
  int abort;
};

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
  extern __shared__ uint8_t raw_smem[];
  uint8_t* sq = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  uint8_t* ring = sq + 2 * C::kBytes;
  Bars* bars = reinterpret_cast<Bars*>(ring + C::kBufs * C::kBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_ready[i], kTile);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_ready[i], kTile);
      mbar_init(&bars->o_full[i], 1);
    }
    mbar_init(&bars->done, 1);
    bars->abort = 0;
    fence_mbarrier_init();
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
  }
  if (warp == kIssuer) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  volatile int* abort = &bars->abort;
  pdl_trigger();
  pdl_wait();                                          // the plan

  const AttnStart st = a.starts[blockIdx.x];
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
  AttnPiece* piece = a.pieces + blockIdx.x;
  int begun_rows = 0;

  if (warp == kProducer) {
    // ---- key and value tiles: lane = box (page part, column block) ----
    const int box = min(kKeys, 1 << a.cache.page_shift);
    const int b = lane & 7, half = lane >> 3;
    const uint64_t policy = policy_evict_normal();
    int buf = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (left > 0 && ok) {
      const int stop = static_cast<int>(min(static_cast<long long>(wk.b.t1), t + left));
      left -= stop - t;
      for (; t < stop && ok; ++t) {
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
        const int loads = __popc(__ballot_sync(0xFFFFFFFFu, take));
        const int in_page = key & ((1 << a.cache.page_shift) - 1);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          ok = ok && mbar_wait(&bars->empty[buf], phase ^ 1u, a.status, abort);
          if (!ok) break;
          if (lane == 0)
            mbar_arrive_expect_tx(&bars->full[buf], static_cast<uint32_t>(loads * box * 128));
          __syncwarp();
          if (take)
            tma_load_4d(ring + buf * C::kBytes + half * kKeys * 128 + b * box * 128,
                        kv == 0 ? &map_k : &map_v, half * 64, in_page, wk.h, page,
                        &bars->full[buf], policy);
          if (++buf == C::kBufs) {
            buf = 0;
            phase ^= 1u;
          }
        }
      }
      if (left > 0) {
        if (!wk.next(a, group)) break;
        t = wk.b.t0;
      }
    }
  } else if (warp == kIssuer) {
    // ---- MMAs ----
    constexpr uint32_t kIdescS = idesc_bf16_f32(kTile, kKeys);
    constexpr uint32_t kIdescO = idesc_bf16_f32(kTile, D) | (1u << 16);     // B is MN-major
    const uint32_t sq_u = smem_u32(sq), ring_u = smem_u32(ring);
    int buf = 0;
    uint32_t phase = 0, q_phase = 0, p_phase = 0;       // bit a: parity of tile a's barriers
    const auto advance = [&] {
      if (++buf == C::kBufs) {
        buf = 0;
        phase ^= 1u;
      }
    };
    const auto scores = [&](int q, uint32_t k_addr) {
      if (lane == 0) {
        const uint32_t qa = sq_u + q * C::kBytes;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks >> 2) * (kKeys * 128) + (ks & 3) * 32;
          mma_f16(tmem + q * 128, smem_desc(qa + off, 16, 1024, 2),
                  smem_desc(k_addr + off, 16, 1024, 2), kIdescS, ks != 0);
        }
        tc_commit(&bars->s_full[q]);
      }
    };
    while (left > 0) {
      const int stop = static_cast<int>(min(static_cast<long long>(wk.b.t1), t + left));
      left -= stop - t;
      int j0[2], j1[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        j0[q] = max(t, wk.b.a0[q]);
        j1[q] = min(stop, wk.b.a1[q]);
        if (j1[q] > j0[q]) {
          mbar_wait(&bars->q_ready[q], (q_phase >> q) & 1u, a.status, abort);
          q_phase ^= 1u << q;
        }
      }
      tc_fence_after();
      mbar_wait(&bars->full[buf], phase, a.status, abort);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (t >= j0[q] && t < j1[q]) scores(q, ring_u + buf * C::kBytes);
      if (lane == 0) tc_commit(&bars->empty[buf]);
      advance();
      for (; t < stop; ++t) {
        const int vb = buf;
        mbar_wait(&bars->full[vb], phase, a.status, abort);
        if (t * kKeys < wk.b.kbeg || (t + 1) * kKeys > wk.b.kend) {
          // values that no row sees may hold anything: make them zeros
          for (int i = lane; i < kKeys * (D / 8); i += 32) {
            const int row = i / (D / 8), key = t * kKeys + row;
            if (key < wk.b.kbeg || key >= wk.b.kend)
              *reinterpret_cast<uint4*>(ring + vb * C::kBytes + tile_at(row, i % (D / 8))) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        advance();
        const bool more = t + 1 < stop;
        bool have_k = false;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (t >= j0[q] && t < j1[q]) {
            mbar_wait(&bars->p_ready[q], (p_phase >> q) & 1u, a.status, abort);
            p_phase ^= 1u << q;
            tc_fence_after();
            if (lane == 0) {
              const uint32_t va = ring_u + vb * C::kBytes;
#pragma unroll
              for (int ks = 0; ks < kKeys / 16; ++ks)
                mma_f16_ts(tmem + C::kTmemO + q * D, tmem + q * 128 + ks * 8,
                           smem_desc(va + ks * 2048, kKeys * 128, 1024, 2), kIdescO,
                           t != j0[q] || ks != 0);
              if (t + 1 == j1[q]) tc_commit(&bars->o_full[q]);
            }
          }
          if (more && t + 1 >= j0[q] && t + 1 < j1[q]) {
            if (!have_k) mbar_wait(&bars->full[buf], phase, a.status, abort);
            have_k = true;
            scores(q, ring_u + buf * C::kBytes);
          }
        }
        if (lane == 0) tc_commit(&bars->empty[vb]);
        if (more) {
          if (!have_k) mbar_wait(&bars->full[buf], phase, a.status, abort);
          if (lane == 0) tc_commit(&bars->empty[buf]);
          advance();
        }
      }
      if (left > 0) {
        if (!wk.next(a, group)) break;
        t = wk.b.t0;
      }
    }
  } else {
    // ---- softmax of query tile q, a thread per row ----
    const int q = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + q * 128 + lanes, to = tmem + C::kTmemO + q * D + lanes;
    const long long hi = st.total * (blockIdx.x + 1) / gridDim.x;
    uint32_t s_phase = 0, o_phase = 0;
    const float c = a.scale * 1.4426950408889634f;      // scores in powers of two
    while (left > 0) {
      const int stop = static_cast<int>(min(static_cast<long long>(wk.b.t1), t + left));
      const bool whole = t == wk.b.t0 && stop == wk.b.t1;
      const int slot = t == wk.b.t0 ? 1 : 0;
      left -= stop - t;
      const int rows = min(kTile, wk.b.rows - q * kTile);
      const int j0 = max(t, wk.b.a0[q]), j1 = min(stop, wk.b.a1[q]);
      const int row0 = wk.b.row0 + q * kTile;
      const int my = row0 + min(row, max(rows, 1) - 1);  // rows past the end act as the last
      const int tok = my / group;
      const int pos = wk.rq.pos0 + tok;
      float m = -INFINITY, l = 0.0f;
      if (j1 > j0) {
        // queries (the last S that read the previous ones has landed)
        constexpr int kLanes = D / 8;
        const int ch = threadIdx.x & (kLanes - 1);
        for (int i = (threadIdx.x & 127) / kLanes; i < kTile; i += 128 / kLanes) {
          uint4 u = make_uint4(0, 0, 0, 0);
          if (i < rows) {
            const int tk = (row0 + i) / group;
            u = *reinterpret_cast<const uint4*>(
                static_cast<const __nv_bfloat16*>(a.q.data) +
                (wk.rq.first + tk) * a.q.token_stride +
                (wk.h * group + row0 + i - tk * group) * a.q.head_stride + ch * 8);
          }
          *reinterpret_cast<uint4*>(sq + q * C::kBytes + tile_at(i, ch)) = u;
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars->q_ready[q]);
        const int vis_hi = min(pos + 1, wk.rq.len);
        const int vis_lo = a.window > 0 ? pos - a.window + 1 : 0;
        // keys that every row of the tile sees
        const int all_hi = min(wk.rq.pos0 + row0 / group + 1, wk.rq.len);
        const int all_lo =
            a.window > 0 ? wk.rq.pos0 + (row0 + rows - 1) / group - a.window + 1 : 0;
        for (int j = j0; j < j1; ++j) {
          mbar_wait(&bars->s_full[q], s_phase, a.status, abort);
          s_phase ^= 1u;
          __syncwarp();
          tc_fence_after();
          uint32_t s[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(ts + i * 32, s[i]);
          tmem_ld_wait();
          if ((j + 1) * kKeys > all_hi || j * kKeys < all_lo) {
            const int h = vis_hi - j * kKeys, lw = vis_lo - j * kKeys;
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (i >= h || i < lw) s[i >> 5][i & 31] = 0xFF800000u;      // -inf
          }
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < 128; ++i) top = fmaxf(top, __uint_as_float(s[i >> 5][i & 31]));
          top *= c;
          // a new reference where some row's maximum has left the old one behind
          const bool grow = top > m + 8.0f;
          if (__any_sync(0xFFFFFFFFu, grow)) {
            const float mn = fmaxf(m, top);
            if (j > j0) {
              const float f = exp2_approx(m - (mn == -INFINITY ? 0.0f : mn));
              l *= f;
#pragma unroll 1
              for (int i = 0; i < D; i += 32) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(to + i, o);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st_32x32b_x32(to + i, o);
              }
            }
            m = mn;
          }
          const float use = m == -INFINITY ? 0.0f : m;  // a row without keys so far
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float x = exp2_approx(fmaf(__uint_as_float(s[i][2 * k]), c, -use));
              const float y = exp2_approx(fmaf(__uint_as_float(s[i][2 * k + 1]), c, -use));
              sum += x + y;
              p[k] = pack_bf16x2(x, y);
            }
            tmem_st_32x32b_x16(ts + i * 16, p);
          }
          l += sum;
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&bars->p_ready[q]);
        }
        mbar_wait(&bars->o_full[q], o_phase, a.status, abort);
        o_phase ^= 1u;
        tc_fence_after();
      }
      // ---- the rows out (a tile that saw no key here: zeros) ----
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const int head = wk.h * group + my - tok * group;
      const int64_t tk = wk.rq.first + tok;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) + tk * a.out.token_stride +
                           head * a.out.head_stride;
      const int64_t at = (2 * static_cast<int64_t>(blockIdx.x) + slot) * a.piece_rows +
                         q * kTile + row;
#pragma unroll 1
      for (int i = 0; i < D; i += 32) {
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
            *reinterpret_cast<uint4*>(a.piece_o + at * D + i + k) =
                make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
      }
      if (row < rows) {
        if (!whole) a.piece_ml[at] = make_float2(m, l);
        else if (a.lse != nullptr) a.lse[tk * a.q.heads + head] = lse_of(m, l);
      }
      if (threadIdx.x == 0 && !whole && slot == 1) {
        const long long end = hi + (wk.b.t1 - stop);
        int last = blockIdx.x + 1;
        while (st.total * (last + 1) / gridDim.x < end) ++last;
        AttnPiece p;
        p.rows = wk.b.rows;
        p.head = wk.h;
        p.first = wk.rq.first;
        p.row0 = wk.b.row0;
        p.last = last;
        p.total = st.total;
        *piece = p;
        begun_rows = wk.b.rows;
      }
      t = stop;
      if (left > 0) {
        if (!wk.next(a, group)) break;
        t = wk.b.t0;
      }
    }
    if (threadIdx.x == 0 && begun_rows == 0) piece->rows = 0;
    tc_fence_before();
  }
  if (warp == kIssuer) {
    // every arrival that the tensor cores still owe this CTA's barriers
    if (lane == 0) tc_commit(&bars->done);
    mbar_wait(&bars->done, 0, a.status, abort);
  }
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int grid,
                   cudaStream_t stream) {
  static PerDeviceOnce once;
  auto kernel = attention_chunk_kernel<D>;
  cudaError_t e =
      set_smem_attr_once(once, reinterpret_cast<const void*>(kernel), Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  // its prologue overlaps the plan; it waits for the plan before it reads anything
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::kSmem;
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
  return a.cache.head_dim == 128 ? launch<128>(a, map_k, map_v, grid, stream)
                                 : launch<64>(a, map_k, map_v, grid, stream);
}

}  // namespace nvmoe
