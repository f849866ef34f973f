// Lengths, page tables, row offsets, positions and cache slots of a serving step.
//
// A request of `before` tokens, of which `cached` stand, brings `new`.  It holds
// ceil(before / page) pages and needs ceil((cached + new) / page): what it lacks comes
// from the front of the pool's ring, what it has left over goes behind the ring's end,
// in the order of the requests.  That is three prefix sums over the requests and a few
// words for each row and page, so a step is bound by latency: the launch, a chain of
// dependent loads (lengths, then pages) and the fetching of code that runs once (loops are
// not unrolled for it).  64 requests of three rows 3.4 us, 300 of up to 100 rows 6.7.
//
// One cluster does it.  Each CTA runs the prefix sums over up to 1024 requests at a time
// for itself, and the CTAs share out the rows and pages, each of which finds its request by
// a search in shared memory.  The barrier of the cluster stands between the reads of the
// lengths and the writes, which may go to the same place.
#include "serve.cuh"

namespace nvmoe {
namespace {

constexpr int kMaxCtas = 8;

// Counts that stay at 2^32 - 1 when they pass it (more than any limit).
struct Sums {
  uint32_t take, give, rows;
};
__device__ __forceinline__ uint32_t add(uint32_t x, uint32_t y) {
  return x + y < x ? 0xFFFFFFFFu : x + y;
}

__device__ __forceinline__ Sums add(const Sums& x, const Sums& y) {
  return {add(x.take, y.take), add(x.give, y.give), add(x.rows, y.rows)};
}
__device__ __forceinline__ Sums shfl_up(const Sums& x, int o) {
  return {__shfl_up_sync(0xFFFFFFFFu, x.take, o), __shfl_up_sync(0xFFFFFFFFu, x.give, o),
          __shfl_up_sync(0xFFFFFFFFu, x.rows, o)};
}

// Sums of the values of the threads before this one; *total: of all.
template <int THREADS>
__device__ __forceinline__ Sums block_scan(const Sums& v, Sums* warps, Sums* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const auto scan = [&](Sums x) {                       // over the lanes up to this one
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const Sums y = shfl_up(x, o);
      if (lane >= o) x = add(x, y);
    }
    return x;
  };
  __syncthreads();
  const Sums upto = scan(v);
  if (lane == 31) warps[warp] = upto;
  __syncthreads();
  Sums before = {0, 0, 0};
  if (THREADS <= 256) {                                 // (a few sums: every thread adds them)
    Sums all = {0, 0, 0};
#pragma unroll 1
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w == warp) before = all;
      all = add(all, warps[w]);
    }
    *total = all;
  } else {
    if (warp == 0) warps[lane] = scan(lane < THREADS / 32 ? warps[lane] : Sums{0, 0, 0});
    __syncthreads();
    *total = warps[31];
    if (warp > 0) before = warps[warp - 1];
  }
  const Sums own = shfl_up(upto, 1);
  return lane == 0 ? before : add(before, own);
}

// The last i in [0, n) with first[i] <= x (ascending, first[0] <= x).
__device__ __forceinline__ int find(const int* first, int n, int x) {
  int lo = 0, hi = n - 1;
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// THREADS: requests of a pass.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1) plan_pages_kernel(const PlanArgs a) {
  // of the pass's requests: first row, page taken, page given back; pages held, and
  // kept; the position of row t is t + shift
  __shared__ int row0[kThreads], take0[kThreads], give0[kThreads];
  __shared__ int held_of[kThreads], kept_of[kThreads], shift_of[kThreads];
  __shared__ Sums warps[32];
  pdl_wait();
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(cluster_size());
  const int worker = rank * kThreads + threadIdx.x, workers = ctas * kThreads;
  const int ps = a.page_shift, page = 1 << ps;
  const int64_t cap = a.max_pages << ps;                // < 2^31
  // (the first pass's lengths at once with the pool's state)
  int32_t in_old = 0, in_cached = 0, in_new = 0;
  const auto read = [&](int r) {
    if (r >= a.batch) return;
    in_old = a.before[r];
    in_cached = a.cached != nullptr ? a.cached[r] : in_old;
    in_new = a.new_tokens[r];
  };
  read(static_cast<int>(threadIdx.x));
  long long ring0 = a.pool.state[0], free = a.pool.state[1];
  long long size = a.pool.size;
  if (ring0 < 0 || ring0 >= size || free < 0 || free > size) {
    record_status(a.status, kErrBadIndex);              // nothing can be taken or given back
    ring0 = free = size = 0;
  }
  const auto ring_at = [&](long long i) {               // (i < 2 * size)
    i += ring0;
    if (i >= size) i -= size;
    return a.pool.ring + i;
  };

  long long wanted_take = 0, wanted_rows = 0;           // of the passes before
  long long done_take = 0, done_give = 0, done_rows = 0;
  for (int r0 = 0; r0 < a.batch; r0 += kThreads) {
    const int r = r0 + threadIdx.x, count = min(kThreads, a.batch - r0);
    int held = 0, kept = 0;                             // pages before; of the tokens that stand
    long long stand = 0, n = 0, take = 0;
    int32_t old = 0;
    bool bad = false, ends = false;
    if (r0 > 0) read(r);
    if (r < a.batch) {
      old = in_old;
      stand = in_cached;
      n = in_new;
      ends = n < 0;
      bad = old < 0 || old > cap || (!ends && (stand < 0 || stand > old || stand + n > cap));
      if (bad) {                                        // left as it is
        record_status(a.status, kErrBadIndex);
        held = kept = old <= 0 ? 0 : static_cast<int>(min((int64_t{old} + page - 1) >> ps, a.max_pages));
        stand = old;
        n = 0;
      } else {
        if (ends) stand = n = 0;
        held = static_cast<int>((old + page - 1ll) >> ps);
        kept = static_cast<int>((stand + page - 1) >> ps);
        const int need = static_cast<int>((stand + n + page - 1) >> ps);
        take = max(0, need - held);
        kept = max(kept, min(held, need));
      }
    }
    // Those that the pages or the rows do not suffice for, counted in order, bring none.
    Sums total, at;
    bool out = false;
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
      at = block_scan<kThreads>({static_cast<uint32_t>(take), static_cast<uint32_t>(held - kept),
                                 static_cast<uint32_t>(n)}, warps, &total);
      if (round == 1) break;                            // without those
      out = (take > 0 && wanted_take + at.take + take > free) ||
            (n > 0 && wanted_rows + at.rows + n > a.rows);
      wanted_take += total.take;
      wanted_rows += total.rows;
      if (out) {
        record_status(a.status, kErrRange);
        take = n = 0;
        kept = static_cast<int>((stand + page - 1) >> ps);
      }
      if (!__syncthreads_or(out)) break;
    }
    const int row = static_cast<int>(done_rows + at.rows);
    row0[threadIdx.x] = row;
    take0[threadIdx.x] = static_cast<int>(done_take + at.take);
    // (what does not fit the ring is dropped, below)
    give0[threadIdx.x] = static_cast<int>(min(done_give + at.give, 0x7FFFFFFFll));
    held_of[threadIdx.x] = held;
    kept_of[threadIdx.x] = kept;
    shift_of[threadIdx.x] = static_cast<int>(stand - row);
    // all have read, and may write
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    if (rank == 0 && r < a.batch) {
      a.kv_len[r] = bad ? old : static_cast<int32_t>(stand + n);
      a.q_start[r] = row;
    }
    const long long begin_take = done_take, begin_give = done_give, begin_rows = done_rows;
    done_take += total.take;
    done_give += total.give;
    done_rows += total.rows;

    // ---- rows (a loop of little code: most of it is fetched for one turn) ----
    if (a.positions != nullptr || a.slots != nullptr) {
#pragma unroll 1
      for (long long t = begin_rows + worker; t < done_rows; t += workers) {
        const int i = find(row0, count, static_cast<int>(t));
        const int pos = static_cast<int>(t) + shift_of[i], k = pos >> ps;
        if (a.positions != nullptr) a.positions[t] = pos;
        if (a.slots != nullptr) {
          const int64_t id = *(k < held_of[i]
                                   ? a.page_table + ((r0 + i) * a.max_pages + k)
                                   : ring_at(static_cast<long long>(take0[i]) + k - held_of[i]));
          a.slots[t] = id * page + (pos & (page - 1));
        }
      }
    }
    // ---- pages taken, and given back (from the last thread on: the rows begin with the
    // first) ----
    const long long taken = done_take - begin_take;
    const long long most = size - free;                 // places behind the ring's end
    const long long given = max(0ll, min(done_give, most) - begin_give);
#pragma unroll 1
    for (long long v = workers - 1 - worker; v < taken + given; v += workers) {
      const bool takes = v < taken;
      const long long u = takes ? begin_take + v : begin_give + v - taken;
      const int* first = takes ? take0 : give0;
      const int i = find(first, count, static_cast<int>(u));
      int32_t* entry = a.page_table + ((r0 + i) * a.max_pages + (takes ? held_of : kept_of)[i] +
                                       (u - first[i]));
      int32_t* place = ring_at(takes ? u : free + u);
      if (takes) *entry = *place;
      else *place = *entry;
    }
    __syncthreads();                                    // before the next pass's words
  }
  if (worker == 0) {
    if (done_give > size - free) {
      record_status(a.status, kErrBadIndex);
      done_give = size - free;
    }
    a.q_start[a.batch] = static_cast<int32_t>(done_rows);
    if (size == 0 && a.pool.state_out == a.pool.state) return;    // (a bad pool stays as it was)
    ring0 += done_take;
    a.pool.state_out[0] = static_cast<int32_t>(ring0 >= size ? ring0 - size : ring0);
    a.pool.state_out[1] = static_cast<int32_t>(free - done_take + done_give);
  }
}

}  // namespace

cudaError_t launch_plan_pages(const PlanArgs& a, cudaStream_t stream) {
  const int64_t rows = a.positions != nullptr || a.slots != nullptr ? a.rows : 0;
  const auto go = [&](auto kernel, int ctas, int threads) {
    // its start overlaps the end of the kernel before
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
  };
  // (64 requests of three rows: 5.0 us on 1024 threads, 3.4 on 256)
  if (a.batch <= 256 && rows <= 1024) return go(plan_pages_kernel<256>, 1, 256);
  int ctas = 1;
  while (ctas < kMaxCtas && rows > int64_t{ctas} * 1024) ctas *= 2;
  return go(plan_pages_kernel<1024>, ctas, 1024);
}

}  // namespace nvmoe
