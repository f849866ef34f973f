// Lengths, page tables, row offsets, positions and cache slots of a serving step.
//
// A request of `before` tokens, of which `cached` stand, brings `new`.  It holds
// ceil(before / page) pages and needs ceil((cached + new) / page): what it lacks comes
// from the front of the pool's ring, what it has left over goes behind the ring's end,
// in the order of the requests.  That is three prefix sums over the requests and a few
// words for each row and page, so a step is bound by latency: the launch and a chain of
// dependent loads (lengths, then pages).
//
// One cluster does it.  Each CTA runs the prefix sums over 1024 requests at a time for
// itself, and the CTAs share out the rows and pages, each of which finds its request by
// a search in shared memory.  The barrier of the cluster stands between the reads of the
// lengths and the writes, which may go to the same place.
#include "serve.cuh"

namespace nvmoe {
namespace {

constexpr int kThreads = 1024;            // requests of a pass
constexpr int kMaxCtas = 8;

struct Sums {
  long long take, give, rows;
};

// Sums of the values of the threads before this one; *total: of all.
__device__ __forceinline__ Sums block_scan(const Sums& v, Sums* warps, Sums* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const auto up = [&](Sums& x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xFFFFFFFFu, x.take, o);
      const long long b = __shfl_up_sync(0xFFFFFFFFu, x.give, o);
      const long long c = __shfl_up_sync(0xFFFFFFFFu, x.rows, o);
      if (lane >= o) {
        x.take += a;
        x.give += b;
        x.rows += c;
      }
    }
  };
  Sums x = v;
  up(x);
  __syncthreads();
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  if (warp == 0) {
    Sums s = warps[lane];
    up(s);
    warps[lane] = s;
  }
  __syncthreads();
  *total = warps[31];
  const Sums before = warp > 0 ? warps[warp - 1] : Sums{0, 0, 0};
  return {before.take + x.take - v.take, before.give + x.give - v.give,
          before.rows + x.rows - v.rows};
}

// The last i in [0, n) with first[i] <= x (ascending, first[0] <= x).
__device__ __forceinline__ int find(const int* first, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

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
  long long ring0 = a.pool.state[0], free = a.pool.state[1];
  if (ring0 < 0 || ring0 >= a.pool.size || free < 0 || free > a.pool.size) {
    record_status(a.status, kErrBadIndex);              // nothing can be taken
    ring0 = free = 0;
  }
  const auto ring_at = [&](long long i) {               // (i < 2 * size)
    i += ring0;
    if (i >= a.pool.size) i -= a.pool.size;
    return a.pool.ring + i;
  };

  Sums wanted = {0, 0, 0}, done = {0, 0, 0};            // of the passes before
  for (int r0 = 0; r0 < a.batch; r0 += kThreads) {
    const int r = r0 + threadIdx.x, count = min(kThreads, a.batch - r0);
    int held = 0, kept = 0;                             // pages before; of the tokens that stand
    long long stand = 0, n = 0, take = 0;
    int32_t old = 0;
    bool bad = false, ends = false;
    if (r < a.batch) {
      old = a.before[r];
      stand = a.cached != nullptr ? a.cached[r] : old;
      n = a.new_tokens[r];
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
    Sums total;
    Sums at = block_scan({take, held - kept, n}, warps, &total);
    const bool out = (take > 0 && wanted.take + at.take + take > free) ||
                     (n > 0 && wanted.rows + at.rows + n > a.rows);
    wanted.take += total.take;
    wanted.rows += total.rows;
    if (out) {
      record_status(a.status, kErrRange);
      take = n = 0;
      kept = static_cast<int>((stand + page - 1) >> ps);
    }
    if (__syncthreads_or(out)) at = block_scan({take, held - kept, n}, warps, &total);
    const int row = static_cast<int>(done.rows + at.rows);
    row0[threadIdx.x] = row;
    take0[threadIdx.x] = static_cast<int>(done.take + at.take);
    // (what does not fit the ring is dropped, below)
    give0[threadIdx.x] = static_cast<int>(min(done.give + at.give, 0x7FFFFFFFll));
    held_of[threadIdx.x] = held;
    kept_of[threadIdx.x] = kept;
    shift_of[threadIdx.x] = static_cast<int>(stand - row);
    cluster_sync();                                     // all have read, and may write
    if (rank == 0 && r < a.batch) {
      a.kv_len[r] = bad ? old : static_cast<int32_t>(stand + n);
      a.q_start[r] = row;
    }
    const Sums begin = done;
    done.take += total.take;
    done.give += total.give;
    done.rows += total.rows;

    // ---- rows ----
    if (a.positions != nullptr || a.slots != nullptr) {
      for (long long t = begin.rows + worker; t < done.rows; t += workers) {
        const int i = find(row0, count, static_cast<int>(t));
        const int pos = static_cast<int>(t) + shift_of[i];
        if (a.positions != nullptr) a.positions[t] = pos;
        if (a.slots != nullptr) {
          const int k = pos >> ps;
          const int64_t id = k < held_of[i]
                                 ? a.page_table[(r0 + i) * a.max_pages + k]
                                 : *ring_at(static_cast<long long>(take0[i]) + k - held_of[i]);
          a.slots[t] = id * page + (pos & (page - 1));
        }
      }
    }
    // ---- pages taken, and given back ----
    for (long long u = begin.take + worker; u < done.take; u += workers) {
      const int i = find(take0, count, static_cast<int>(u));
      a.page_table[(r0 + i) * a.max_pages + held_of[i] + (u - take0[i])] = *ring_at(u);
    }
    const long long most = a.pool.size - free;          // places behind the ring's end
    for (long long u = begin.give + worker; u < min(done.give, most); u += workers) {
      const int i = find(give0, count, static_cast<int>(u));
      *ring_at(free + u) = a.page_table[(r0 + i) * a.max_pages + kept_of[i] + (u - give0[i])];
    }
    __syncthreads();                                    // before the next pass's words
  }
  if (worker == 0) {
    if (done.give > a.pool.size - free) {
      record_status(a.status, kErrBadIndex);
      done.give = a.pool.size - free;
    }
    a.q_start[a.batch] = static_cast<int32_t>(done.rows);
    ring0 += done.take;
    a.pool.state_out[0] = static_cast<int32_t>(ring0 >= a.pool.size ? ring0 - a.pool.size : ring0);
    a.pool.state_out[1] = static_cast<int32_t>(free - done.take + done.give);
  }
}

}  // namespace

cudaError_t launch_plan_pages(const PlanArgs& a, cudaStream_t stream) {
  const int64_t rows = a.positions != nullptr || a.slots != nullptr ? a.rows : 0;
  int ctas = 1;
  while (ctas < kMaxCtas && rows > int64_t{ctas} * kThreads) ctas *= 2;
  // its start overlaps the end of the kernel before
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, plan_pages_kernel, a);
}

}  // namespace nvmoe
