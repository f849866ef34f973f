// Drafted tokens held against the target's probabilities, with given random numbers.
//
// Request r has the rows s .. s + n of target and draft (n drafted tokens); row i of
// either is the distribution of token i + 1.  Token s + i + 1 stands while
// u_i q(x) < p(x), in order; the token after the last one that stands is drawn by the
// inverse of the running sum from p of that row, or, where a drafted token was turned
// down, from max(p - q, 0): the first token whose running sum passes v times the whole.
// So what is drawn has the target's distribution, whatever the draft's (Leviathan,
// Kalman and Matias, "Fast Inference from Transformers via Speculative Decoding", 2023).
//
// Of all the rows only one of p, and of q, is read whole: the bound is HBM for large
// batches, for few requests the launch and four dependent loads.  A cluster takes a
// request, its CTAs and their warps one run of the vocabulary each.  They find the sums
// of the runs, exchange them through distributed shared memory, and the warp in whose
// run the sum is passed reads that once more (from L2) to find the token.
//
// Which token that is must not hang on how a sum is rounded: a row of 2^17 tokens has
// as many borders, and fp32 sums would put the wrong token out for every few hundredth
// row.  Sums are pairs of fp32 numbers, value and rest, and p - q is exact that way.  What
// they lose grows with the square of their length n, where the rest takes what the value
// lost without being cut back: n (n + 3) 2^-48 of themselves at most (with q: without it
// half).  So a thread with more than 24 additions to each of its sums puts blocks of 8
// together, 32 of them as pairs that are cut back (3 * 2^-48 for each), and these in fp64.
// With the joins of lanes and warps, 15 deep, and the ends of a ragged row, running sums are
// off by 2^-38 of themselves at most, for every vocabulary that memory holds; as a rule,
// when errors do not all point one way, by 2^-45.  (fp64 throughout, of which an SM has two
// adds a cycle, took more than twice the time of the pairs even where it only joined lanes
// and warps.)
//
// Those 64 requests take 17 us, of which 6 are what two requests of few tokens take (the
// launch, the loads before the row is known, the joins): loads are asked for one by one as
// their predecessors are used (four at a time, then all four used: 21.5), and the row's
// ragged ends are apart from the loop, whose code is fetched anew by each launch.
#include "attn.cuh"
#include "serve.cuh"

namespace nvmoe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCtas = 8, kCtasPerSm = 4;
// Vectors of a row on their way to a thread.  (2 / 3 / 4: 64 requests of 129280 tokens with
// two CTAs each 29.2 / 25.5 / 23.3 us, with eight 17 all three.)
constexpr int kAhead = 4;

// Within [0, 1]; NaN is 0.
__device__ __forceinline__ float probability(float x) { return __saturatef(x); }
__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// A sum as a value and what it lacks, |rest| at most half a step of the value.
struct alignas(8) Sum {
  float hi, lo;
};
// (Knuth's exact sum of two numbers, the rests, and Dekker's of a large and a small one)
__device__ __forceinline__ Sum operator+(const Sum& x, const Sum& y) {
  const float t = x.hi + y.hi, b = t - x.hi;
  const float e = ((x.hi - (t - b)) + (y.hi - b)) + (x.lo + y.lo);
  const float hi = t + e;
  return {hi, e - (hi - t)};
}
__device__ __forceinline__ Sum operator-(const Sum& x, const Sum& y) {
  return x + Sum{-y.hi, -y.lo};
}
__device__ __forceinline__ bool operator>(const Sum& x, const Sum& y) {
  return x.hi > y.hi || (x.hi == y.hi && x.lo > y.lo);
}
__device__ __forceinline__ double wide(const Sum& x) { return static_cast<double>(x.hi) + x.lo; }
__device__ __forceinline__ Sum narrow(double x) {
  const float hi = static_cast<float>(x);
  return {hi, static_cast<float>(x - hi)};
}
__device__ __forceinline__ bool positive(const Sum& x) { return x.hi > 0.0f; }
__device__ __forceinline__ Sum shfl(const Sum& x, int lane) {
  return {__shfl_sync(0xFFFFFFFFu, x.hi, lane), __shfl_sync(0xFFFFFFFFu, x.lo, lane)};
}

// Additions to a thread's sum that need no blocks; additions of a block, blocks of a
// stretch.
constexpr int kPlain = 24, kBlock = 8, kBlocks = 32;

// Two sums side by side (one instruction for both), a lane's while it runs over a row.
struct Sums {
  uint64_t hi = 0, lo = 0;
  __device__ __forceinline__ void add(uint64_t x) {
    const uint64_t t = add_f32x2(hi, x), b = sub(t, hi);
    lo = add_f32x2(lo, add_f32x2(sub(hi, sub(t, b)), sub(x, b)));
    hi = t;
  }
  static __device__ __forceinline__ uint64_t sub(uint64_t x, uint64_t y) {
    return fma_f32x2(y, f32x2(-1.0f, -1.0f), x);        // (a product with -1 is exact)
  }
  __device__ __forceinline__ Sum value() const {
    float a, b, c, d;
    f32x2_split(hi, a, b);
    f32x2_split(lo, c, d);
    return Sum{a, c} + Sum{b, d};
  }
};

// The weights of a row: p, or what p has over q, or p without one token.
template <typename T>
struct Row {
  static constexpr int kVec = 16 / sizeof(T);
  static constexpr int kAdds = kVec / 4;               // to each of a thread's sums, of a vector
  static constexpr int kStretch = kBlocks * kBlock / kAdds;      // vectors
  const T* p;
  const T* q;                // null: p alone
  int vocab, without;        // a token that does not count, or -1
  int shift;                 // elements of p's first 16 bytes that lie before the row
  bool together;             // q's lie likewise

  __device__ __forceinline__ int vectors() const { return (vocab + shift + kVec - 1) / kVec; }
  static __device__ __forceinline__ int shift_of(const T* x) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  }

  // The elements of vector v, all within the row, of p or of a q that lies otherwise.
  __device__ __forceinline__ uint4 load(const T* x, int v) const {
    return *reinterpret_cast<const uint4*>(x + v * kVec - shift);
  }
  __device__ __forceinline__ uint4 load_apart(const T* x, int v) const {
    x += v * kVec - shift;
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      if constexpr (sizeof(T) == 4)
        w[k] = __float_as_uint(x[k]);
      else
        w[k / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(x[k])) << (k % 2 * 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // Elements 2 k and 2 k + 1 of a vector.
  static __device__ __forceinline__ void pair(const uint4& u, int k, float& x, float& y) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 4) {
      x = __uint_as_float(w[2 * k & 3]);
      y = __uint_as_float(w[(2 * k + 1) & 3]);
    } else {
      x = __uint_as_float(w[k & 3] << 16);
      y = __uint_as_float(w[k & 3] & 0xFFFF0000u);
    }
  }
  // A vector without element k.
  static __device__ __forceinline__ uint4 drop(uint4 u, int k) {
    const int word = k * static_cast<int>(sizeof(T)) / 4;
    const uint32_t keep = sizeof(T) == 4 ? 0u : (k % 2 == 0 ? 0xFFFF0000u : 0xFFFFu);
    if (word == 0) u.x &= keep;
    if (word == 1) u.y &= keep;
    if (word == 2) u.z &= keep;
    if (word == 3) u.w &= keep;
    return u;
  }
  __device__ __forceinline__ Sum weight(int e) const {
    if (e >= vocab || e == without) return {0.0f, 0.0f};
    const float a = probability(load_one(p + e));
    const float b = q != nullptr ? fminf(probability(load_one(q + e)), a) : 0.0f;
    const float d = a - b;
    return {d, (a - d) - b};
  }

  // A lane's sum over the whole vectors v0, v0 + step, .. below v1.  The next kAhead are on
  // their way at any time.  LONG: put together from blocks.
  template <bool LONG, bool DIFFERENCE, bool TOGETHER, int kAhead>
  __device__ __forceinline__ Sum sum_of(int v0, int v1, int step) const {
    const int drops = !DIFFERENCE && without >= 0 ? (without + shift) / kVec : -1;
    static_assert(kBlock % (kAhead * kAdds) == 0, "blocks of whole turns");
    Sum total = {0.0f, 0.0f};
    int added = 0;
    Sums s[2];
    uint4 pv[kAhead], qv[kAhead];
    const auto fetch = [&](int u, int v) {
      pv[u] = qv[u] = make_uint4(0, 0, 0, 0);
      if (v < v1) {
        pv[u] = load(p, v);
        if (DIFFERENCE) qv[u] = TOGETHER ? load(q, v) : load_apart(q, v);
      }
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(u, v0 + u * step);
#pragma unroll 1
    for (int v = v0; v < v1; v += kAhead * step) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (!DIFFERENCE && v + u * step == drops) pv[u] = drop(pv[u], (without + shift) % kVec);
#pragma unroll
        for (int k = 0; k < kVec / 2; ++k) {
          float a0, a1;
          pair(pv[u], k, a0, a1);
          a0 = probability(a0);
          a1 = probability(a1);
          const uint64_t a = f32x2(a0, a1);
          if (DIFFERENCE) {
            // p - min(p, q) and what that difference lacks: exact
            float b0, b1;
            pair(qv[u], k, b0, b1);
            const uint64_t b = f32x2(fminf(fmaxf(b0, 0.0f), a0), fminf(fmaxf(b1, 0.0f), a1));
            const uint64_t d = Sums::sub(a, b);
            s[k & 1].lo = add_f32x2(s[k & 1].lo, Sums::sub(Sums::sub(a, d), b));
            s[k & 1].add(d);
          } else {
            s[k & 1].add(a);
          }
        }
        fetch(u, v + (u + kAhead) * step);
      }
      added += kAhead * kAdds;
      if (LONG && (added % kBlock == 0 || v + kAhead * step >= v1)) {
        total = total + (s[0].value() + s[1].value());
        s[0] = s[1] = Sums{};
      }
    }
    return LONG ? total : s[0].value() + s[1].value();
  }
  // The same over all vectors; the row's first and last, if not whole, element by element.
  template <bool LONG>
  __device__ __forceinline__ Sum sum(int v0, int v1, int step) const {
    const int whole = (vocab + shift) / kVec;           // vectors up to the last whole one's end
    Sum edge = {0.0f, 0.0f};
    const auto elements = [&](int e0, int e1) {
#pragma unroll 1
      for (int e = e0; e < e1; ++e) edge = edge + weight(e);
    };
    if (whole < v1 && whole >= v0 && (whole - v0) % step == 0)
      elements(max(0, whole * kVec - shift), vocab);
    v1 = min(v1, whole);
    if (v0 == 0 && shift > 0 && v1 > 0) {
      elements(0, kVec - shift);
      v0 = step;
    }
    const auto stretch = [&](int end) {
      return q == nullptr ? sum_of<LONG, false, true, kAhead>(v0, end, step)
                          : together ? sum_of<LONG, true, true, kAhead>(v0, end, step)
                                     : sum_of<LONG, true, false, 1>(v0, end, step);
    };
    if (!LONG) return edge + stretch(v1);
    const bool one = v0 + kStretch * step >= v1;
    double far = 0.0;                                   // of the stretches before
#pragma unroll 1
    while (true) {
      edge = edge + stretch(min(v1, v0 + kStretch * step));
      if (one) return edge;
      far += wide(edge);
      edge = Sum{0.0f, 0.0f};
      v0 += kStretch * step;
      if (v0 >= v1) return narrow(far);
    }
  }
};

// Sum over the lanes up to this one.
__device__ __forceinline__ Sum scan_lanes(Sum x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sum y = {__shfl_up_sync(0xFFFFFFFFu, x.hi, o), __shfl_up_sync(0xFFFFFFFFu, x.lo, o)};
    if (lane >= o) x = x + y;
  }
  return x;
}

// Of the lanes' runs, `upto` the sum to the end of each and `own` that of the run: the
// first that passes x, else (by rounding) the last that holds anything; -1 if none does.
__device__ __forceinline__ int pick(const Sum& upto, const Sum& own, const Sum& x, bool* passes) {
  const uint32_t passed = __ballot_sync(0xFFFFFFFFu, positive(own) && upto > x);
  *passes = passed != 0;
  if (passed != 0) return __ffs(passed) - 1;
  const uint32_t any = __ballot_sync(0xFFFFFFFFu, positive(own));
  return any != 0 ? 31 - __clz(any) : -1;
}

template <typename T, bool LONG>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) draft_verify_kernel(const VerifyArgs a) {
  __shared__ Sum run_sum[2][kMaxCtas * kWarps];          // of all CTAs' warps
  __shared__ Sum warp_sum[kWarps];
  __shared__ int stands;
  pdl_wait();
  const int r = blockIdx.x / cluster_size(), rank = static_cast<int>(cluster_ctarank());
  const int ctas = static_cast<int>(cluster_size());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t begin = a.q_start[r], end = a.q_start[r + 1];
  const bool bad = begin < 0 || end < begin || end > a.rows;
  const int n = bad ? -1 : static_cast<int>(end - begin) - 1;        // drafted tokens
  if (n < 0) {                                          // (the whole cluster)
    if (rank == 0 && threadIdx.x == 0) {
      if (bad) record_status(a.status, kErrBadIndex);
      a.accepted[r] = 0;
      a.next_token[r] = -1;
      if (a.cached != nullptr) a.cached[r] = a.kv_len[r];
    }
    return;
  }
  cluster_arrive_relaxed();                             // (started: waited for below)
  const T* target = static_cast<const T*>(a.target) + begin * a.target_stride;
  const T* draft = a.draft == nullptr ? nullptr
                                      : static_cast<const T*>(a.draft) + begin * a.draft_stride;
  // ---- how many stand: a lane a token ----
  if (warp == 0) {
    int k = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      bool ok = false;
      if (i < n) {
        const int x = a.tokens[begin + i + 1];
        if (x < 0 || x >= a.vocab) {
          record_status(a.status, kErrBadIndex);        // does not stand
        } else {
          const float p = probability(load_one(target + i * a.target_stride + x));
          const float q =
              draft != nullptr ? probability(load_one(draft + i * a.draft_stride + x)) : 1.0f;
          // (a product of two fp32 numbers is exact in fp64)
          ok = static_cast<double>(a.accept_u[begin + i]) * q < static_cast<double>(p);
        }
      }
      const uint32_t not_ok = ~__ballot_sync(0xFFFFFFFFu, ok);
      if (not_ok != 0) {
        k = i0 + __ffs(not_ok) - 1;
        break;
      }
      k = i0 + 32;
    }
    if (lane == 0) stands = min(k, n);
  }
  __syncthreads();
  const int k = stands;
  Row<T> row;
  row.p = target + k * a.target_stride;
  row.q = k < n && draft != nullptr ? draft + k * a.draft_stride : nullptr;
  row.vocab = a.vocab;
  row.without = k < n && draft == nullptr ? a.tokens[begin + k + 1] : -1;
  row.shift = Row<T>::shift_of(row.p);
  row.together = row.q != nullptr && Row<T>::shift_of(row.q) == row.shift;

  const int runs = ctas * kWarps, run = rank * kWarps + warp;
  const long long vectors = row.vectors();
  const int v0 = static_cast<int>(vectors * run / runs);
  const int v1 = static_cast<int>(vectors * (run + 1) / runs);
  // a lane's runs of all: kMaxCtas * kWarps / 32 neighbours
  constexpr int kPer = kMaxCtas * kWarps / 32;
  Sum own[kPer], mine, upto, whole;
  for (int round = 0; round < 2; ++round) {
    Sum s = row.template sum<LONG>(v0 + lane, v1, 32);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      s = s + Sum{__shfl_xor_sync(0xFFFFFFFFu, s.hi, o), __shfl_xor_sync(0xFFFFFFFFu, s.lo, o)};
    if (round == 0) cluster_wait();                     // the others' shared memory is there
    if (lane < ctas) st_cluster_f32x2(&run_sum[round][run], lane, s.hi, s.lo);
    cluster_sync();
    mine = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int k = lane * kPer + i;
      own[i] = k < runs ? run_sum[round][k] : Sum{0.0f, 0.0f};
      mine = mine + own[i];
    }
    upto = scan_lanes(mine);
    whole = shfl(upto, 31);
    // nothing left over: the target's own row (and if that holds nothing, no token)
    if (positive(whole) || (row.q == nullptr && row.without < 0)) break;
    row.q = nullptr;
    row.without = -1;
  }
  if (rank == 0 && threadIdx.x == 0) {
    a.accepted[r] = k;
    if (a.cached != nullptr) a.cached[r] = a.kv_len[r] - (n - k);
    if (!positive(whole)) {
      record_status(a.status, kErrRange);
      a.next_token[r] = -1;
    }
  }
  if (!positive(whole)) return;

  // ---- the run in which the sum passes x = u * whole ----
  const float u = fmaxf(a.sample_u[r], 0.0f);           // (NaN: 0)
  Sum x = {u * whole.hi, 0.0f};
  x = x + Sum{fmaf(u, whole.hi, -x.hi), u * whole.lo};
  bool passes;
  int l = pick(upto, mine, x, &passes);
  // (every lane walks over its own; lane l's count)
  Sum next = upto - mine, before = next;
  int at = -1;
  bool passed = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const Sum after = next + own[i];
    if (!passed && positive(own[i])) {
      before = next;
      at = lane * kPer + i;
      passed = after > x;
    }
    next = after;
  }
  at = __shfl_sync(0xFFFFFFFFu, at, l);
  if (at / kWarps != rank) return;
  before = shfl(before, l);
  // ---- a thread of that CTA takes neighbouring vectors of the run ----
  const int w0 = static_cast<int>(vectors * at / runs), w1 = static_cast<int>(vectors * (at + 1) / runs);
  const int per = (w1 - w0 + kThreads - 1) / kThreads;
  const int a0 = min(w1, w0 + static_cast<int>(threadIdx.x) * per), a1 = min(w1, a0 + per);
  mine = row.template sum<LONG>(a0, a1, 1);
  const Sum in_warp = scan_lanes(mine);
  if (lane == 31) warp_sum[warp] = in_warp;
  __syncthreads();
  Sum held = lane < kWarps ? warp_sum[lane] : Sum{0.0f, 0.0f};
  upto = before + scan_lanes(held);
  l = pick(upto, held, x, &passes);
  if (l != warp) return;
  before = shfl(upto - held, l);
  upto = before + in_warp;
  l = pick(upto, mine, x, &passes);
  before = shfl(upto - mine, l);
  // ---- its elements, a lane each ----
  const int e0 = max(0, __shfl_sync(0xFFFFFFFFu, a0, l) * Row<T>::kVec - row.shift);
  const int e1 = min(a.vocab, __shfl_sync(0xFFFFFFFFu, a1, l) * Row<T>::kVec - row.shift);
  double done = LONG ? wide(before) : 0.0;
  int token = -1;
  for (int e = e0; e < e1; e += 32) {
    mine = e + lane < e1 ? row.weight(e + lane) : Sum{0.0f, 0.0f};
    const Sum here = scan_lanes(mine);
    upto = before + here;
    l = pick(upto, mine, x, &passes);
    if (l >= 0) token = e + l;
    if (passes) break;
    if (LONG) {                                         // (these may be thousands)
      done += wide(shfl(here, 31));
      before = narrow(done);
    } else {
      before = shfl(upto, 31);
    }
  }
  if (lane == 0) a.next_token[r] = token;
}

template <typename T>
cudaError_t launch(const VerifyArgs& a, cudaStream_t stream) {
  // A CTA for every 4096 tokens, up to 8, for every 8192 where there are more of them than
  // SMs, and as many as are resident at once.  (Clusters of more than two CTAs leave places
  // free in each group of SMs: 76 requests of 129280 tokens take 19.2 us with 7 CTAs each and
  // 23.2 with 8, which are as many as there are places; 64 requests 18.2 with 4, 16.9 with 8;
  // 64 of 32003 tokens 8.8 and 9.8.)
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t places = int64_t{kCtasPerSm} * sms;
  int ctas = 1;
  while (ctas < kMaxCtas && a.vocab > int64_t{ctas} * (int64_t{a.batch} * ctas <= sms ? 4096 : 8192) &&
         int64_t{a.batch} * (ctas + 1) <= (ctas < 2 ? places : places * 15 / 16))
    ++ctas;
  // additions to each of a thread's sums
  const int64_t run = ceil_div(int64_t{a.vocab} / Row<T>::kVec + 2, ctas * kWarps);
  const bool plain = ceil_div(run, 32) * Row<T>::kAdds <= kPlain;
  // its start overlaps the end of the kernel before
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // (blocks for all: 64 requests of 129280 tokens 17.7 us where this takes 17.2)
  return cudaLaunchKernelEx(
      &cfg, plain ? draft_verify_kernel<T, false> : draft_verify_kernel<T, true>, a);
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyArgs& a, cudaStream_t stream) {
  return a.bf16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

}  // namespace nvmoe
