// Beam search: the selection over beams and vocabulary, and the reordering of
// the recurrent states that follows it.
//
// Selection.  Candidate (w, t) of a request scores
//   scores[w] + x[w][t] - lse_w,   lse_w = log sum_t exp(x[w][t]).
// Within a beam the order is that of x, so a beam's K best tokens need no
// lse, and the scan kernel finds both in one pass over the logits: a CTA takes
// a span of one row, its warps interleaved, each lane a vector of 32 bytes a
// round.  What is listed is the vector, by its largest value, as the K best
// values lie in the K best vectors: a lane whose vector reaches a threshold
// appends it to its warp's list in shared memory, without a barrier, and only
// the last K are taken apart.  (With every value listed by itself a round ran
// twice the instructions.)  The threshold: every lane keeps the largest value
// it has seen, a warp takes the r-th largest of its lanes' (of the first round
// before any is listed, then after 2, 4, 8, ... rounds), and the least of the
// eight warps' is reached by at least 8 r >= K vectors of the span.  About
// 40 (1 + ln n) vectors of n rounds reach it for K = 16.  A list that grows past
// 128 all the same (ties, ascending rows) is cut back to its K best.  The merge
// kernel, one CTA per request, adds the spans' sums and picks the K best of the
// rows' lists.
//
// Bound.  Reading the logits once would take 7.9 us for 64 x 8 x 50257 in bf16 and
// 15.7 in fp32; both kernels take 24.6 and 32.2 (34.4 and 31.1 with 16 bytes a
// round and values listed).  Two things bound the scan, about alike: instructions
// (unpacking, maximum, exponential and sum of 16 values are some 110 of the 130
// that a warp runs a round; issue slots are 57 % busy) and an uneven spread (512
// rows on 592 places leave 3 or 4 CTAs on an SM, 38 % of the warps active, and
// beginning and end of a row, which no other row's rounds cover, are 5 us of it).
// The loads are one round ahead; two ahead move more registers than they hide
// (1 us).  A call that takes sums again in fp64 is longer: 155 us for fp32 logits.
//
// Order keys.  (value, lower index first) is one 64-bit number: the fp32 value
// mapped to an order-preserving integer above the complement of the index.
// All keys differ, so ranks by counting give a sorted list.
//
// Sums.  A warp's terms are exp(x - m) with one m, which follows the maximum
// only when that has risen by more than 2: no rescaling in the common round.
// (x - m is formed first: x log2 e would overflow for logits of the type's
// lowest value.)
//
// Exactness.  Scores of one beam differ exactly as their logits do; across
// beams the order hangs on lse_w.  A term 2^t of a row's fp32 sum is off by 2
// ulp of ex2.approx (2^-22) and by ln 2 |t| (2^-24 + 2^-24 + 2^-26) from x - m,
// the product and log2 e, a lane's tree of 8 adds 3 2^-24, and these add up in
// fp64.  t is at most 3 above 0; below it the terms' weights keep their mean
// |t| under log2 V.  So a lse is off by at most 4.2e-7 + 9.3e-8 log2 V = eps / 2,
// and candidates of two beams are in order where their scores are more than eps
// apart.  Where two neighbours in the chosen order come from different beams and
// lie within eps, or a candidate that was not chosen lies within eps of the last
// chosen one and comes from another beam, the CTA takes those beams' sums again
// in fp64 and orders once more (4 % of calls at 64 x 8 x 50257, K = 16, normal
// logits).  That is enough: if a candidate b was put behind a of another beam
// against the exact order, they lie within eps, and so do all between them; the
// chain from a to b changes beams next to an entry of a's beam and next to one of
// b's, so both are taken again.  The other beams' candidates were more than eps
// from what they might change places with, and an exact sum moves a score by
// eps / 2 at most, so their order stands.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "ia_device.cuh"
#include "ia_internal.h"
#include "ia_launch.h"

namespace ia {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxW = 64, kMaxK = 64;
constexpr int kVec = 32;                      // bytes per lane and round
template <typename T>
constexpr int kPer = kVec / static_cast<int>(sizeof(T));   // its values
constexpr int kWarps = kThreads / 32;
constexpr int kKeep = 128;                    // a warp's list is cut back to K when it is longer
constexpr int kCap = kKeep + 32;              // and grows by at most this much in a round
constexpr int kSlots = kCap / 32;
constexpr float kSlack = 2.f;
constexpr int kMergeMost = 2048;              // entries one merge takes (or one per beam and place, if more)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ uint32_t ordered(float x) {   // monotone; x is not NaN; -0 counts as 0
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t make_key(float x, uint32_t idx) {
  return static_cast<uint64_t>(ordered(x)) << 32 | (0xffffffffu - idx);
}
__device__ __forceinline__ float key_value(uint64_t k) { return unordered(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return 0xffffffffu - static_cast<uint32_t>(k); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The K best of n keys in `buf` (n <= kCap), sorted, in buf[0 .. min(n, K));
// returns that count.  One warp.  Out of line: it is rare, and its registers
// would cost the scan one of four CTAs per SM.
__device__ __noinline__ int cut_back(uint64_t* buf, int n, int K, int lane) {
  const unsigned full = 0xffffffffu;
  uint64_t key[kSlots];
  uint64_t a = 0, b = 0;   // the lane's largest and second
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int j = 32 * i + lane;
    key[i] = j < n ? buf[j] : 0;
    if (key[i] > a) b = a, a = key[i];
    else if (key[i] > b) b = key[i];
  }
  // A key that at least K keys reach: the K-th largest of the lanes' largest,
  // or for K > 32 the least of the lanes' second largest.
  uint64_t thr;
  if (K <= 32) {
    int rank = 0;
#pragma unroll 4
    for (int l = 0; l < 32; ++l) rank += __shfl_sync(full, a, l) > a;
    const unsigned who = __ballot_sync(full, a && rank == K - 1);
    thr = who ? __shfl_sync(full, a, __ffs(who) - 1) : 0;
  } else {
    thr = b;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(full, thr, o);
      thr = other < thr ? other : thr;
    }
  }
  __syncwarp();
  int m = 0;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const bool in = key[i] && key[i] >= thr;
    const unsigned who = __ballot_sync(full, in);
    if (in) buf[m + __popc(who & ((1u << lane) - 1))] = key[i];
    m += __popc(who);
  }
  __syncwarp();
  int rank[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    rank[i] = K;
    if (32 * i >= m) continue;
    const int j = 32 * i + lane;
    key[i] = j < m ? buf[j] : 0;
    int r = 0;
#pragma unroll 4
    for (int l = 0; l < m; ++l) r += buf[l] > key[i];
    if (j < m) rank[i] = r;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (rank[i] < K) buf[rank[i]] = key[i];
  __syncwarp();
  return min(m, K);
}

constexpr int kAll = kWarps * kMaxK;   // keys the CTA's merge takes
static_assert(kWarps * kCap >= kMaxK * kPer<__nv_bfloat16>, "the best vectors' values fit the lists");
struct ScanSmem {
  uint64_t buf[kWarps][kCap];   // of vectors: (largest value, number)
  uint64_t all[kAll];
  uint64_t top[kMaxK];      // the best vectors, sorted
  volatile float lead[kWarps];   // r-th largest of the lanes' largest values, per warp
  int count[kWarps];        // of the warps' lists
  int total, found;
  float m[kWarps];
  double s[kWarps];
};

template <typename T>
__device__ __forceinline__ float to_f(T x) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(x);
  else return x;
}

// A lane's values of one round, as loaded.
template <typename T>
struct Vec {
  uint32_t w[8];
  __device__ __forceinline__ void load(const T* p) {   // from a 32-byte boundary
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  }
  __device__ __forceinline__ void load_part(const T* p, int n) {   // n < kPer values from anywhere
    clear();
#pragma unroll
    for (int i = 0; i < kPer<T>; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 2) {
          const uint32_t u = __bfloat16_as_ushort(p[i]);
          w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | u << 16 : (w[i / 2] & 0xffff0000u) | u;
        } else {
          w[i] = __float_as_uint(p[i]);
        }
      }
  }
  __device__ __forceinline__ void clear() {   // -inf
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
  }
  __device__ __forceinline__ float max() const {   // of those that are numbers
    if constexpr (sizeof(T) == 2) {
      __nv_bfloat162 m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        m[i] = __hmax2(reinterpret_cast<const __nv_bfloat162&>(w[2 * i]), reinterpret_cast<const __nv_bfloat162&>(w[2 * i + 1]));
      m[0] = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
      return fmaxf(__low2float(m[0]), __high2float(m[0]));
    } else {
      float m = __uint_as_float(w[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = fmaxf(m, __uint_as_float(w[i]));
      return m;
    }
  }
  __device__ __forceinline__ uint64_t pair(int i) const {
    if constexpr (sizeof(T) == 2) return f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    else return f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
};

__device__ __forceinline__ bool live(float score, bool fin) { return !fin && isfinite(score); }

// One CTA per (row, span).  keys [rows][splits][K] (0: none), ms [rows][splits]
// references m (-inf: nothing above -inf), sums [rows][splits] of exp(x - m) in
// fp64 (NaN: no distribution).
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) beam_scan_kernel(const T* __restrict__ logits, const float* __restrict__ scores,
                                                             const unsigned char* __restrict__ finished, int V, int K,
                                                             int splits, uint64_t* __restrict__ keys, float* __restrict__ ms,
                                                             double* __restrict__ sums) {
  __shared__ ScanSmem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned full = 0xffffffffu;
  const unsigned at = blockIdx.x, row = at / static_cast<unsigned>(splits);
  const int split = static_cast<int>(at - row * splits);
  griddep_launch_dependents();
  const float score = scores[row];
  const bool fin = finished && finished[row];
  const T* x = logits + static_cast<long long>(row) * V;
  // Vector 0 holds the values before the first 32-byte boundary, vectors 1 ..
  // nvec kPer values each, and nvec + 1 the rest.
  constexpr int P = kPer<T>;
  const int head = min(V, static_cast<int>(((kVec - (reinterpret_cast<uintptr_t>(x) & (kVec - 1))) & (kVec - 1)) / sizeof(T)));
  const int nvec = (V - head) / P;
  const int span = nvec / splits + 1;
  const int v0 = min(nvec, split * span), v1 = min(nvec, v0 + span);   // counted from vector 1

  Vec<T> f, f1;            // this round's values and, on their way, the next one's
  auto load = [&](int vec, Vec<T>& d) {
    if (vec < v1) d.load(x + head + static_cast<long long>(vec) * P);
    else d.clear();
  };
  const int first = v0 + warp * 32 + lane;
  load(first, f);
  if (!live(score, fin)) return;   // the merge does not read this row's lists

  uint64_t* buf = sm.buf[warp];
  const int r = (K + kWarps - 1) / kWarps;
  float tv = -kInf;        // smaller values are not wanted
  float best = -kInf;      // the lane's largest value
  float m = -kInf;         // the warp's reference
  uint64_t minus_m = 0;    // -m twice
  double s = 0.0;          // the lane's sum
  auto announce = [&]() {
    uint32_t o = ordered(best), M = 0;
    for (int i = 0; i < r; ++i) {
      M = __reduce_max_sync(full, o);
      if (lane == __ffs(__ballot_sync(full, o == M)) - 1) o = 0;
    }
    if (lane == 0) sm.lead[warp] = unordered(M);
  };
  auto take = [&](const Vec<T>& f, uint32_t id, int round) {
    const float tm = f.max();
    if (__any_sync(full, tm > m + kSlack)) {
      float M = tm;
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(full, M, o));
      s *= exp(static_cast<double>(m) - static_cast<double>(M));   // the first time: 0 * 0
      m = M;
      minus_m = f2_pack(-m, -m);
    }
    // (nothing above -inf yet: every term is 0, or NaN)
    uint64_t e2[P / 2];
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      float lo, hi;
      f2_unpack(f2_mul(f2_add(f.pair(i), minus_m), f2_pack(kLog2e, kLog2e)), lo, hi);
      e2[i] = f2_pack(ex2(lo), ex2(hi));
    }
#pragma unroll
    for (int i = 0; i < P / 2; i += 4) {   // 8 terms at a time
      float lo, hi;
      f2_unpack(f2_add(f2_add(e2[i], e2[i + 1]), f2_add(e2[i + 2], e2[i + 3])), lo, hi);
      s += static_cast<double>(lo + hi);
    }
    best = fmaxf(best, tm);
    if ((round & (round + 1)) == 0) {   // rounds 0, 1, 3, 7, ...
      if (round > 0) announce();
      float least = sm.lead[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) least = fminf(least, sm.lead[w]);
      tv = fmaxf(tv, least);
    }
    if (__any_sync(full, tm >= tv && tm > -kInf)) {
      if (tm >= tv && tm > -kInf) buf[atomicAdd(&sm.count[warp], 1)] = make_key(tm, id);
      __syncwarp();
      const int count = sm.count[warp];
      if (count > kKeep) {
        const int left = cut_back(buf, count, K, lane);
        if (lane == 0) sm.count[warp] = left;
        if (left == K) tv = fmaxf(tv, key_value(buf[K - 1]));
        __syncwarp();
      }
    }
  };

  if (lane == 0) sm.count[warp] = 0;
  best = fmaxf(best, f.max());
  announce();              // of the first round's values, so that few of them are listed
  __syncthreads();
  int round = 0;
#pragma unroll 1
  for (int vec = first; vec - lane < v1; vec += kThreads, ++round) {
    load(vec + kThreads, f1);
    take(f, vec + 1, round);
    f = f1;
  }
  if (warp == 0) {   // the ends
    const int tail = V - head - nvec * P;
    const int n = lane == 0 && split == 0 ? head : lane == 1 && split == splits - 1 ? tail : 0;
    f.load_part(lane == 0 ? x : x + V - tail, n);
    if (__any_sync(full, n > 0)) take(f, lane == 0 ? 0 : nvec + 1, round);
  }
  // the CTA's list from what the warps' lists hold above the last threshold
  announce();
  int count = sm.count[warp];
  if (count > kMaxK) count = cut_back(buf, count, K, lane);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(full, s, o);
  if (lane == 0) {
    sm.m[warp] = m;
    sm.s[warp] = s;
  }
  if (tid == 0) sm.total = sm.found = 0;
  __syncthreads();
  float least = sm.lead[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) least = fminf(least, sm.lead[w]);
  for (int i = lane; i < count; i += 32)
    if (key_value(buf[i]) >= least) sm.all[atomicAdd(&sm.total, 1)] = buf[i];
  __syncthreads();
  const int total = sm.total;
  for (int i = tid; i < total; i += kThreads) {
    const uint64_t key = sm.all[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < total; ++j) rank += sm.all[j] > key;
    if (rank < K) sm.top[rank] = key;
  }
  __syncthreads();
  // The K best values are among the K best vectors: whatever is left out has K
  // vectors' maxima before it.
  const int tops = min(total, K);
  const float bound = tops == K ? key_value(sm.top[K - 1]) : -kInf;
  uint64_t* found = sm.buf[0];
  for (int i = tid; i < tops * P; i += kThreads) {
    const uint32_t id = key_index(sm.top[i / P]), e = i % P;
    const uint32_t idx = id == 0 ? e : head + (id - 1) * P + e;
    if (idx < static_cast<uint32_t>(id == 0 ? head : V)) {
      const float v = to_f(x[idx]);
      if (v >= bound && v > -kInf) found[atomicAdd(&sm.found, 1)] = make_key(v, idx);
    }
  }
  __syncthreads();
  const int n = sm.found;
  uint64_t* mine = keys + static_cast<size_t>(at) * K;
  for (int i = tid; i < n; i += kThreads) {
    const uint64_t key = found[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += found[j] > key;
    if (rank < K) mine[rank] = key;
  }
  for (int i = n + tid; i < K; i += kThreads) mine[i] = 0;

  // maximum and sum of the CTA.  A NaN logit made its lane's sum NaN; +inf made inf - inf.
  if (warp == 0) {
    const float mw = lane < kWarps ? sm.m[lane] : -kInf;
    float M = mw;
#pragma unroll
    for (int o = 4; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(full, M, o));
    double t = 0.0;
    if (lane < kWarps) t = mw == -kInf ? sm.s[lane] : sm.s[lane] * exp(static_cast<double>(mw) - static_cast<double>(M));
#pragma unroll
    for (int o = 4; o; o >>= 1) t += __shfl_xor_sync(full, t, o);
    if (lane == 0) {
      ms[at] = M;
      sums[at] = t;
    }
  }
}

// A candidate's exact order: higher score, then lower beam, higher logit, lower
// token.  The logit decides within a beam, where the sum of beam score, logit
// and lse may round two logits (1e-30 and 3e-30, say) to one score.
struct Cand {
  double score;
  uint64_t at;    // beam << 32 | token
  float logit;    // 0 for a finished beam
};
__device__ __forceinline__ bool better(const Cand& a, const Cand& b) {
  if (a.score != b.score) return a.score > b.score;
  if (a.logit != b.logit && a.at >> 32 == b.at >> 32) return a.logit > b.logit;
  return a.at < b.at;
}

constexpr int kHeld = (kMergeMost > kMaxW * kMaxK ? kMergeMost : kMaxW * kMaxK) / kThreads;   // entries per thread of the merge
constexpr int kMergeEntries = kMergeMost > kMaxW * kMaxK ? kMergeMost : kMaxW * kMaxK;
// of n candidates spread over the threads, the K-th best of the threads' best
// is reached by at most K ceil(n / threads)
constexpr int kFew = kMaxK * (kMergeEntries / kThreads);
static_assert(kFew >= kThreads, "one entry per thread fits without narrowing");
// fp32 and finite: scores below the type's range count as its lowest
__device__ __forceinline__ float as_float(double s) { return fmaxf(static_cast<float>(s), -3.402823466e38f); }

struct MergeSmem {
  union {
    struct {              // until the beams' sums are formed
      float span_m[kMergeMost];
      double span_s[kMergeMost];
    };
    Cand few[kFew];
  };
  Cand best[kMaxK];
  alignas(16) float tbest[kThreads];   // read four at a time
  double lse[kMaxW];      // NaN: no candidates
  double red[kThreads / 32];
  float redm[kThreads / 32];
  unsigned thr;
  int nfew, again;
  unsigned char redo[kMaxW];
};

static_assert(alignof(MergeSmem) == 16 && offsetof(MergeSmem, tbest) % 16 == 0, "its float4 reads");

// lse of one row in fp64, by the whole CTA.
template <typename T>
__device__ __noinline__ double exact_lse(const T* x, int V, MergeSmem& sm) {
  const unsigned full = 0xffffffffu, n = V;   // unsigned: a thread's last index may pass 2^31 by its stride
  const int tid = threadIdx.x;
  float m = -kInf;
#pragma unroll 8
  for (unsigned i = tid; i < n; i += kThreads) m = fmaxf(m, to_f(x[i]));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(full, m, o));
  __syncthreads();
  if ((tid & 31) == 0) sm.redm[tid >> 5] = m;
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, sm.redm[w]);
  double part[4] = {0.0, 0.0, 0.0, 0.0};   // four in flight; a fixed order
  unsigned i = tid;
  for (; i + 3 * kThreads < n; i += 4 * kThreads) {
#pragma unroll
    for (int k = 0; k < 4; ++k) part[k] += exp(static_cast<double>(to_f(x[i + k * kThreads])) - m);
  }
  for (; i < n; i += kThreads) part[0] += exp(static_cast<double>(to_f(x[i])) - m);
  double s = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(full, s, o);
  if ((tid & 31) == 0) sm.red[tid >> 5] = s;
  __syncthreads();
  double t = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) t += sm.red[w];
  __syncthreads();
  return m + log(t);
}

// One CTA per request.
template <typename T>
__global__ void __launch_bounds__(kThreads) beam_merge_kernel(
    const T* __restrict__ logits, const float* __restrict__ scores, const unsigned char* __restrict__ finished,
    int end_token, int W, int V, int K, int splits, double eps, const uint64_t* __restrict__ keys, const float* __restrict__ ms,
    const double* __restrict__ sums, float* __restrict__ out_scores, int* __restrict__ out_parents,
    int* __restrict__ out_tokens) {
  __shared__ MergeSmem sm;
  const int tid = threadIdx.x;
  const long long g = blockIdx.x;
  const double nan = __longlong_as_double(0x7ff8000000000000ll);
  griddep_wait();

  const int per_row = splits * K;
  const int n = W * per_row;
  uint64_t key[kHeld];   // this thread's entries tid, tid + kThreads, .. of the rows' lists
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int i = tid + j * kThreads;
    key[j] = i < n ? keys[g * n + i] : 0;   // (a finished or dead beam's are not looked at)
  }
  // the spans' maxima and sums, then one thread per beam
  for (int i = tid; i < W * splits; i += kThreads) {
    const long long at = g * W * splits + i;
    const long long row = g * W + i / splits;
    const bool in = live(scores[row], finished && finished[row]);
    sm.span_m[i] = in ? ms[at] : 0.f;
    sm.span_s[i] = in ? sums[at] : nan;
  }
  __syncthreads();
  for (int w = tid; w < W; w += kThreads) {
    double lse = nan;
    float M = -kInf;
    for (int p = 0; p < splits; ++p) M = fmaxf(M, sm.span_m[w * splits + p]);
    if (M > -kInf && M < kInf) {
      double t = 0.0;
      for (int p = 0; p < splits; ++p) {
        const float mp = sm.span_m[w * splits + p];
        // a span of nothing but -inf has sum 0 (NaN if it holds one)
        t += sm.span_s[w * splits + p] * (mp == M || mp == -kInf ? 1.0 : exp(static_cast<double>(mp) - static_cast<double>(M)));
      }
      lse = M + log(t);
    }
    sm.lse[w] = lse;
    sm.redo[w] = 0;
  }
  __syncthreads();

  // entry tid + j kThreads as a candidate; false if it is none
  auto entry = [&](int j, Cand& c) -> bool {
    const int i = tid + j * kThreads;
    if (i >= n) return false;
    const int w = i / per_row;
    const long long row = g * W + w;
    const float sc = scores[row];
    if (finished && finished[row]) {
      if (i != w * per_row || !isfinite(sc)) return false;
      c.score = sc;
      c.at = static_cast<uint64_t>(w) << 32 | static_cast<uint32_t>(end_token);
      c.logit = 0.f;
      return true;
    }
    const double lse = sm.lse[w];
    if (!(lse == lse) || !key[j]) return false;
    c.logit = key_value(key[j]);
    c.score = static_cast<double>(sc) + (static_cast<double>(c.logit) - lse);
    c.at = static_cast<uint64_t>(w) << 32 | key_index(key[j]);
    return true;
  };

  const Cand none = {-__builtin_huge_val(), ~0ull, 0.f};
  for (int round = 0; round < 2; ++round) {
    if (tid == 0) {
      sm.nfew = 0;
      sm.again = 0;
      sm.thr = 0;
    }
    // A bound that at least K candidates reach: the K-th largest of the
    // threads' best in fp32 (rounding keeps the order)
    float mine = -kInf;
    Cand top = none;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (j * kThreads >= n) break;
      Cand c;
      if (entry(j, c) && better(c, top)) top = c, mine = as_float(c.score);
    }
    sm.tbest[tid] = mine;
    __syncthreads();
    if (mine > -kInf) {
      int reach = 0;
#pragma unroll 4
      for (int i = 0; i < kThreads; i += 4) {
        const float4 o = *reinterpret_cast<const float4*>(sm.tbest + i);
        reach += (o.x >= mine) + (o.y >= mine) + (o.z >= mine) + (o.w >= mine);
      }
      if (reach >= K) atomicMax(&sm.thr, ordered(mine));
    }
    __syncthreads();
    const unsigned thr = sm.thr;
    // listed with it: what lies within eps of the bound, so all that is that close
    // to the last chosen one (2^-22: the roundings to fp32)
    const float least = thr ? unordered(thr) : -kInf;
    const float near = least - fmaf(fabsf(least), 0x1p-22f, static_cast<float>(eps));
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (j * kThreads >= n) break;
      Cand c;
      if (!entry(j, c) || as_float(c.score) < near) continue;
      const int at = atomicAdd(&sm.nfew, 1);
      if (at < kFew) sm.few[at] = c;
    }
    __syncthreads();
    const bool many = sm.nfew > kFew;
    if (many) {   // more of them than fit: the bound from exact scores, through the same list
      __syncthreads();
      if (tid == 0) {
        sm.nfew = 0;
        sm.best[0] = none;
      }
      sm.few[tid] = top;
      __syncthreads();
      int rank = 0;
      for (int i = 0; i < kThreads; ++i) rank += better(sm.few[i], top);
      if (rank == K - 1 && top.at != ~0ull) sm.best[0] = top;
      __syncthreads();
      const Cand bound = sm.best[0];
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        if (j * kThreads >= n) break;
        Cand c;
        if (entry(j, c) && !better(bound, c)) sm.few[atomicAdd(&sm.nfew, 1)] = c;
      }
    }
    __syncthreads();
    const int m = sm.nfew;
    for (int i = tid; i < K; i += kThreads) sm.best[i] = none;
    __syncthreads();
    for (int i = tid; i < m; i += kThreads) {
      const Cand c = sm.few[i];
      int rank = 0;
      for (int j = 0; j < m; ++j) rank += better(sm.few[j], c);
      if (rank < K) sm.best[rank] = c;
    }
    __syncthreads();
    if (round == 1 || W == 1) break;
    // candidates of different beams that fp32 sums cannot tell apart: neighbours
    // among the chosen, and what is left out just behind the last of them
    auto compare = [&](const Cand& a, const Cand& b) {
      const uint32_t wa = static_cast<uint32_t>(a.at >> 32), wb = static_cast<uint32_t>(b.at >> 32);
      if (wa == wb || a.score - b.score > eps) return;
      sm.again = 1;
      if (sm.lse[wa] == sm.lse[wa]) sm.redo[wa] = 1;   // (a finished beam has no sum)
      if (sm.lse[wb] == sm.lse[wb]) sm.redo[wb] = 1;
    };
    for (int i = tid; i < K - 1; i += kThreads)
      if (sm.best[i + 1].at != ~0ull) compare(sm.best[i], sm.best[i + 1]);
    const Cand last = sm.best[K - 1];
    if (last.at != ~0ull)
      for (int i = tid; i < m; i += kThreads)
        if (better(last, sm.few[i])) compare(last, sm.few[i]);
    if (many)   // what is close to the last one is not all listed: every beam with a sum
      for (int w = tid; w < W; w += kThreads)
        if (sm.lse[w] == sm.lse[w]) sm.again = sm.redo[w] = 1;
    __syncthreads();
    if (!sm.again) break;
    for (int w = 0; w < W; ++w)
      if (sm.redo[w]) {
        const double e = exact_lse(logits + (g * W + w) * V, V, sm);
        if (tid == 0) sm.lse[w] = e;
      }
    __syncthreads();
  }
  for (int i = tid; i < K; i += kThreads) {
    const Cand c = sm.best[i];
    const bool any = c.at != ~0ull;
    out_scores[g * K + i] = static_cast<float>(c.score);
    out_parents[g * K + i] = any ? static_cast<int>(c.at >> 32) : -1;
    out_tokens[g * K + i] = any ? static_cast<int>(c.at & 0xffffffffu) : -1;
  }
}

// Spans per row: three CTAs for every SM when the rows are fewer (512 rows of
// 50257 in bf16: 26.4 us in one span each, 29.4 in two), spans of at least two rounds of
// every warp, and no more list entries per request than one merge takes.
int beam_splits(long long rows, int W, int V, int K, int per) {   // per: values of a vector
  const long long want = (static_cast<long long>(num_sms()) * 3 + rows - 1) / rows;
  const long long by_len = std::max(1, V / (2 * kThreads * per));
  const long long by_merge = std::max(1, kMergeMost / (W * K));
  return static_cast<int>(std::max(1LL, std::min({want, by_len, by_merge})));
}

struct BeamWs {
  size_t keys, ms, sums, total;
};
BeamWs beam_ws(long long rows, int splits, int K) {
  BeamWs w;
  w.sums = 0;
  w.keys = w.sums + sizeof(double) * rows * splits;
  w.ms = w.keys + sizeof(uint64_t) * rows * splits * K;
  w.total = w.ms + sizeof(float) * rows * splits;
  return w;
}

template <typename T>
cudaError_t run_select(int G, int W, int V, int K, const void* logits, const float* scores, const unsigned char* fin,
                       int end_token, float* os, int* op, int* ot, char* ws, cudaStream_t st) {
  const long long rows = static_cast<long long>(G) * W;
  const int splits = beam_splits(rows, W, V, K, kPer<T>);
  const BeamWs o = beam_ws(rows, splits, K);
  auto* keys = reinterpret_cast<uint64_t*>(ws + o.keys);
  auto* ms = reinterpret_cast<float*>(ws + o.ms);
  auto* sums = reinterpret_cast<double*>(ws + o.sums);
  const T* x = static_cast<const T*>(logits);
  beam_scan_kernel<T><<<static_cast<unsigned>(rows * splits), kThreads, 0, st>>>(x, scores, fin, V, K, splits, keys, ms, sums);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const double eps = 2.0 * (4.2e-7 + 9.3e-8 * std::log2(static_cast<double>(std::max(V, 8))));
  return launch_after(beam_merge_kernel<T>, static_cast<unsigned>(G), kThreads, 0, st, true, x, scores, fin, end_token, W, V, K,
                      splits, eps, keys, ms, sums, os, op, ot);
}

// ------------------------------------------------------------- state reorder
// Reads each followed state once and writes each sequence's: HBM bounds it (16 x 4
// sequences of 16 heads, M 64, d 128, 135 MB each way: 41.0 us, 85 % of the copy
// rate).
//
// Up to three arrays, each [sequences][len] floats.
struct Parts {
  const float* in[3];
  float* out[3];
  long long len[3];    // floats per sequence
  int n;
};

// One vector of VEC floats at one position of a request's sequences per
// thread: with buffers apart, a gather (a parent followed by several beams
// comes from L2 after its first read).
template <int VEC>
__global__ void __launch_bounds__(kThreads) reorder_kernel(const __grid_constant__ Parts p, int win, int wout,
                                                           const int* __restrict__ parents) {
  const long long g = blockIdx.x;
  const int j = blockIdx.z;
  const int par = parents[g * wout + j];
  const bool zero = par < 0 || par >= win;
  for (int a = 0; a < p.n; ++a) {
    const float* in = p.in[a] + (g * win + (zero ? 0 : par)) * p.len[a];
    float* out = p.out[a] + (g * wout + j) * p.len[a];
    const long long stride = static_cast<long long>(gridDim.y) * kThreads * VEC;
    long long i = (static_cast<long long>(blockIdx.y) * kThreads + threadIdx.x) * VEC;
    if constexpr (VEC == 4) {
      const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
      for (; i + 3 * stride < p.len[a]; i += 4 * stride) {
        float4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = zero ? z : *reinterpret_cast<const float4*>(in + i + u * stride);
#pragma unroll
        for (int u = 0; u < 4; ++u) *reinterpret_cast<float4*>(out + i + u * stride) = v[u];
      }
      for (; i < p.len[a]; i += stride)
        *reinterpret_cast<float4*>(out + i) = zero ? z : *reinterpret_cast<const float4*>(in + i);
    } else {
      for (; i < p.len[a]; i += stride) out[i] = zero ? 0.f : in[i];
    }
  }
}

// In place: a thread reads its position of all of a request's beams before it
// writes any, so no beam is overwritten before a follower has read it; beams
// that follow themselves are neither written nor, unless followed, read.
template <int VEC>
__global__ void __launch_bounds__(128) reorder_in_place_kernel(const __grid_constant__ Parts p, int w,
                                                               const int* __restrict__ parents) {
  extern __shared__ __align__(16) float stage[];   // [w][128][VEC]: a thread touches its own column only
  __shared__ int par[64];
  __shared__ unsigned char need[64];
  const long long g = blockIdx.x;
  if (threadIdx.x < 64) need[threadIdx.x] = 0;
  __syncthreads();
  if (threadIdx.x < w) {
    const int q = parents[g * w + threadIdx.x];
    par[threadIdx.x] = q;
    if (q >= 0 && q < w && q != static_cast<int>(threadIdx.x)) need[q] = 1;   // several threads write the same 1
  }
  __syncthreads();
  for (int a = 0; a < p.n; ++a) {
    float* base = p.out[a] + g * w * p.len[a];
    for (long long i = (static_cast<long long>(blockIdx.y) * 128 + threadIdx.x) * VEC; i < p.len[a];
         i += static_cast<long long>(gridDim.y) * 128 * VEC) {
      for (int j = 0; j < w; ++j)
        if (need[j]) {
          float* s = stage + (j * 128 + threadIdx.x) * VEC;
          const float* v = base + j * p.len[a] + i;
          if constexpr (VEC == 4) *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(v);
          else *s = *v;
        }
      for (int j = 0; j < w; ++j) {
        const int q = par[j];
        if (q == j) continue;
        const bool zero = q < 0 || q >= w;
        const float* s = stage + ((zero ? 0 : q) * 128 + threadIdx.x) * VEC;
        float* v = base + j * p.len[a] + i;
        if constexpr (VEC == 4) *reinterpret_cast<float4*>(v) = zero ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(s);
        else *v = zero ? 0.f : *s;
      }
    }
  }
}

cudaError_t run_reorder(const Parts& p, long long groups, int win, int wout, const int* parents, cudaStream_t st) {
  bool vec = true;
  long long longest = 0;
  for (int a = 0; a < p.n; ++a) {
    vec = vec && p.len[a] % 4 == 0 && (reinterpret_cast<uintptr_t>(p.in[a]) & 15) == 0 &&
          (reinterpret_cast<uintptr_t>(p.out[a]) & 15) == 0;
    longest = std::max(longest, p.len[a]);
  }
  const int width = vec ? 4 : 1;
  mark_launch_begin(st);
  if (p.in[0] == p.out[0]) {
    const size_t bytes = sizeof(float) * 128 * width * win;
    auto kern = vec ? reorder_in_place_kernel<4> : reorder_in_place_kernel<1>;
    if (cudaError_t e = allow_smem(kern, bytes); e != cudaSuccess) return e;
    const long long bx = std::max(1LL, std::min((longest + 128 * width - 1) / (128 * width), (16LL * num_sms() + groups - 1) / groups));
    kern<<<dim3(static_cast<unsigned>(groups), static_cast<unsigned>(bx)), 128, bytes, st>>>(p, win, parents);
  } else {
    const long long per = static_cast<long long>(kThreads) * width * 4;
    const long long bx = std::max(1LL, std::min((longest + per - 1) / per, (16LL * num_sms() + groups * wout - 1) / (groups * wout)));
    auto kern = vec ? reorder_kernel<4> : reorder_kernel<1>;
    kern<<<dim3(static_cast<unsigned>(groups), static_cast<unsigned>(bx), static_cast<unsigned>(wout)), kThreads, 0, st>>>(
        p, win, wout, parents);
  }
  mark_launch_end(st);
  return cudaGetLastError();
}

// Checks shared by both reorder calls; bytes: of one sequence's state.
ia_status_t check_reorder(int B, int win, int wout, const int* parents, const void* in, void* out, size_t bytes) {
  if (win <= 0 || wout <= 0 || win > kMaxW || wout > kMaxW || B % win != 0) return IA_ERR_INVALID_ARG;
  if (!parents || !in || !out || !aligned16(in) || !aligned16(out) || (reinterpret_cast<uintptr_t>(parents) & 3u))
    return IA_ERR_INVALID_ARG;
  const uintptr_t x = reinterpret_cast<uintptr_t>(in), y = reinterpret_cast<uintptr_t>(out);
  const size_t nx = bytes * B, ny = bytes * (B / win) * wout;
  if (x == y ? win != wout : (x < y + ny && y < x + nx)) return IA_ERR_INVALID_ARG;
  return IA_OK;
}

int per_vector(ia_dtype_t dt) { return dt == IA_F32 ? kPer<float> : kPer<__nv_bfloat16>; }
bool valid_beam(int G, int W, int V, int K, ia_dtype_t dt) {
  return G > 0 && W > 0 && W <= kMaxW && V > 0 && K > 0 && K <= kMaxK && (dt == IA_F32 || dt == IA_BF16);
}

}  // namespace
}  // namespace ia

using namespace ia;

extern "C" {

size_t ia_beam_select_workspace_bytes(int G, int W, int V, int K, ia_dtype_t dtype) {
  if (!valid_beam(G, W, V, K, dtype)) return 0;
  const long long rows = static_cast<long long>(G) * W;
  return beam_ws(rows, beam_splits(rows, W, V, K, per_vector(dtype)), K).total;
}

ia_status_t ia_beam_select(int G, int W, int V, int K, ia_dtype_t dtype, const void* logits, const float* scores,
                           const unsigned char* finished, int end_token, float* out_scores, int* out_parents,
                           int* out_tokens, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_beam(G, W, V, K, dtype) || !logits || !scores || !out_scores || !out_parents || !out_tokens)
    return IA_ERR_INVALID_ARG;
  const void* ptrs[] = {logits, scores, out_scores, out_parents, out_tokens, workspace};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return IA_ERR_INVALID_ARG;
  if (finished && (end_token < 0 || end_token >= V)) return IA_ERR_INVALID_ARG;
  if (static_cast<long long>(G) * W * beam_splits(static_cast<long long>(G) * W, W, V, K, per_vector(dtype)) > (1LL << 31) - 1)
    return IA_ERR_UNSUPPORTED;   // one block per row and span
  if (!workspace || workspace_bytes < ia_beam_select_workspace_bytes(G, W, V, K, dtype)) return IA_ERR_WORKSPACE;
  if (inject_launch_failure()) return IA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  mark_launch_begin(st);
  const cudaError_t e =
      dtype == IA_BF16
          ? run_select<__nv_bfloat16>(G, W, V, K, logits, scores, finished, end_token, out_scores, out_parents, out_tokens, ws, st)
          : run_select<float>(G, W, V, K, logits, scores, finished, end_token, out_scores, out_parents, out_tokens, ws, st);
  mark_launch_end(st);
  return map_cuda(e);
}

ia_status_t ia_state_reorder(const ia_shape_t* s, int beams_in, int beams_out, const int* parents, const void* state_in,
                             void* state_out, void* stream) {
  if (!valid_dims(s, false)) return IA_ERR_INVALID_ARG;
  const size_t bytes = ia_state_bytes(s) / s->B;
  if (ia_status_t r = check_reorder(s->B, beams_in, beams_out, parents, state_in, state_out, bytes); r != IA_OK) return r;
  if (inject_launch_failure()) return IA_ERR_CUDA;
  const long long unit = 2LL * s->H * s->M, Bi = s->B, Bo = static_cast<long long>(s->B / beams_in) * beams_out;
  const float* in = static_cast<const float*>(state_in);
  float* out = static_cast<float*>(state_out);
  Parts p = {};
  p.n = 3;
  const long long len[3] = {unit * s->d_xi, unit * s->d_v, unit};
  long long oi = 0, oo = 0;
  for (int a = 0; a < 3; ++a) {
    p.in[a] = in + oi;
    p.out[a] = out + oo;
    p.len[a] = len[a];
    oi += len[a] * Bi;
    oo += len[a] * Bo;
  }
  return map_cuda(run_reorder(p, s->B / beams_in, beams_in, beams_out, parents, static_cast<cudaStream_t>(stream)));
}

ia_status_t ia_linear_state_reorder(const ia_linear_shape_t* s, int beams_in, int beams_out, const int* parents,
                                    const float* state_in, float* state_out, void* stream) {
  const size_t total = ia_linear_state_bytes(s);
  if (!total) return IA_ERR_INVALID_ARG;
  if (ia_status_t r = check_reorder(s->B, beams_in, beams_out, parents, state_in, state_out, total / s->B); r != IA_OK)
    return r;
  if (inject_launch_failure()) return IA_ERR_CUDA;
  Parts p = {};
  p.n = 1;
  p.in[0] = state_in;
  p.out[0] = state_out;
  p.len[0] = static_cast<long long>(s->H) * s->d_k * s->d_v;
  return map_cuda(run_reorder(p, s->B / beams_in, beams_in, beams_out, parents, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
