// Beam search: the selection over beams and vocabulary, and the reordering of
// the recurrent states that follows it.
//
// Selection.  Candidate (w, t) of a request scores
//   scores[w] + x[w][t] - lse_w,   lse_w = log sum_t exp(x[w][t]).
// Within a beam the order is that of x, so a beam's K best tokens need no
// lse, and the scan kernel finds both in one pass over the logits (which HBM
// bounds): each CTA takes a span of one row, keeps a running maximum and sum
// of exponentials per thread, and a shared buffer of the values that reach
// the K-th best seen so far.  The merge kernel, one CTA per request, adds the
// spans' sums and picks the K best of the rows' lists.
//
// Order keys.  (value, lower index first) is one 64-bit number: the fp32 value
// mapped to an order-preserving integer above the complement of the index.
// All keys differ, which bounds every buffer: of n keys spread over 256
// threads the K-th largest of the threads' maxima is at most the K-th largest
// key, and only K threads hold keys that reach it, so at most K * ceil(n/256)
// keys do.
//
// Exactness.  Scores of one beam differ exactly as their logits do; across
// beams the order hangs on lse_w, whose fp32 sums are off by at most kLseEps/2
// (a term: 2 ulp of ex2.approx, |t| 2^-24 1.5 ln 2 from the argument, which
// weighs at most 16 e^-11 for the terms below 2^-16; 7 additions inside a tile;
// the tiles add up in fp64).  Where two neighbours in the chosen order come
// from different beams and lie closer than that, the CTA takes those beams'
// sums again in fp64 and orders once more.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ia_device.cuh"
#include "ia_internal.h"
#include "ia_launch.h"

namespace ia {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxW = 64, kMaxK = 64;
constexpr int kPer = 8;                       // values per thread and tile
constexpr int kTile = kThreads * kPer;        // 2048
constexpr int kCap = kTile + 512;             // candidate buffer: a tile on top of 512 kept ones
constexpr int kMergeMost = 4096;              // entries one merge takes
constexpr double kLseEps = 4e-6;
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

// Shared memory of the scan kernel.
struct ScanSmem {
  uint64_t buf[kCap];
  uint64_t few[kMaxK * ((kCap + kThreads - 1) / kThreads)];
  uint64_t tmax[kThreads];
  uint64_t thr;      // no key below this one can be among the K best
  int count, nfew;
  float m[kThreads / 32];
  double s[kThreads / 32];
};

// The K-th largest of the threads' values (0 if fewer than K are not 0), in
// sm.thr if it is larger than what stands there.  All threads call it.
__device__ __forceinline__ void raise_threshold(ScanSmem& sm, uint64_t mine, int K) {
  sm.tmax[threadIdx.x] = mine;
  __syncthreads();
  if (mine) {
    int rank = 0;
    for (int i = 0; i < kThreads; ++i) rank += sm.tmax[i] > mine;
    if (rank == K - 1 && mine > sm.thr) sm.thr = mine;
  }
  __syncthreads();
}

// Keeps the K best keys of the buffer, sorted, in buf[0 .. count).
__device__ __forceinline__ void compact(ScanSmem& sm, int K) {
  const int n = sm.count;
  uint64_t best = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) best = max(best, sm.buf[i]);
  if (threadIdx.x == 0) sm.nfew = 0;
  raise_threshold(sm, best, K);
  const uint64_t thr = sm.thr;
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (sm.buf[i] >= thr) sm.few[atomicAdd(&sm.nfew, 1)] = sm.buf[i];
  __syncthreads();
  const int m = sm.nfew;
  for (int i = threadIdx.x; i < m; i += kThreads) {
    const uint64_t key = sm.few[i];
    int rank = 0;
    for (int j = 0; j < m; ++j) rank += sm.few[j] > key;
    if (rank < K) sm.buf[rank] = key;
    if (rank == K - 1) sm.thr = key;   // only this thread writes; the value is at least the old one
  }
  if (threadIdx.x == 0) sm.count = min(m, K);
  __syncthreads();
}

template <typename T>
__device__ __forceinline__ float to_f(T x) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(x);
  else return x;
}

// kPer values from a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[kPer]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
}

__device__ __forceinline__ bool live(float score, bool fin) { return !fin && isfinite(score); }

// One CTA per (row, span).  keys [rows][splits][K] (0: none), ms [rows][splits]
// maxima, sums [rows][splits] of exp(x - max) in fp64 (NaN: no distribution).
template <typename T>
__global__ void __launch_bounds__(kThreads) beam_scan_kernel(const T* __restrict__ logits, const float* __restrict__ scores,
                                                             const unsigned char* __restrict__ finished, int V, int K,
                                                             int splits, uint64_t* __restrict__ keys, float* __restrict__ ms,
                                                             double* __restrict__ sums) {
  __shared__ ScanSmem sm;
  const int tid = threadIdx.x;
  const long long at = blockIdx.x, row = at / splits;
  const int split = static_cast<int>(at - row * splits);
  griddep_launch_dependents();
  if (!live(scores[row], finished && finished[row])) return;   // the merge does not read this row's lists
  if (tid == 0) sm.thr = 0, sm.count = 0;
  __syncthreads();

  const T* x = logits + row * V;
  // values before the first 16-byte boundary, then whole vectors of kPer, then the rest
  const int head = min(V, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T)));
  const int nvec = (V - head) / kPer;
  const int v0 = static_cast<int>(static_cast<long long>(nvec) * split / splits);
  const int v1 = static_cast<int>(static_cast<long long>(nvec) * (split + 1) / splits);

  float m = -kInf;
  double s = 0.0;
  auto take = [&](const float (&f)[kPer], int idx, bool first) {   // idx: index of f[0]; unused places hold -inf
    float tm = f[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) tm = fmaxf(tm, f[i]);
    if (tm > m) {
      s *= exp(static_cast<double>(m) - static_cast<double>(tm));
      m = tm;
    }
    float e[kPer];
    const float base = m == -kInf ? 0.f : m;   // nothing above -inf yet: every term is 0 (or NaN)
#pragma unroll
    for (int i = 0; i < kPer; ++i) e[i] = ex2((f[i] - base) * kLog2e);
    s += static_cast<double>(((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7])));
    if (first) {   // no threshold yet: it comes from the threads' best
      uint64_t best = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (f[i] > -kInf) best = max(best, make_key(f[i], idx + i));
      raise_threshold(sm, best, K);
    }
    const uint64_t thr = sm.thr;
    const float tv = thr ? key_value(thr) : -kInf;
    if (tm >= tv && tm > -kInf) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (f[i] >= tv && f[i] > -kInf) {
          const uint64_t key = make_key(f[i], idx + i);
          if (key >= thr) sm.buf[atomicAdd(&sm.count, 1)] = key;
        }
    }
    __syncthreads();
    if (sm.count > kCap - kTile) compact(sm, K);
    else __syncthreads();
  };

  const int ntile = (v1 - v0 + kThreads - 1) / kThreads;
  for (int t = 0; t < ntile; ++t) {
    const int vec = v0 + t * kThreads + tid;
    float f[kPer];
    if (vec < v1) load8(x + head + static_cast<long long>(vec) * kPer, f);
    else
#pragma unroll
      for (int i = 0; i < kPer; ++i) f[i] = -kInf;
    take(f, head + vec * kPer, t == 0);
  }
  {   // the ends: head values by the first span, tail values by the last (each fewer than one vector)
    const int tail0 = head + nvec * kPer;
    const int n_head = split == 0 ? head : 0, n_tail = split == splits - 1 ? V - tail0 : 0;
    const int idx = tid < n_head ? tid : tid - n_head < n_tail ? tail0 + tid - n_head : -1;
    float f[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) f[i] = -kInf;
    if (idx >= 0) f[0] = to_f(x[idx]);
    take(f, idx, ntile == 0);
  }
  compact(sm, K);
  if (tid < K) keys[at * K + tid] = tid < sm.count ? sm.buf[tid] : 0;

  // maximum and sum of the CTA.  A NaN logit made its thread's sum NaN; +inf made inf - inf.
  const unsigned full = 0xffffffffu;
  float M = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(full, M, o));
  if ((tid & 31) == 0) sm.m[tid >> 5] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) M = fmaxf(M, sm.m[w]);
  double part = m == -kInf ? s : s * exp(static_cast<double>(m) - static_cast<double>(M));
#pragma unroll
  for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(full, part, o);
  if ((tid & 31) == 0) sm.s[tid >> 5] = part;
  __syncthreads();
  if (tid == 0) {
    double t = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) t += sm.s[w];
    ms[at] = M;
    sums[at] = t;
  }
}

struct Cand {   // a candidate's exact order: higher score, then lower beam and token
  double score;
  uint64_t at;   // beam << 32 | token
};
__device__ __forceinline__ bool better(const Cand& a, const Cand& b) {
  return a.score > b.score || (a.score == b.score && a.at < b.at);
}

struct MergeSmem {
  Cand few[(kMaxK + 1) * (kMergeMost / kThreads)];
  Cand best[kMaxK + 1];
  double tscore[kThreads];
  uint64_t tat[kThreads];
  double lse[kMaxW];      // NaN: no candidates
  double red[kThreads / 32];
  float redm[kThreads / 32];
  Cand thr;
  int nfew, again;
  unsigned char redo[kMaxW];
};

// lse of one row in fp64, by the whole CTA.
template <typename T>
__device__ double exact_lse(const T* x, int V, MergeSmem& sm) {
  const unsigned full = 0xffffffffu;
  const int tid = threadIdx.x;
  float m = -kInf;
  for (int i = tid; i < V; i += kThreads) m = fmaxf(m, to_f(x[i]));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(full, m, o));
  __syncthreads();
  if ((tid & 31) == 0) sm.redm[tid >> 5] = m;
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, sm.redm[w]);
  double s = 0.0;
  for (int i = tid; i < V; i += kThreads) s += exp(static_cast<double>(to_f(x[i])) - m);
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
    int end_token, int W, int V, int K, int splits, const uint64_t* __restrict__ keys, const float* __restrict__ ms,
    const double* __restrict__ sums, float* __restrict__ out_scores, int* __restrict__ out_parents,
    int* __restrict__ out_tokens) {
  __shared__ MergeSmem sm;
  const int tid = threadIdx.x;
  const long long g = blockIdx.x;
  const double nan = __longlong_as_double(0x7ff8000000000000ll);
  griddep_wait();

  for (int w = tid; w < W; w += kThreads) {
    const long long row = g * W + w;
    double lse = nan;
    if (live(scores[row], finished && finished[row])) {
      float M = -kInf;
      for (int p = 0; p < splits; ++p) M = fmaxf(M, ms[row * splits + p]);
      if (M > -kInf && M < kInf) {
        double t = 0.0;
        for (int p = 0; p < splits; ++p) {
          const float mp = ms[row * splits + p];
          // a span of nothing but -inf has sum 0 (NaN if it holds one)
          t += sums[row * splits + p] * (mp == -kInf ? 1.0 : exp(static_cast<double>(mp) - static_cast<double>(M)));
        }
        lse = M + log(t);
      }
    }
    sm.lse[w] = lse;
    sm.redo[w] = 0;
  }
  __syncthreads();

  const int per_row = splits * K;
  const int n = W * per_row;
  // entry i of the rows' lists as a candidate; false if it is none
  auto entry = [&](int i, Cand& c) -> bool {
    const int w = i / per_row, j = i - w * per_row;
    const long long row = g * W + w;
    const float sc = scores[row];
    if (finished && finished[row]) {
      if (j != 0 || !isfinite(sc)) return false;
      c.score = sc;
      c.at = static_cast<uint64_t>(w) << 32 | static_cast<uint32_t>(end_token);
      return true;
    }
    const double lse = sm.lse[w];
    if (!(lse == lse)) return false;
    const uint64_t key = keys[row * per_row + j];
    if (!key) return false;
    c.score = static_cast<double>(sc) + (static_cast<double>(key_value(key)) - lse);
    c.at = static_cast<uint64_t>(w) << 32 | key_index(key);
    return true;
  };

  const Cand none = {-__builtin_huge_val(), ~0ull};
  const int K1 = K + 1;   // one more than wanted, to see how close the first one left out is
  for (int round = 0; round < 2; ++round) {
    if (tid == 0) {
      sm.nfew = 0;
      sm.again = 0;
      sm.thr = none;
    }
    Cand mine = none;
    for (int i = tid; i < n; i += kThreads) {
      Cand c;
      if (entry(i, c) && better(c, mine)) mine = c;
    }
    sm.tscore[tid] = mine.score;
    sm.tat[tid] = mine.at;
    __syncthreads();
    if (mine.at != ~0ull) {
      int rank = 0;
      for (int i = 0; i < kThreads; ++i) rank += better(Cand{sm.tscore[i], sm.tat[i]}, mine);
      if (rank == K1 - 1) sm.thr = mine;
    }
    __syncthreads();
    const Cand thr = sm.thr;
    for (int i = tid; i < n; i += kThreads) {
      Cand c;
      if (entry(i, c) && !better(thr, c)) sm.few[atomicAdd(&sm.nfew, 1)] = c;
    }
    __syncthreads();
    const int m = sm.nfew;
    for (int i = tid; i < K1; i += kThreads) sm.best[i] = none;
    __syncthreads();
    for (int i = tid; i < m; i += kThreads) {
      const Cand c = sm.few[i];
      int rank = 0;
      for (int j = 0; j < m; ++j) rank += better(sm.few[j], c);
      if (rank < K1) sm.best[rank] = c;
    }
    __syncthreads();
    if (round == 1) break;
    // neighbours from different beams that fp32 sums cannot tell apart
    for (int i = tid; i < K; i += kThreads) {
      const Cand a = sm.best[i], b = sm.best[i + 1];
      const uint32_t wa = static_cast<uint32_t>(a.at >> 32), wb = static_cast<uint32_t>(b.at >> 32);
      if (b.at == ~0ull || wa == wb || a.score - b.score > kLseEps) continue;
      sm.again = 1;
      if (sm.lse[wa] == sm.lse[wa]) sm.redo[wa] = 1;   // (a finished beam has no sum)
      if (sm.lse[wb] == sm.lse[wb]) sm.redo[wb] = 1;
    }
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

// Spans per row: enough CTAs for every SM to hold several, spans of at least
// four tiles, and no more list entries per request than one merge takes.
int beam_splits(long long rows, int W, int V, int K) {
  const long long want = (static_cast<long long>(num_sms()) * 4 + rows - 1) / rows;
  const long long by_len = std::max(1, V / (4 * kTile));
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
  const int splits = beam_splits(rows, W, V, K);
  const BeamWs o = beam_ws(rows, splits, K);
  auto* keys = reinterpret_cast<uint64_t*>(ws + o.keys);
  auto* ms = reinterpret_cast<float*>(ws + o.ms);
  auto* sums = reinterpret_cast<double*>(ws + o.sums);
  const T* x = static_cast<const T*>(logits);
  beam_scan_kernel<T><<<static_cast<unsigned>(rows * splits), kThreads, 0, st>>>(x, scores, fin, V, K, splits, keys, ms, sums);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(beam_merge_kernel<T>, static_cast<unsigned>(G), kThreads, 0, st, true, x, scores, fin, end_token, W, V, K,
                      splits, keys, ms, sums, os, op, ot);
}

// ------------------------------------------------------------- state reorder
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
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e != cudaSuccess) return e;
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

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

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
  return beam_ws(rows, beam_splits(rows, W, V, K), K).total;
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
  if (static_cast<long long>(G) * W * beam_splits(static_cast<long long>(G) * W, W, V, K) > (1LL << 31) - 1)
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
