// Layer norm over rows of D values, forward and backward.
//
//   mean = sum(x)/D,  var = sum((x - mean)^2)/D,  rstd = 1/sqrt(var + eps)
//   y  = (x - mean) rstd w + b
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),  g = dy w,  xhat = (x - mean) rstd
//   dw = sum_rows dy xhat,  db = sum_rows dy
//
// Both directions touch every value once (2 and 3 row-sized streams), so HBM
// bounds them.  A row is held in registers by a group of threads (a warp where
// its registers suffice), which makes the variance a second pass over
// registers instead of a difference of large sums: about the mean of the warp's
// own values, so that several warps exchange mean, squares and number once
// instead of first one sum and then the other.  The rows to come are on
// their way meanwhile: every thread copies its own vectors of the next rows
// into its own slots of shared memory (cp.async), two or three rows ahead, which
// takes neither registers nor barriers.  One row ahead in registers kept 32 KB
// per SM in flight, half of what HBM's latency asks for.
//
// Loads and stores are 16 bytes wide whatever the row length: a group takes
// every TG-th row with TG a multiple of the values per vector, so all its rows
// start at the same offset from a 16-byte boundary, and its vectors are laid
// from that boundary; a copy stops at the row's end, and the vectors across a
// row's ends are stored value by value.
//
// The backward pass keeps a thread's columns fixed while its group walks rows,
// so dw and db accumulate in registers in fp32; the groups of a block add
// theirs in shared memory, the block writes one partial row, and a second
// kernel adds the blocks' rows in a fixed order: no atomics, equal bits from
// equal calls.  Rows wider than the registers hold (12280 columns) are read
// again from L2 instead.
//
// Measured (a graph of calls; rows of up to 126 MB stay in L2): 16384 x 1024 bf16
// forward 14.9 us, backward 24.6 (67 and 101 MB: 10.2 and 15.4 at HBM's rate);
// 131072 x 128 fp32 22.4 and 37.7 (20.5, 30.7); 5003 x 777 fp32 9.5 and 15.8 (4.7,
// 7.1); 2048 x 8192 bf16 25.1 and 31.7 (10.2, 15.4).  The forms that hold 24 values a
// thread spill (backward 64 to 128 bytes a thread).  Instructions bound bf16 rows
// of the forward pass (two exchanges a row and sizes and addresses formed per
// copy: 394 a warp and row at D = 1024, 17.3 us), beside the launch and the first
// rows' latency; ragged rows pay for their ends, and rows above 4096 columns read
// the weights again for every row.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "ia_device.cuh"
#include "ia_internal.h"
#include "ia_launch.h"
#include "ia_rows.h"

namespace ia {
namespace {

constexpr int kMaxHeld = 12280;   // widest row held in registers (512 threads, 24 values, less what an offset takes)

__device__ __forceinline__ uint64_t f2_twice(float x) { return f2_pack(x, x); }
__device__ __forceinline__ float f2_sum(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return lo + hi;
}

// One value as fp32, and back.
template <typename T>
__device__ __forceinline__ float ld1(const T* p, long long i) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(p[i]);
  else return p[i];
}
template <typename T>
__device__ __forceinline__ void st1(T* p, long long i, float f) {
  if constexpr (sizeof(T) == 2) p[i] = __float2bfloat16(f);
  else p[i] = f;
}

// 16 bytes: V values of a row from column c on.
template <typename T>
struct Vec {
  static constexpr int V = 16 / sizeof(T);
  uint4 u;
  // In flight to `slot` (own to the thread) until the copies' group is awaited.
  // Values at and past D become zero; those before the row (c < 0) are the
  // previous row's and are cleared by get().
  // ALIGNED: whole vectors only; slots of columns past D are cleared beforehand.
  // mis: the row's first element modulo V.
  template <bool ALIGNED>
  static __device__ __forceinline__ void fetch(uint4* slot, const T* row, int c, int D, int mis) {
    if (ALIGNED) {
      if (c < D) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slot)), "l"(row + c) : "memory");
      return;
    }
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(slot)), "l"(row + copy_column(c, D, mis)),
                 "r"(copy_bytes(c, D, sizeof(T)))
                 : "memory");
  }
  template <bool ALIGNED>
  __device__ __forceinline__ void store(T* row, int c, int D) const {
    if (c >= 0 && c + V <= D) {
      *reinterpret_cast<uint4*>(row + c) = u;
    } else if (!ALIGNED) {
      float f[V];
      get(f);
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (c + e >= 0 && c + e < D) st1(row, c + e, f[e]);
    }
  }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (V == 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {   // a bf16 is the high half of an fp32
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
    }
  }
  // The row's values in pairs (the arithmetic is packed: with single
  // instructions the backward pass of bf16 rows was bound by issue slots).
  template <bool ALIGNED>
  __device__ __forceinline__ void get_row(uint64_t* p, int c) const {
    float f[V];
    get(f);
    if (!ALIGNED && c < 0)
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (c + e < 0) f[e] = 0.f;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) p[i] = f2_pack(f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ void put_pairs(const uint64_t* p) {
    float f[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f2_unpack(p[i], f[2 * i], f[2 * i + 1]);
    put(f);
  }
  __device__ __forceinline__ void put(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (V == 8) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[i] = __float_as_uint(f[i]);
      }
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Rows of a thread in shared memory (the current one among them), by its
// vectors per row: 64 to 130 KB per SM in flight.
constexpr int fwd_depth(int nv) { return nv == 1 ? 4 : 3; }
constexpr int bwd_depth(int nv2) { return nv2 <= 2 ? 6 : nv2 <= 4 ? 4 : nv2 <= 8 ? 3 : 2; }
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N groups of the thread's copies have landed.
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Sums NV values over the lanes of a group in one warp (tpr threads a group, a
// power of two up to 32 or a multiple of 32).  All lanes call it together.
template <int NV>
__device__ __forceinline__ void warp_sum(float (&x)[NV], int tpr) {
  if (tpr >= 32) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < NV; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
  } else {
    for (int o = tpr >> 1; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < NV; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
  }
}

// Sums NV values over a group: in its warps, then one word per warp in shared
// memory.  `slot` alternates between two buffers so that one barrier per call
// is enough.
template <int NV>
__device__ __forceinline__ void group_sum(float (&x)[NV], int tpr, int group, int gt, float* buf, int slot) {
  warp_sum<NV>(x, tpr);
  if (tpr <= 32) return;
  float* b = buf + (group * 2 + slot) * 32 * NV;
  const int w = gt >> 5, nw = tpr >> 5;
  if ((gt & 31) == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) b[w * NV + i] = x[i];
  named_sync(1 + group, tpr);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float t = 0.f;
    for (int k = 0; k < nw; ++k) t += b[k * NV + i];
    x[i] = t;
  }
}

// V parameters in pairs from column c on (`none` outside the row, and without a pointer).
template <int V, bool ALIGNED>
__device__ __forceinline__ void load_params(const float* __restrict__ p, int c, int D, float none, uint64_t* q) {
  if (p && (ALIGNED ? c < D : (c % 4 == 0 && c >= 0 && c + V <= D))) {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(p + c + e));
      q[e / 2] = f2_pack(u.x, u.y), q[e / 2 + 1] = f2_pack(u.z, u.w);
    }
  } else if (ALIGNED || !p) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) q[i] = f2_twice(none);
  } else {
    float f[V];
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = c + e >= 0 && c + e < D ? __ldg(p + c + e) : none;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) q[i] = f2_pack(f[2 * i], f[2 * i + 1]);
  }
}

// Forward: blocks of 256 threads per SM, by values per thread (ragged rows of 16
// values spill with three blocks: 20000 x 777 fp32 38.1 us, 27.7 with two).
// Backward: one block of up to 512 threads per SM.
constexpr int fwd_ctas(int E, bool aligned) { return E == 8 ? 4 : E == 16 ? (aligned ? 3 : 2) : 1; }

// NV vectors per thread: vector j of thread t covers the columns from
// (j tpr + t) V - mis on, mis the group's offset from a 16-byte boundary.
// HOLD: weights and biases stay in registers.
template <typename T, int NV, bool HOLD, bool ALIGNED>
__global__ void __launch_bounds__(HOLD ? 256 : 512, HOLD ? fwd_ctas(NV * Vec<T>::V, ALIGNED) : 1) ln_fwd_kernel(long long rows, int D, int tpr, const T* x,
                                                     const float* __restrict__ w, const float* __restrict__ b, float eps,
                                                     T* y, float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  constexpr int V = Vec<T>::V, E = NV * V, kAhead = fwd_depth(NV);
  __shared__ float4 buf[16 * 2 * 16];   // [groups][2][warps]: mean, squares about it, number of values
  const int group = threadIdx.x / tpr, gt = threadIdx.x - group * tpr, groups = blockDim.x / tpr;
  const float inv = 1.f / static_cast<float>(D);
  const long long step = static_cast<long long>(gridDim.x) * groups;
  long long row = static_cast<long long>(blockIdx.x) * groups + group;
  const int mis = static_cast<int>(row * D % V);
  int slot = 0, at = 0;
  extern __shared__ uint4 ring[];   // [kAhead][NV][threads]
  const T* ahead = x + row * D;     // the row to fetch next
  int left = row < rows ? static_cast<int>((rows - 1 - row) / step) + 1 : 0;   // rows that are not fetched yet
  auto fetch = [&](int k) {
    if (left > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        Vec<T>::template fetch<ALIGNED>(ring + (k * NV + j) * blockDim.x + threadIdx.x, ahead, (j * tpr + gt) * V - mis, D, mis);
      ahead += step * D;
      --left;
    }
    copies_commit();
  };
  if (ALIGNED)
    for (int k = 0; k < kAhead * NV; ++k)
      if ((k % NV * tpr + gt) * V >= D) ring[k * blockDim.x + threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int k = 0; k < kAhead - 1; ++k) fetch(k);
  uint64_t held_w[HOLD ? E / 2 : 1], held_b[HOLD ? E / 2 : 1];
  if (HOLD)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load_params<V, ALIGNED>(w, (j * tpr + gt) * V - mis, D, 1.f, held_w + j * V / 2);
      load_params<V, ALIGNED>(b, (j * tpr + gt) * V - mis, D, 0.f, held_b + j * V / 2);
    }
  // values of the row that this warp holds, where several share it
  float count[1] = {0.f};
  if (tpr > 32) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * tpr + gt) * V - mis;
      count[0] += static_cast<float>(max(0, min(D, c + V) - max(0, c)));
    }
    warp_sum<1>(count, 32);
  }
  const float warp_inv = tpr <= 32 ? inv : count[0] > 0.f ? 1.f / count[0] : 0.f;
  const int nw = tpr >> 5;
  int nw2 = 1;   // a power of two from nw on
  while (nw2 < nw) nw2 *= 2;
  const int sub = tpr < 32 ? group % (32 / tpr) : 0;   // rows of a warp's groups follow one another
  T* out_row = y + row * D;
  for (; row - sub < rows; row += step, out_row += step * D) {
    const bool in = row < rows;
    fetch(at == 0 ? kAhead - 1 : at - 1);
    copies_wait<kAhead - 1>();
    uint64_t v[E / 2];
    float s[1];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      Vec<T> q;
      q.u = ring[(at * NV + j) * blockDim.x + threadIdx.x];
      q.template get_row<ALIGNED>(v + j * V / 2, (j * tpr + gt) * V - mis);
    }
    at = at + 1 == kAhead ? 0 : at + 1;
    uint64_t t = 0ull;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) t = f2_add(t, v[i]);
    s[0] = f2_sum(t);
    warp_sum<1>(s, tpr);
    const float near = s[0] * warp_inv;   // the mean of the warp's values
    const uint64_t minus = f2_twice(-near);
    t = 0ull;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * tpr + gt) * V - mis;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) v[j * V / 2 + i] = f2_add(v[j * V / 2 + i], minus);
      if (!ALIGNED && (c < 0 || c + V > D)) {   // centred values outside the row do not count
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          float lo, hi;
          f2_unpack(v[j * V / 2 + i], lo, hi);
          const int k = c + 2 * i;
          v[j * V / 2 + i] = f2_pack(k >= 0 && k < D ? lo : 0.f, k + 1 >= 0 && k + 1 < D ? hi : 0.f);
        }
      }
      if (c < D)
#pragma unroll
        for (int i = 0; i < V / 2; ++i) t = f2_fma(v[j * V / 2 + i], v[j * V / 2 + i], t);
    }
    s[0] = f2_sum(t);
    warp_sum<1>(s, tpr);
    float mean = near;
    if (tpr > 32) {
      // The warps' means m, squares M about them and numbers n of values join
      // in one exchange: mean = sum n m / D, squares = sum M + n (m - mean)^2.
      float4* p = buf + (group * 2 + slot) * 16;
      if ((gt & 31) == 0) p[gt >> 5] = make_float4(near, s[0], count[0], 0.f);
      slot ^= 1;
      named_sync(1 + group, tpr);
      const int k = gt & (nw2 - 1);
      const float4 m = k < nw ? p[k] : make_float4(0.f, 0.f, 0.f, 0.f);
      mean = m.z * m.x;
      for (int o = 1; o < nw2; o *= 2) mean += __shfl_xor_sync(0xffffffffu, mean, o);
      mean *= inv;
      const float d = m.x - mean;
      s[0] = fmaf(m.z * d, d, m.y);
      for (int o = 1; o < nw2; o *= 2) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
    }
    const float rstd = __frsqrt_rn(fmaf(s[0], inv, eps));
    const uint64_t r2 = f2_twice(rstd), d2 = f2_twice((near - mean) * rstd);   // (x - near) rstd + d2 is xhat
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * tpr + gt) * V - mis;
      if (c >= D || !in) continue;
      uint64_t wv[V / 2], bv[V / 2], r[V / 2];
      if (!HOLD) {
        load_params<V, ALIGNED>(w, c, D, 1.f, wv);
        load_params<V, ALIGNED>(b, c, D, 0.f, bv);
      }
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const int k = j * V / 2 + i;
        r[i] = f2_fma(f2_fma(v[k], r2, d2), HOLD ? held_w[k] : wv[i], HOLD ? held_b[k] : bv[i]);
      }
      Vec<T> out;
      out.put_pairs(r);
      out.template store<ALIGNED>(out_row, c, D);
    }
    if (gt == 0 && in) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
  }
}

// part: [gridDim.x][2][D] partial sums of dw and db (null: neither is wanted).
// HOLD: the weights stay in registers too.
template <typename T, int NV, bool HOLD, bool ALIGNED>
__global__ void __launch_bounds__(512, 1) ln_bwd_kernel(long long rows, int D, int tpr, const T* dy, const T* x,
                                                     const float* __restrict__ w, const float* __restrict__ mean_in,
                                                     const float* __restrict__ rstd_in, T* dx, float* __restrict__ part) {
  constexpr int V = Vec<T>::V, E = NV * V, kAhead = bwd_depth(2 * NV);
  __shared__ float buf[16 * 2 * 32 * 2];
  const int group = threadIdx.x / tpr, gt = threadIdx.x - group * tpr, groups = blockDim.x / tpr;
  const float inv = 1.f / static_cast<float>(D);
  griddep_launch_dependents();
  const long long step = static_cast<long long>(gridDim.x) * groups;
  long long row = static_cast<long long>(blockIdx.x) * groups + group;
  const int mis = static_cast<int>(row * D % V);
  uint64_t aw[E / 2], ab[E / 2], held[HOLD ? E / 2 : 1];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) aw[i] = ab[i] = 0ull;
  if (HOLD)
#pragma unroll
    for (int j = 0; j < NV; ++j) load_params<V, ALIGNED>(w, (j * tpr + gt) * V - mis, D, 1.f, held + j * V / 2);
  int slot = 0, at = 0;
  extern __shared__ uint4 ring[];   // [kAhead][2 NV][threads]; at the end the groups' sums, [groups][2][D]
  long long ahead = row * D;   // offset of the row to fetch next
  int left = row < rows ? static_cast<int>((rows - 1 - row) / step) + 1 : 0;   // rows that are not fetched yet
  auto fetch = [&](int k) {
    if (left > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * tpr + gt) * V - mis;
        uint4* q = ring + (k * 2 * NV + j) * blockDim.x + threadIdx.x;
        Vec<T>::template fetch<ALIGNED>(q, x + ahead, c, D, mis);
        Vec<T>::template fetch<ALIGNED>(q + NV * blockDim.x, dy + ahead, c, D, mis);
      }
      ahead += step * D;
      --left;
    }
    copies_commit();
  };
  if (ALIGNED)
    for (int k = 0; k < kAhead * 2 * NV; ++k)
      if ((k % NV * tpr + gt) * V >= D) ring[k * blockDim.x + threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
  float next_mean, next_rstd;   // a row ahead: their latency is an iteration's
  auto statistics = [&](long long r) {
    next_mean = r < rows ? mean_in[r] : 0.f;
    next_rstd = r < rows ? rstd_in[r] : 0.f;
  };
  statistics(row);
#pragma unroll
  for (int k = 0; k < kAhead - 1; ++k) fetch(k);
  const int sub = tpr < 32 ? group % (32 / tpr) : 0;   // rows of a warp's groups follow one another
  T* out_row = dx + row * D;
  for (; row - sub < rows; row += step, out_row += step * D) {
    const bool in = row < rows;
    const float mean = next_mean, rstd = next_rstd;
    statistics(row + step);
    fetch(at == 0 ? kAhead - 1 : at - 1);
    copies_wait<kAhead - 1>();
    uint64_t hat[E / 2], g[E / 2];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * tpr + gt) * V - mis;
      const uint4* q = ring + (at * 2 * NV + j) * blockDim.x + threadIdx.x;
      Vec<T> r;
      r.u = in ? q[0] : make_uint4(0u, 0u, 0u, 0u);   // (a warp's last rows: this group has none, and adds nothing)
      r.template get_row<ALIGNED>(hat + j * V / 2, c);
      r.u = in ? q[NV * blockDim.x] : make_uint4(0u, 0u, 0u, 0u);
      r.template get_row<ALIGNED>(g + j * V / 2, c);
    }
    at = at + 1 == kAhead ? 0 : at + 1;
    const uint64_t minus = f2_twice(-mean), r2 = f2_twice(rstd);
    uint64_t t0 = 0ull, t1 = 0ull;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint64_t wv[V / 2];
      if (!HOLD) load_params<V, ALIGNED>(w, (j * tpr + gt) * V - mis, D, 1.f, wv);
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {   // outside the row g is 0 and adds nothing
        const int i = j * V / 2 + k;
        hat[i] = f2_mul(f2_add(hat[i], minus), r2);
        aw[i] = f2_fma(g[i], hat[i], aw[i]);
        ab[i] = f2_add(ab[i], g[i]);
        g[i] = f2_mul(g[i], HOLD ? held[i] : wv[k]);
        t0 = f2_add(t0, g[i]);
        t1 = f2_fma(g[i], hat[i], t1);
      }
    }
    float s[2] = {f2_sum(t0), f2_sum(t1)};
    group_sum<2>(s, tpr, group, gt, buf, slot);
    slot ^= 1;
    const uint64_t c1 = f2_twice(-s[0] * inv), c2 = f2_twice(-s[1] * inv);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * tpr + gt) * V - mis;
      if (c >= D || !in) continue;
      uint64_t r[V / 2];
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        const int i = j * V / 2 + k;
        r[k] = f2_mul(r2, f2_fma(hat[i], c2, f2_add(g[i], c1)));
      }
      Vec<T> out;
      out.put_pairs(r);
      out.template store<ALIGNED>(out_row, c, D);
    }
  }
  if (!part) return;
  float* out = part + static_cast<long long>(blockIdx.x) * 2 * D;
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (groups > 1) __syncthreads();   // every thread is done with its slots
  float* own = groups == 1 ? out : reinterpret_cast<float*>(ring) + group * 2 * D;   // this group's sums
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * tpr + gt) * V - mis;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint64_t* p = (k ? ab : aw) + j * V / 2;
      float* q = own + k * D;
      if (ALIGNED) {
        if (c < D)
#pragma unroll
          for (int i = 0; i < V / 2; i += 2) *reinterpret_cast<ulonglong2*>(q + c + 2 * i) = make_ulonglong2(p[i], p[i + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          float lo, hi;
          f2_unpack(p[i], lo, hi);
          const int at2 = c + 2 * i;
          if (at2 >= 0 && at2 < D) q[at2] = lo;
          if (at2 + 1 >= 0 && at2 + 1 < D) q[at2 + 1] = hi;
        }
      }
    }
  }
  if (groups == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += blockDim.x) {   // the groups in order
    float t = 0.f;
    for (int gr = 0; gr < groups; ++gr) t += reinterpret_cast<const float*>(ring)[gr * 2 * D + c];
    out[c] = t;
  }
}

// ---- rows too wide for registers: one block per row, values read again
template <typename T>
__global__ void __launch_bounds__(512) ln_fwd_wide_kernel(long long rows, int D, const T* x, const float* w,
                                                          const float* b, float eps, T* y, float* mean_out,
                                                          float* rstd_out) {
  __shared__ float buf[2 * 32];
  int slot = 0;
  for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + row * D;
    float s[1] = {0.f};
    for (int c = threadIdx.x; c < D; c += 512) s[0] += ld1(xr, c);
    group_sum<1>(s, 512, 0, threadIdx.x, buf, slot);
    slot ^= 1;
    const float mean = s[0] / D;
    s[0] = 0.f;
    for (int c = threadIdx.x; c < D; c += 512) {
      const float d = ld1(xr, c) - mean;
      s[0] = fmaf(d, d, s[0]);
    }
    group_sum<1>(s, 512, 0, threadIdx.x, buf, slot);
    slot ^= 1;
    const float rstd = 1.f / sqrtf(s[0] / D + eps);
    for (int c = threadIdx.x; c < D; c += 512) {
      const float r = fmaf((ld1(xr, c) - mean) * rstd, w ? w[c] : 1.f, b ? b[c] : 0.f);
      st1(y, row * D + c, r);
    }
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
  }
}

// Column sums first read every value, so they run before dx may overwrite it.
template <typename T>
__global__ void __launch_bounds__(256) ln_columns_wide_kernel(long long rows, int D, const T* dy, const T* x,
                                                              const float* mean, const float* rstd, float* part) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= D) return;
  float aw = 0.f, ab = 0.f;
  for (long long r = blockIdx.y; r < rows; r += gridDim.y) {
    const float d = ld1(dy, r * D + c);
    aw = fmaf(d, (ld1(x, r * D + c) - mean[r]) * rstd[r], aw);
    ab += d;
  }
  part[static_cast<long long>(blockIdx.y) * 2 * D + c] = aw;
  part[static_cast<long long>(blockIdx.y) * 2 * D + D + c] = ab;
}

template <typename T>
__global__ void __launch_bounds__(512) ln_bwd_wide_kernel(long long rows, int D, const T* dy, const T* x, const float* w,
                                                          const float* mean_in, const float* rstd_in, T* dx) {
  __shared__ float buf[2 * 32 * 2];
  int slot = 0;
  for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
    const T *xr = x + row * D, *dr = dy + row * D;
    const float mean = mean_in[row], rstd = rstd_in[row];
    float s[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < D; c += 512) {
      const float g = ld1(dr, c) * (w ? w[c] : 1.f);
      s[0] += g;
      s[1] = fmaf(g, (ld1(xr, c) - mean) * rstd, s[1]);
    }
    group_sum<2>(s, 512, 0, threadIdx.x, buf, slot);
    slot ^= 1;
    const float c1 = s[0] / D, c2 = s[1] / D;
    for (int c = threadIdx.x; c < D; c += 512) {
      const float g = ld1(dr, c) * (w ? w[c] : 1.f);
      const float r = rstd * (g - c1 - (ld1(xr, c) - mean) * rstd * c2);
      st1(dx, row * D + c, r);
    }
  }
}

// dw[c], db[c] = sums of the partial rows: 32 columns x 32 row lanes per block,
// a lane's loads in flight together, the lanes' sums added in order.
__global__ void __launch_bounds__(1024) ln_reduce_kernel(int D, int nparts, const float* __restrict__ part,
                                                         float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sm[32][33];
  griddep_wait();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;   // columns of [2 D]
  float t = 0.f;
  if (c < 2 * D)
#pragma unroll 1
    for (int i = r; i < nparts; i += 256) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = i + 32 * k < nparts ? part[static_cast<long long>(i + 32 * k) * 2 * D + c] : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) t += v[k];
    }
  sm[r][threadIdx.x & 31] = t;
  __syncthreads();
  if (r == 0 && c < 2 * D) {
#pragma unroll
    for (int i = 1; i < 32; ++i) t += sm[i][threadIdx.x & 31];
    if (c < D) {
      if (dw) dw[c] = t;
    } else if (db) {
      db[c - D] = t;
    }
  }
}

struct LnPlan {
  int nv, tpr, groups;
  long long blocks;
};

int slots(int D, int V) { return D % V ? D + V - 1 : D; }   // values from the first vector's start to the row's end, at most

// Threads per row for E values each: a multiple of 32, or a part of a warp;
// blocks of up to `most` threads, as many as are resident; TG, the number of
// groups, a multiple of the values per vector.
LnPlan plan_rows(long long rows, int D, int V, int E, int most, long long most_blocks) {
  LnPlan p;
  p.nv = E / V;
  const int need = (slots(D, V) + E - 1) / E;
  p.tpr = 8;
  while (p.tpr < 32 && p.tpr < need) p.tpr *= 2;
  if (need > 32) p.tpr = (need + 31) / 32 * 32;
  p.groups = std::max(1, std::min(most, 16 * 32) / p.tpr);
  int unit = D % V ? V : 1;   // blocks that make groups * blocks a multiple of V (for rows that need it)
  for (int g = p.groups; unit > 1 && g % 2 == 0; g /= 2) unit /= 2;
  p.blocks = std::min((rows + p.groups - 1) / p.groups, most_blocks);
  p.blocks = std::max(1LL, p.blocks / unit) * unit;   // down, to stay resident together
  return p;
}

// Values per thread: 8 or 16, part of a warp per row up to 128 columns and one
// warp up to 512; 24 for the rows that 512 threads do not hold with 16.
LnPlan fwd_plan(long long rows, int D, int V) {
  const int n = slots(D, V), E = n <= 256 ? 8 : n <= 4096 ? 16 : 24;
  return plan_rows(rows, D, V, E, E == 24 ? 512 : 256, static_cast<long long>(fwd_ctas(E, D % V == 0)) * num_sms());
}
LnPlan bwd_plan(long long rows, int D, int V) {
  const int n = slots(D, V), E = n <= 256 ? 8 : n <= 8192 ? 16 : 24;
  return plan_rows(rows, D, V, E, 512, num_sms());
}

template <typename T, typename F>
cudaError_t by_values(int nv, F f) {
  constexpr int k = 8 / Vec<T>::V;   // vectors of 8 values
  if (nv == k) return f(std::integral_constant<int, k>());
  if (nv == 2 * k) return f(std::integral_constant<int, 2 * k>());
  return f(std::integral_constant<int, 3 * k>());
}

template <typename T>
cudaError_t ln_fwd(long long rows, int D, const void* x, const float* w, const float* b, float eps, void* y, float* mean,
                   float* rstd, cudaStream_t st) {
  const T* xt = static_cast<const T*>(x);
  T* yt = static_cast<T*>(y);
  if (D > kMaxHeld) {
    const long long blocks = std::min<long long>(rows, 4LL * num_sms());
    ln_fwd_wide_kernel<T><<<static_cast<unsigned>(blocks), 512, 0, st>>>(rows, D, xt, w, b, eps, yt, mean, rstd);
    return cudaGetLastError();
  }
  const LnPlan p = fwd_plan(rows, D, Vec<T>::V);
  return by_values<T>(p.nv, [&](auto nv) {
    constexpr bool hold = nv() * Vec<T>::V <= 16;
    constexpr int n = nv();
    auto kern = D % Vec<T>::V == 0 ? ln_fwd_kernel<T, n, hold, true> : ln_fwd_kernel<T, n, hold, false>;
    const int threads = p.tpr * p.groups, sm = fwd_depth(n) * n * threads * 16;
    if (cudaError_t e = allow_smem(kern, sm); e != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(p.blocks), threads, sm, st>>>(rows, D, p.tpr, xt, w, b, eps, yt, mean, rstd);
    return cudaGetLastError();
  });
}

// Blocks of the backward pass, and so partial rows of dw and db.
long long bwd_blocks(long long rows, int D, bool bf16) {
  if (D > kMaxHeld) return std::min<long long>(rows, 2LL * num_sms());
  return bwd_plan(rows, D, bf16 ? 8 : 4).blocks;
}

template <typename T>
cudaError_t ln_bwd(long long rows, int D, const void* dy, const void* x, const float* w, const float* mean,
                   const float* rstd, void* dx, float* dw, float* db, float* part, cudaStream_t st) {
  const T *dt = static_cast<const T*>(dy), *xt = static_cast<const T*>(x);
  T* ot = static_cast<T*>(dx);
  const long long blocks = bwd_blocks(rows, D, sizeof(T) == 2);
  cudaError_t e;
  if (D > kMaxHeld) {
    if (part) {
      const dim3 grid(static_cast<unsigned>((D + 255) / 256), static_cast<unsigned>(blocks));
      ln_columns_wide_kernel<T><<<grid, 256, 0, st>>>(rows, D, dt, xt, mean, rstd, part);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    ln_bwd_wide_kernel<T><<<static_cast<unsigned>(std::min<long long>(rows, 4LL * num_sms())), 512, 0, st>>>(
        rows, D, dt, xt, w, mean, rstd, ot);
    e = cudaGetLastError();
  } else {
    const LnPlan p = bwd_plan(rows, D, Vec<T>::V);
    const int threads = p.tpr * p.groups;
    e = by_values<T>(p.nv, [&](auto nv) {
      constexpr bool hold = nv() * Vec<T>::V <= 16;
      constexpr int n = nv();
      auto kern = D % Vec<T>::V == 0 ? ln_bwd_kernel<T, n, hold, true> : ln_bwd_kernel<T, n, hold, false>;
      // (the groups' sums fit in the ring: 8 D bytes a group, D <= nv V tpr, against 32 nv bytes a thread and row of it)
      const int sm = bwd_depth(2 * n) * 2 * n * threads * 16;
      if (cudaError_t e2 = allow_smem(kern, sm); e2 != cudaSuccess) return e2;
      kern<<<static_cast<unsigned>(blocks), threads, sm, st>>>(rows, D, p.tpr, dt, xt, w, mean, rstd, ot, part);
      return cudaGetLastError();
    });
  }
  if (e != cudaSuccess || !part) return e;
  // (the wide form's last kernel does not write the partial rows: no overlap there)
  return launch_after(ln_reduce_kernel, (2 * D + 31) / 32, 1024, 0, st, D <= kMaxHeld, D, static_cast<int>(blocks), part, dw, db);
}

bool valid_norm(long long rows, int D, ia_dtype_t dt) {
  return rows > 0 && D > 0 && (dt == IA_F32 || dt == IA_BF16) && rows <= (1LL << 62) / D / 8;
}
constexpr int kMaxD = 1 << 24;

}  // namespace
}  // namespace ia

using namespace ia;

extern "C" {

ia_status_t ia_layer_norm_fwd(long long rows, int D, ia_dtype_t dtype, const void* x, const float* weight,
                              const float* bias, float eps, void* y, float* mean, float* rstd, void* stream) {
  if (!valid_norm(rows, D, dtype) || !x || !y || !(eps >= 0.f) || std::isinf(eps)) return IA_ERR_INVALID_ARG;
  const void* ptrs[] = {x, weight, bias, y, mean, rstd};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return IA_ERR_INVALID_ARG;
  if (D > kMaxD) return IA_ERR_UNSUPPORTED;
  if (inject_launch_failure()) return IA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  mark_launch_begin(st);
  const cudaError_t e = dtype == IA_BF16 ? ln_fwd<__nv_bfloat16>(rows, D, x, weight, bias, eps, y, mean, rstd, st)
                                         : ln_fwd<float>(rows, D, x, weight, bias, eps, y, mean, rstd, st);
  mark_launch_end(st);
  return map_cuda(e);
}

size_t ia_layer_norm_bwd_workspace_bytes(long long rows, int D, ia_dtype_t dtype) {
  if (!valid_norm(rows, D, dtype) || D > kMaxD) return 0;
  return 2 * sizeof(float) * static_cast<size_t>(D) * static_cast<size_t>(bwd_blocks(rows, D, dtype == IA_BF16));
}

ia_status_t ia_layer_norm_bwd(long long rows, int D, ia_dtype_t dtype, const void* dy, const void* x,
                              const float* weight, const float* mean, const float* rstd, void* dx, float* dweight,
                              float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_norm(rows, D, dtype) || !dy || !x || !mean || !rstd || !dx) return IA_ERR_INVALID_ARG;
  const void* ptrs[] = {dy, x, weight, mean, rstd, dx, dweight, dbias, workspace};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return IA_ERR_INVALID_ARG;
  if (D > kMaxD) return IA_ERR_UNSUPPORTED;
  const bool sums = dweight || dbias;
  if (sums && (!workspace || workspace_bytes < ia_layer_norm_bwd_workspace_bytes(rows, D, dtype)))
    return IA_ERR_WORKSPACE;
  if (inject_launch_failure()) return IA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* part = sums ? static_cast<float*>(workspace) : nullptr;
  mark_launch_begin(st);
  const cudaError_t e =
      dtype == IA_BF16 ? ln_bwd<__nv_bfloat16>(rows, D, dy, x, weight, mean, rstd, dx, dweight, dbias, part, st)
                       : ln_bwd<float>(rows, D, dy, x, weight, mean, rstd, dx, dweight, dbias, part, st);
  mark_launch_end(st);
  return map_cuda(e);
}

}  // extern "C"
