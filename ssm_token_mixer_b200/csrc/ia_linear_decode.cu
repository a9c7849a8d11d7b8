// One token of the linear-attention mixer:
//   S' = lambda S + k v^T,  o = scale q^T S'
// with S [d_k][d_v] fp32 read and written once: 8 d_k d_v bytes per (b,h), so
// HBM bounds it (latency at small batches).
//
// Where lambda > 1/2, lambda S is formed as S + (lambda - 1) S with expm1: lambda
// rounded to fp32 is off by up to 2^-25, every step the same way, which 4096 steps
// of a lambda near 1 make 1.2e-4 of a state.  Below 1/2 that sum would cancel, and
// a product is the accurate form.  The two have loops of their own; a choice per
// entry took 4 to 10 % more time.
//
// A CTA takes CW columns of one (b,h) and all its rows: thread (r, c) holds
// VEC columns of the rows r, r + R, ..., four or eight loaded before the first
// is used, so that an SM has 128 KB in flight; the sum over rows is a sum over
// r at the end, in shared memory and in a fixed order.  With few (b,h) the
// slices are narrower (32 columns, one 128-byte line per row), which puts the
// step on four times as many SMs without any exchange between them.
//
// With parents, a sequence reads its parent's state and writes its own: the
// reordering of a beam search rides on a read and a write that happen anyway.
//
// Measured: 64 sequences of 16 heads of 128 x 128 through parents into another
// buffer 18.2 us (114 MB: 95 % of the copy rate; 24.0 with 16 rows in flight, two
// CTAs per SM and plain stores, 20.4 with stores that L2 need not keep), in
// place 14.1 us (part of the 67 MB of states stays in L2); 256 of 64 x 64 22.4 us
// through parents of 8 beams (111 MB; 49.5 before); one sequence 2.6 us, the
// launch and one read's latency.
#include <algorithm>
#include <type_traits>

#include "ia_device.cuh"
#include "ia_internal.h"
#include "ia_linear.h"

namespace ia {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float ld(const T* p, long long i) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(p[i]);
  else return p[i];
}
template <typename T>
__device__ __forceinline__ void st(T* p, long long i, float x) {
  if constexpr (sizeof(T) == 2) p[i] = __float2bfloat16(x);
  else p[i] = x;
}

template <int VEC>
struct Vec {
  float v[VEC];
};
template <int VEC>
__device__ __forceinline__ Vec<VEC> load_vec(const float* p) {
  Vec<VEC> r;
  if constexpr (VEC == 4) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    r.v[0] = x.x, r.v[1] = x.y, r.v[2] = x.z, r.v[3] = x.w;
  } else {
    r.v[0] = *p;
  }
  return r;
}
// apart: the state goes to another buffer, whose lines L2 need not keep while
// parents are still to be read.
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const Vec<VEC>& r, bool apart) {
  if constexpr (VEC == 4) {
    const float4 x = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
    if (apart) __stcs(reinterpret_cast<float4*>(p), x);
    else *reinterpret_cast<float4*>(p) = x;
  } else {
    *p = r.v[0];
  }
}

// tc: threads across the CW columns; R = kThreads / tc row groups
// kDepth: rows of a thread in flight, for five or four CTAs per SM.
template <typename T, int VEC, int kDepth>
__global__ void __launch_bounds__(kThreads, kDepth == 4 ? 5 : 4) lin_decode_kernel(
    int H, int dk, int dv, int cw, int tc, const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
    const float* __restrict__ log_decay, float scale, const float* sin, const int* __restrict__ parents, int beams,
    float* sout, T* __restrict__ o, int* err) {   // sout may be sin: every entry is read and written by one thread
  __shared__ float sk[256], sq[256];
  __shared__ float part[kThreads * VEC];
  const int tid = threadIdx.x;
  const long long bh = blockIdx.x;
  const int h = static_cast<int>(bh % H);
  const int col = static_cast<int>(blockIdx.y) * cw + (tid % tc) * VEC;
  const int r0 = tid / tc, R = kThreads / tc;
  const bool apart = sout != sin;
  const bool active = r0 < R && (tid % tc) * VEC < cw && col < dv;

  long long src = bh;
  bool zero = false;
  if (parents) {
    const long long b = bh / H;
    const int p = parents[b];
    zero = p < 0 || p >= beams;
    src = zero ? bh : (b / beams * beams + p) * H + h;
  }
  const float graw = log_decay[h];
  if (!(graw <= 0.f) && tid == 0) atomicOr(err, kErrParamRange);
  const float gl = lin_log_decay(graw);

  const float* in = sin + src * dk * dv + col;
  float* out = sout + bh * dk * dv + col;
  Vec<VEC> s[kDepth];
  auto fetch = [&](int base) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int i = base + d * R;
      if (active && !zero && i < dk) s[d] = load_vec<VEC>(in + static_cast<long long>(i) * dv);
      else
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[d].v[e] = 0.f;
    }
  };
  fetch(r0);
  const bool slow = gl > kLinSlow;
  const float a = lin_decay(gl);
  if (tid < dk) {
    sk[tid] = ld(k, bh * dk + tid);
    sq[tid] = ld(q, bh * dk + tid);
  }
  Vec<VEC> vv, acc;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    vv.v[e] = active ? ld(v, bh * dv + col + e) : 0.f;
    acc.v[e] = 0.f;
  }
  __syncthreads();
  auto rows = [&](auto near_one) {
    for (int base = r0; base < dk; base += kDepth * R) {
      if (base != r0) fetch(base);
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int i = base + d * R;
        if (!active || i >= dk) continue;
        const float ki = sk[i], qi = sq[i];
        Vec<VEC> n;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float x = s[d].v[e];
          n.v[e] = near_one() ? fmaf(ki, vv.v[e], fmaf(a, x, x)) : fmaf(a, x, ki * vv.v[e]);
          acc.v[e] = fmaf(qi, n.v[e], acc.v[e]);
        }
        store_vec<VEC>(out + static_cast<long long>(i) * dv, n, apart);
      }
    }
  };
  if (slow) rows(std::true_type());
  else rows(std::false_type());
#pragma unroll
  for (int e = 0; e < VEC; ++e) part[tid * VEC + e] = acc.v[e];
  __syncthreads();
  // part is [r][tc * VEC]; one thread per column adds its R partial sums
  const int width = tc * VEC;
  if (tid < cw && blockIdx.y * cw + tid < dv) {
    float t = 0.f;
    for (int r = 0; r < R; ++r) t += part[r * width + tid];
    st(o, bh * dv + static_cast<int>(blockIdx.y) * cw + tid, scale * t);
  }
}

template <typename T>
cudaError_t launch(const ia_linear_shape_t& s, const void* q, const void* k, const void* v, const float* log_decay,
                   float scale, const float* sin, const int* parents, int beams, float* sout, void* o, int* err,
                   cudaStream_t st) {
  const long long bh = static_cast<long long>(s.B) * s.H;
  const bool vec = s.d_v % 4 == 0;
  const int lanes = vec ? 4 : 1;
  // whole rows (up to 128 columns) once they give every SM a CTA, else slices of 32 columns
  const int want = bh >= num_sms() ? 128 : 32;
  const int cw = std::min(want, (s.d_v + lanes - 1) / lanes * lanes);
  const int tc = (cw + lanes - 1) / lanes;
  const dim3 grid(static_cast<unsigned>(bh), static_cast<unsigned>((s.d_v + cw - 1) / cw));
  mark_launch_begin(st);
  auto go = [&](auto kern) {
    kern<<<grid, kThreads, 0, st>>>(s.H, s.d_k, s.d_v, cw, tc, static_cast<const T*>(q), static_cast<const T*>(k),
                                    static_cast<const T*>(v), log_decay, scale, sin, parents, beams, sout,
                                    static_cast<T*>(o), err);
  };
  // Rows of a thread: with few, a kernel of fewer registers and one more CTA per
  // SM (256 sequences of 16 heads of 64 x 64: 18.0 us, and 23 with eight rows).
  const int rows = (s.d_k + kThreads / tc - 1) / (kThreads / tc);
  if (vec) {
    if (rows <= 4) go(lin_decode_kernel<T, 4, 4>);
    else go(lin_decode_kernel<T, 4, 8>);
  } else {
    go(lin_decode_kernel<T, 1, 8>);
  }
  mark_launch_end(st);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_decode(const ia_linear_shape_t& s, const void* q, const void* k, const void* v,
                              const float* log_decay, float scale, const float* state_in, const int* parents,
                              int beams, float* state_out, void* o, int* err, cudaStream_t st) {
  return s.in_dtype == IA_BF16
             ? launch<__nv_bfloat16>(s, q, k, v, log_decay, scale, state_in, parents, beams, state_out, o, err, st)
             : launch<float>(s, q, k, v, log_decay, scale, state_in, parents, beams, state_out, o, err, st);
}

}  // namespace ia
