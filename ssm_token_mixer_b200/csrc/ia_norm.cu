// Layer norm over rows of D values, forward and backward.
//
//   mean = sum(x)/D,  var = sum((x - mean)^2)/D,  rstd = 1/sqrt(var + eps)
//   y  = (x - mean) rstd w + b
//   dx = rstd (g - mean(g) - xhat mean(g xhat)),  g = dy w,  xhat = (x - mean) rstd
//   dw = sum_rows dy xhat,  db = sum_rows dy
//
// Both directions touch every value once (2 and 3 row-sized streams), so HBM
// bounds them.  A row is held in registers by a group of threads (a warp up to
// 512 columns, else up to 512 threads), which makes the variance a second pass
// over registers instead of a difference of large sums.  The backward pass
// keeps a group's columns fixed while it walks rows, so dw and db accumulate
// in registers in fp32; the groups of a block add theirs in shared memory, the
// block writes one partial row, and a second kernel adds the blocks' rows in a
// fixed order: no atomics, equal bits from equal calls.  Rows wider than the
// registers hold (12288 columns) are read again from L2 instead.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "ia_device.cuh"
#include "ia_internal.h"
#include "ia_launch.h"

namespace ia {
namespace {

constexpr int kMaxHeld = 12288;   // widest row held in registers

// V consecutive values as fp32.  V = 4 (or 1 for rows that do not start on a
// 4-value boundary).
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float* f) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 2) f[0] = __bfloat162float(p[0]);
    else f[0] = p[0];
  } else if constexpr (sizeof(T) == 2) {
    static_assert(V == 4 || V == 8, "");
    uint32_t w[V / 2];
    if constexpr (V == 8) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x, w[1] = u.y;
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {   // a bf16 is the high half of an fp32
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 u = *reinterpret_cast<const float4*>(p + i);
      f[i] = u.x, f[i + 1] = u.y, f[i + 2] = u.z, f[i + 3] = u.w;
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float* f) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 2) p[0] = __float2bfloat16(f[0]);
    else p[0] = f[0];
  } else if constexpr (sizeof(T) == 2) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sums NV values over a group of tpr threads (a multiple of 32): shuffles, then
// one word per warp in shared memory.  `slot` alternates between two buffers so
// that one barrier per call is enough.
template <int NV>
__device__ __forceinline__ void group_sum(float (&x)[NV], int tpr, int group, int gt, float* buf, int slot) {
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = warp_sum(x[i]);
  if (tpr == 32) return;
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

// E values per thread in E / V vectors: vector j of thread t covers columns
// (j * tpr + t) * V ...
template <typename T, int E, int V>
__global__ void __launch_bounds__(512) ln_fwd_kernel(long long rows, int D, int tpr, const T* x,
                                                     const float* __restrict__ w, const float* __restrict__ b, float eps,
                                                     T* y, float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  __shared__ float buf[16 * 2 * 32];
  const int group = threadIdx.x / tpr, gt = threadIdx.x - group * tpr, groups = blockDim.x / tpr;
  const float inv = 1.f / static_cast<float>(D);
  int slot = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * groups + group; row < rows;
       row += static_cast<long long>(gridDim.x) * groups) {
    const T* xr = x + row * D;
    float v[E];
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < E / V; ++j) {
      const int c = (j * tpr + gt) * V;
      if (c < D) load_v<T, V>(xr + c, v + j * V);
      else
#pragma unroll
        for (int e = 0; e < V; ++e) v[j * V + e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s[0] += v[e];
    group_sum<1>(s, tpr, group, gt, buf, slot);
    slot ^= 1;
    const float mean = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < E / V; ++j)
      if ((j * tpr + gt) * V < D)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = v[j * V + e] - mean;
          s[0] = fmaf(d, d, s[0]);
        }
    group_sum<1>(s, tpr, group, gt, buf, slot);
    slot ^= 1;
    const float rstd = 1.f / sqrtf(s[0] * inv + eps);
    T* yr = y + row * D;
#pragma unroll
    for (int j = 0; j < E / V; ++j) {
      const int c = (j * tpr + gt) * V;
      if (c < D) {
        float wv[V], bv[V], r[V];
#pragma unroll
        for (int e = 0; e < V; ++e) wv[e] = 1.f, bv[e] = 0.f;
        if (w) load_v<float, V>(w + c, wv);
        if (b) load_v<float, V>(b + c, bv);
#pragma unroll
        for (int e = 0; e < V; ++e) r[e] = fmaf((v[j * V + e] - mean) * rstd, wv[e], bv[e]);
        store_v<T, V>(yr + c, r);
      }
    }
    if (gt == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
  }
}

// part: [gridDim.x][2][D] partial sums of dw and db (null: neither is wanted)
template <typename T, int E, int V>
__global__ void __launch_bounds__(512) ln_bwd_kernel(long long rows, int D, int tpr, const T* dy, const T* x,
                                                     const float* __restrict__ w, const float* __restrict__ mean_in,
                                                     const float* __restrict__ rstd_in, T* dx, float* __restrict__ part) {
  __shared__ float buf[16 * 2 * 32 * 2];
  extern __shared__ float acc_sm[];   // [2][D] when the block has several groups
  const int group = threadIdx.x / tpr, gt = threadIdx.x - group * tpr, groups = blockDim.x / tpr;
  const float inv = 1.f / static_cast<float>(D);
  griddep_launch_dependents();
  float aw[E], ab[E];
#pragma unroll
  for (int e = 0; e < E; ++e) aw[e] = ab[e] = 0.f;
  int slot = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * groups + group; row < rows;
       row += static_cast<long long>(gridDim.x) * groups) {
    const T *xr = x + row * D, *dr = dy + row * D;
    float hat[E], g[E];
#pragma unroll
    for (int j = 0; j < E / V; ++j) {
      const int c = (j * tpr + gt) * V;
      if (c < D) {
        load_v<T, V>(xr + c, hat + j * V);
        load_v<T, V>(dr + c, g + j * V);
      }
    }
    const float mean = mean_in[row], rstd = rstd_in[row];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < E / V; ++j) {
      const int c = (j * tpr + gt) * V;
      if (c < D) {
        float wv[V];
#pragma unroll
        for (int e = 0; e < V; ++e) wv[e] = 1.f;
        if (w) load_v<float, V>(w + c, wv);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int i = j * V + e;
          hat[i] = (hat[i] - mean) * rstd;
          aw[i] = fmaf(g[i], hat[i], aw[i]);
          ab[i] += g[i];
          g[i] *= wv[e];
          s[0] += g[i];
          s[1] = fmaf(g[i], hat[i], s[1]);
        }
      }
    }
    group_sum<2>(s, tpr, group, gt, buf, slot);
    slot ^= 1;
    const float c1 = s[0] * inv, c2 = s[1] * inv;
    T* xo = dx + row * D;
#pragma unroll
    for (int j = 0; j < E / V; ++j) {
      const int c = (j * tpr + gt) * V;
      if (c < D) {
        float r[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int i = j * V + e;
          r[e] = rstd * (g[i] - c1 - hat[i] * c2);
        }
        store_v<T, V>(xo + c, r);
      }
    }
  }
  if (!part) return;
  float* out = part + static_cast<long long>(blockIdx.x) * 2 * D;
  if (groups == 1) {
#pragma unroll
    for (int j = 0; j < E / V; ++j) {
      const int c = (j * tpr + gt) * V;
      if (c < D) {
        store_v<float, V>(out + c, aw + j * V);
        store_v<float, V>(out + D + c, ab + j * V);
      }
    }
    return;
  }
  for (int gr = 0; gr < groups; ++gr) {   // one group after the other: a fixed order
    if (gr == group) {
#pragma unroll
      for (int j = 0; j < E / V; ++j) {
        const int c = (j * tpr + gt) * V;
        if (c < D)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            acc_sm[c + e] = (gr ? acc_sm[c + e] : 0.f) + aw[j * V + e];
            acc_sm[D + c + e] = (gr ? acc_sm[D + c + e] : 0.f) + ab[j * V + e];
          }
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < 2 * D; c += blockDim.x) out[c] = acc_sm[c];
}

// ---- rows too wide for registers: one block per row, values read again
template <typename T>
__device__ __forceinline__ float ld1(const T* p, long long i) {
  float f;
  load_v<T, 1>(p + i, &f);
  return f;
}

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
      store_v<T, 1>(y + row * D + c, &r);
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
      store_v<T, 1>(dx + row * D + c, &r);
    }
  }
}

// dw[c], db[c] = sums of the partial rows: 32 columns x 8 row lanes per block,
// the lanes' sums added in order.
__global__ void __launch_bounds__(256) ln_reduce_kernel(int D, int nparts, const float* __restrict__ part,
                                                        float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float sm[8][33];
  griddep_wait();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;   // columns of [2 D]
  float t = 0.f;
  if (c < 2 * D)
    for (int i = r; i < nparts; i += 8) t += part[static_cast<long long>(i) * 2 * D + c];
  sm[r][threadIdx.x & 31] = t;
  __syncthreads();
  if (r == 0 && c < 2 * D) {
#pragma unroll
    for (int i = 1; i < 8; ++i) t += sm[i][threadIdx.x & 31];
    if (c < D) {
      if (dw) dw[c] = t;
    } else if (db) {
      db[c - D] = t;
    }
  }
}

struct LnPlan {
  int E, V, tpr, groups;
};

// Vectors of 4 (8 for bf16) values where the row length keeps every row on a
// 16-byte boundary, else single values; a warp per row up to 512 columns, then
// as many threads as 8, 16 or 24 values each need.
LnPlan ln_plan(int D, bool bf16) {
  LnPlan p;
  const int wide = bf16 ? 8 : 4;
  p.V = D % wide == 0 ? wide : 1;
  p.E = D <= 4096 ? 8 : D <= 8192 ? 16 : 24;
  if (D <= 512) {
    p.tpr = 32;
    p.E = D <= 256 ? 8 : 16;
  } else {
    p.tpr = ((D + p.E - 1) / p.E + 31) / 32 * 32;
  }
  p.groups = p.tpr == 32 ? 8 : std::max(1, 512 / p.tpr);
  return p;
}

template <typename T, int V, typename F>
cudaError_t by_e(int E, F f) {
  switch (E) {
    case 8: return f(std::integral_constant<int, 8>(), std::integral_constant<int, V>());
    case 16: return f(std::integral_constant<int, 16>(), std::integral_constant<int, V>());
    default: return f(std::integral_constant<int, 24>(), std::integral_constant<int, V>());
  }
}
template <typename T, typename F>
cudaError_t by_plan(const LnPlan& p, F f) {
  if (p.V == 1) return by_e<T, 1>(p.E, f);
  if constexpr (sizeof(T) == 2) return by_e<T, 8>(p.E, f);
  else return by_e<T, 4>(p.E, f);
}

template <typename T>
cudaError_t ln_fwd(long long rows, int D, const void* x, const float* w, const float* b, float eps, void* y, float* mean,
                   float* rstd, cudaStream_t st) {
  const T* xt = static_cast<const T*>(x);
  T* yt = static_cast<T*>(y);
  const long long sms = num_sms();
  if (D > kMaxHeld) {
    ln_fwd_wide_kernel<T><<<static_cast<unsigned>(std::min(rows, 4 * sms)), 512, 0, st>>>(rows, D, xt, w, b, eps, yt, mean, rstd);
    return cudaGetLastError();
  }
  const LnPlan p = ln_plan(D, sizeof(T) == 2);
  const int threads = p.tpr * p.groups;
  const long long blocks = std::min((rows + p.groups - 1) / p.groups, sms * (2048 / threads));
  return by_plan<T>(p, [&](auto e, auto v) {
    ln_fwd_kernel<T, e(), v()><<<static_cast<unsigned>(blocks), threads, 0, st>>>(rows, D, p.tpr, xt, w, b, eps, yt, mean, rstd);
    return cudaGetLastError();
  });
}

// Blocks of the backward pass, and so partial rows of dw and db: two per SM.
long long bwd_blocks(long long rows, int D, bool bf16) {
  const long long most = 2LL * num_sms();
  if (D > kMaxHeld) return std::min(rows, most);
  const LnPlan p = ln_plan(D, bf16);
  return std::min((rows + p.groups - 1) / p.groups, most);
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
    const LnPlan p = ln_plan(D, sizeof(T) == 2);
    const int threads = p.tpr * p.groups;
    const size_t sm = part && p.groups > 1 ? 2 * sizeof(float) * D : 0;
    e = by_plan<T>(p, [&](auto ee, auto v) {
      ln_bwd_kernel<T, ee(), v()><<<static_cast<unsigned>(blocks), threads, sm, st>>>(rows, D, p.tpr, dt, xt, w, mean,
                                                                                      rstd, ot, part);
      return cudaGetLastError();
    });
  }
  if (e != cudaSuccess || !part) return e;
  // (the wide form's last kernel does not write the partial rows: no overlap there)
  return launch_after(ln_reduce_kernel, (2 * D + 31) / 32, 256, 0, st, D <= kMaxHeld, D, static_cast<int>(blocks), part, dw, db);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
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
