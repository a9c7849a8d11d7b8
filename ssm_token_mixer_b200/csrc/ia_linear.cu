// Linear attention with one decay per head: the C-ABI entry points, the plan
// of the segments, the CUDA-core kernel of the chunked form and the
// composition of the segments' states.
//
// Chunk algebra (C tokens, local positions p = 0 .. C-1 counted in the
// direction of the problem, S the state entering the chunk):
//   A_ts  = x_t . y_s                       C x C
//   P_ts  = lambda^(p_t - p_s) A_ts for p_s <= p_t, else 0
//   out_t = scale (sum_s P_ts z_s + lambda^(p_t + 1) x_t S)
//   S    <- lambda^L S + sum_s lambda^(L-1-p_s) y_s z_s^T      (L tokens in it)
// Every power of lambda that appears has an exponent >= 0, so nothing
// overflows for any decay.  lambda^L S is formed as S + (lambda^L - 1) S with
// expm1 where lambda^L > 1/2, whose relative error does not add up over hundreds
// of chunks when lambda is close to 1, and as a product below, where that sum
// would cancel (and leave 0 for a lambda^L under 2^-25).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "ia_device.cuh"
#include "ia_internal.h"
#include "ia_launch.h"
#include "ia_linear.h"

namespace ia {
namespace {

constexpr int kThreads = 128;
constexpr int C = 32;   // tokens per chunk: fewer operations per token than 64, and more CTAs per SM

// Element i of p as fp32 to shared memory, 0 outside: an asynchronous copy for
// fp32 (complete after cp.async.wait_all of the same thread).
template <bool BF16>
__device__ __forceinline__ void fetch(float* dst, const void* p, long long i, bool in) {
  if constexpr (BF16) {
    *dst = in ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : 0.f;
  } else {
    const float* src = static_cast<const float*>(p) + (in ? i : 0);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 4 : 0) : "memory");
  }
}

// Four elements, all in or all out.
__device__ __forceinline__ void fetch4(float* dst, const void* p, long long i, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(static_cast<const float*>(p) + (in ? i : 0)),
               "r"(in ? 16 : 0)
               : "memory");
}

// Row stride in floats of a shared tile of `w` columns: a multiple of 4 whose
// quarter is odd, so that float4 reads of consecutive rows by consecutive
// lanes fall into different banks.
__host__ __device__ inline int lin_pad(int w) { return ((w + 3) / 4 | 1) * 4; }

struct SimtSmem {
  int X, Y, S, Z, A, total;   // float offsets
};
__host__ __device__ inline SimtSmem simt_smem(int dx) {
  SimtSmem s;
  const int dxs = lin_pad(dx);
  s.X = 0;
  s.Y = s.X + C * dxs;
  s.S = s.Y + C * dxs;
  s.Z = s.S + ((dx + 3) / 4 * 4) * lin_pad(kLinZB);
  s.A = s.Z + C * lin_pad(kLinZB);
  s.total = s.A + C * lin_pad(C);
  return s;
}

// The CUDA-core kernel: fp32 throughout, any widths up to 256, one CTA per
// (b,h, block of 64 z columns, segment), R x 4 outputs per thread and step.
// With R = 4 it reads 16 bytes of shared memory per 8 multiply-adds of a lane,
// about what an SM can supply, so it is bound by the FP32 pipe and shared
// memory together.  Small CTAs (four per SM at widths up to 64) let one compute
// while another loads or waits at a barrier.  Measured: fp32 prefill of B8 H16
// N2048 d64 400 us (4.0 G multiply-adds, 28 % of the pipe's rate), of B2 H4 N300
// 48 x 80 in 10 segments 21.1 us, of one chunk 9.5 us.  bf16 of the widths that the
// tensor cores do not take is no faster: prefill of B4 H16 N2048 d96 609 us, training
// 1760 (d128 on the tensor cores 48 and 157).
template <bool BF16, bool STATE_ONLY, int T>
__global__ void __launch_bounds__(T, 512 / T) lin_simt_kernel(const __grid_constant__ LinArgs a) {
  extern __shared__ __align__(16) float sm[];
  __shared__ int bad;          // least position in the chunk whose z holds a NaN or an infinity, C if none
  __shared__ float pw[C + 1];  // lambda^n
  constexpr int R = T == 128 ? 4 : 2;   // rows per thread and step
  const int tid = threadIdx.x;
  const int nseg = STATE_ONLY ? a.nseg - 1 : a.nseg;
  const long long stream = blockIdx.x / nseg;
  const int seg = static_cast<int>(blockIdx.x - stream * nseg);
  const long long bh = stream / a.first[a.nprob];
  const int block = static_cast<int>(stream - bh * a.first[a.nprob]);
  int pi = 0;
  while (pi + 1 < a.nprob && block >= a.first[pi + 1]) ++pi;
  const LinProblem& pr = a.p[pi];
  const int dx = pr.dx, dz = pr.dz;
  const int z0 = (block - a.first[pi]) * kLinZB;
  const int zw = min(kLinZB, dz - z0);
  const int h = static_cast<int>(bh % a.H);

  const SimtSmem o = simt_smem(dx);
  const int dxs = lin_pad(dx), zs = lin_pad(kLinZB), as = lin_pad(C);
  const int dx4 = (dx + 3) / 4 * 4, zw4 = (zw + 3) / 4 * 4;
  const bool wide = !BF16 && dx % 4 == 0 && dz % 4 == 0;   // rows of whole 16-byte pieces
  float *X = sm + o.X, *Y = sm + o.Y, *S = sm + o.S, *Z = sm + o.Z, *A = sm + o.A;

  const float graw = a.log_decay[h];
  if (!(graw <= 0.f) && tid == 0) atomicOr(a.err, kErrParamRange);
  const float g = lin_log_decay(graw);
  if (tid <= C) pw[tid] = expf(g * tid);
  const int warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();
  griddep_wait();   // the segments' states, when a pass before this one built them

  // entering state
  const float* s0 = seg == 0 ? pr.state_in : STATE_ONLY ? nullptr : pr.seg;
  const long long soff = seg == 0 ? bh * dx * static_cast<long long>(dz)
                                  : (bh * (a.nseg - 1) + seg - 1) * dx * static_cast<long long>(dz);
  for (int e = tid; e < dx4 * zw4; e += T) {
    const int i = e / zw4, j = e - i * zw4;
    S[i * zs + j] = (s0 && i < dx && j < zw) ? s0[soff + static_cast<long long>(i) * dz + z0 + j] : 0.f;
  }

  const int c_first = seg * a.cps, c_last = min(a.nch, c_first + a.cps);
  for (int c = c_first; c < c_last; ++c) {
    const int chunk = pr.reverse ? a.nch - 1 - c : c;
    const int t0 = chunk * C;
    const int L = min(C, a.N - t0);
    const int Lw = pr.reverse ? C : L;
    __syncthreads();
    if (tid == 0) bad = C;
    __syncthreads();
    const long long row0 = bh * a.N + t0;
    // A warp per row, its lanes along the columns; every copy is in flight
    // before the first is waited for (a chunk cost six DRAM round trips with
    // plain loads, half of its 10 us).
    auto check = [&](int t, int j) {   // (each thread checks what it copied)
      if (!isfinite(Z[t * zs + j])) {   // 0 * z of the masked half would reach the tokens before it
        atomicMin(&bad, pr.reverse ? C - 1 - t : t);
        Z[t * zs + j] = 0.f;
      }
    };
    if (wide) {
      const int nx = dx / 4, nz = zw / 4;
#pragma unroll 4
      for (int e = tid; e < C * nx; e += T) {
        const int t = e / nx, i = (e - t * nx) * 4;
        if (!STATE_ONLY) fetch4(X + t * dxs + i, pr.x, (row0 + t) * dx + i, t < L);
        fetch4(Y + t * dxs + i, pr.y, (row0 + t) * dx + i, t < L);
      }
#pragma unroll 4
      for (int e = tid; e < C * nz; e += T) {
        const int t = e / nz, j = (e - t * nz) * 4;
        fetch4(Z + t * zs + j, pr.z, (row0 + t) * dz + z0 + j, t < L);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      for (int e = tid; e < C * nz; e += T) {
        const int t = e / nz, j = (e - t * nz) * 4;
        for (int d = 0; d < 4; ++d) check(t, j + d);
      }
    } else {
      for (int i = lane; i < dx4; i += 32) {
#pragma unroll 8
        for (int t = warp; t < C; t += T / 32) {
          const bool in = t < L && i < dx;
          if (!STATE_ONLY) fetch<BF16>(X + t * dxs + i, pr.x, (row0 + t) * dx + i, in);
          fetch<BF16>(Y + t * dxs + i, pr.y, (row0 + t) * dx + i, in);
        }
      }
      for (int j = lane; j < zw4; j += 32) {
#pragma unroll 8
        for (int t = warp; t < C; t += T / 32)
          fetch<BF16>(Z + t * zs + j, pr.z, (row0 + t) * dz + z0 + j, t < L && j < zw);
      }
      if (!BF16) asm volatile("cp.async.wait_all;" ::: "memory");
      for (int j = lane; j < zw4; j += 32)
        for (int t = warp; t < C; t += T / 32) check(t, j);
    }
    __syncthreads();
    if (!STATE_ONLY) {
      // A = X Y^T, masked and decayed; thread rows t, t + C/4, .. so that the
      // lanes of a warp read neighbouring rows of Y
      constexpr int Q = C / 4, QR = C / R;
      for (int tile = tid; tile < QR * Q; tile += T) {
        const int tr = tile / Q, tc = tile % Q;
        float acc[R][4] = {};
#pragma unroll 2
        for (int i = 0; i < dx4; i += 4) {
          float4 xv[R], yv[4];
#pragma unroll
          for (int r = 0; r < R; ++r) xv[r] = *reinterpret_cast<const float4*>(X + (tr + r * QR) * dxs + i);
#pragma unroll
          for (int r = 0; r < 4; ++r) yv[r] = *reinterpret_cast<const float4*>(Y + (tc + r * Q) * dxs + i);
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              acc[r][s] = fmaf(xv[r].x, yv[s].x, acc[r][s]);
              acc[r][s] = fmaf(xv[r].y, yv[s].y, acc[r][s]);
              acc[r][s] = fmaf(xv[r].z, yv[s].z, acc[r][s]);
              acc[r][s] = fmaf(xv[r].w, yv[s].w, acc[r][s]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const int t = tr + r * QR, u = tc + s * Q;
            const int far = pr.reverse ? u - t : t - u;
            A[t * as + u] = far < 0 ? 0.f : acc[r][s] * pw[far];
          }
      }
      __syncthreads();
      // out = scale (A Z + lambda^(p+1) X S)
      const int jt = zw4 / 4;
      for (int tile = tid; tile < QR * jt; tile += T) {
        const int tr = tile / jt, j0 = (tile - tr * jt) * 4;
        float acc[R][4] = {}, acc2[R][4] = {};
        auto gemm = [&](const float* lhs, int ls, const float* rhs, int K, float (&c4)[R][4]) {
#pragma unroll 2
          for (int i = 0; i < K; i += 4) {
            float4 xv[R], sv[4];
#pragma unroll
            for (int r = 0; r < R; ++r) xv[r] = *reinterpret_cast<const float4*>(lhs + (tr + r * QR) * ls + i);
#pragma unroll
            for (int r = 0; r < 4; ++r) sv[r] = *reinterpret_cast<const float4*>(rhs + (i + r) * zs + j0);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const float xs[4] = {xv[r].x, xv[r].y, xv[r].z, xv[r].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                c4[r][0] = fmaf(xs[k], sv[k].x, c4[r][0]);
                c4[r][1] = fmaf(xs[k], sv[k].y, c4[r][1]);
                c4[r][2] = fmaf(xs[k], sv[k].z, c4[r][2]);
                c4[r][3] = fmaf(xs[k], sv[k].w, c4[r][3]);
              }
            }
          }
        };
        gemm(X, dxs, S, dx4, acc2);
        gemm(A, as, Z, C, acc);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int t = tr + r * QR;
          if (t >= L) continue;
          const float hd = pw[(pr.reverse ? C - 1 - t : t) + 1];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j0 + j >= zw) continue;
            float val = a.scale * fmaf(hd, acc2[r][j], acc[r][j]);
            if ((pr.reverse ? C - 1 - t : t) >= bad) val = __int_as_float(0x7fc00000);
            const long long at = (row0 + t) * dz + z0 + j0 + j;
            if (BF16) static_cast<__nv_bfloat16*>(pr.out)[at] = __float2bfloat16(val);
            else static_cast<float*>(pr.out)[at] = val;
          }
        }
      }
      __syncthreads();
    }
    // S <- lambda^L S + sum_s (lambda^(L-1-p_s) y_s) z_s^T
    for (int t = warp; t < C; t += T / 32) {
      const float w = t < L ? pw[Lw - 1 - (pr.reverse ? C - 1 - t : t)] : 0.f;
      for (int i = lane; i < dx4; i += 32) Y[t * dxs + i] *= w;
    }
    __syncthreads();
    const bool slow = g * Lw > kLinSlow;
    const float dec = bad < C ? __int_as_float(0x7fc00000) : lin_decay(g * Lw);
    const int jt = zw4 / 4;
    for (int tile = tid; tile < (dx4 / 4) * jt; tile += T) {
      const int i0 = (tile / jt) * 4, j0 = (tile % jt) * 4;
      float acc[4][4] = {};
#pragma unroll 8
      for (int s = 0; s < C; ++s) {
        const float4 y = *reinterpret_cast<const float4*>(Y + s * dxs + i0);
        const float4 z = *reinterpret_cast<const float4*>(Z + s * zs + j0);
        const float ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[r][0] = fmaf(ys[r], z.x, acc[r][0]);
          acc[r][1] = fmaf(ys[r], z.y, acc[r][1]);
          acc[r][2] = fmaf(ys[r], z.z, acc[r][2]);
          acc[r][3] = fmaf(ys[r], z.w, acc[r][3]);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float4* sp = reinterpret_cast<float4*>(S + (i0 + r) * zs + j0);
        float4 s = *sp;
        s.x = fmaf(dec, s.x, slow ? s.x : 0.f) + acc[r][0];
        s.y = fmaf(dec, s.y, slow ? s.y : 0.f) + acc[r][1];
        s.z = fmaf(dec, s.z, slow ? s.z : 0.f) + acc[r][2];
        s.w = fmaf(dec, s.w, slow ? s.w : 0.f) + acc[r][3];
        *sp = s;
      }
    }
  }
  __syncthreads();
  float* dst = nullptr;
  long long doff = 0;
  if (STATE_ONLY) {
    dst = pr.seg;
    doff = (bh * (a.nseg - 1) + seg) * dx * static_cast<long long>(dz);
  } else if (pr.state_out && seg == a.nseg - 1) {
    dst = pr.state_out;
    doff = bh * dx * static_cast<long long>(dz);
  }
  if (dst)
    for (int e = tid; e < dx * zw; e += T) {
      const int i = e / zw, j = e - i * zw;
      dst[doff + static_cast<long long>(i) * dz + z0 + j] = S[i * zs + j];
    }
}

// One thread per state entry walks the segments: the running state entering
// segment s + 1 is lambda^(tokens of segment s) times the one entering s plus
// what segment s built from zero (segment 0 already started from state_in).
// Every segment but a direction's first holds only whole chunks, and the
// first one's own length does not matter as nothing enters it.
__global__ void __launch_bounds__(kThreads) lin_carry_kernel(const __grid_constant__ LinArgs a, int chunk) {
  griddep_launch_dependents();
  griddep_wait();
  const LinProblem& pr = a.p[blockIdx.z];
  const long long per = static_cast<long long>(pr.dx) * pr.dz;
  const long long e = static_cast<long long>(blockIdx.y) * kThreads + threadIdx.x;
  if (e >= per) return;
  const long long bh = blockIdx.x;
  const double far = static_cast<double>(lin_log_decay(a.log_decay[bh % a.H])) * chunk * a.cps;
  const bool slow = far > kLinSlow;
  const float decf = static_cast<float>(slow ? expm1(far) : exp(far));
  float* s = pr.seg + bh * (a.nseg - 1) * per + e;
  float run = s[0];
  constexpr int kBatch = 8;   // loads in flight
  for (int i = 1; i < a.nseg - 1; i += kBatch) {
    float v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) v[j] = i + j < a.nseg - 1 ? s[(i + j) * per] : 0.f;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (i + j < a.nseg - 1) {
        run = fmaf(decf, run, slow ? run : 0.f) + v[j];
        s[(i + j) * per] = run;
      }
  }
}

template <bool BF16>
cudaError_t simt_launch(const LinArgs& a, int max_dx, bool state_only, cudaStream_t st) {
  const size_t bytes = sizeof(float) * simt_smem(max_dx).total;
  const long long grid = static_cast<long long>(a.BH) * a.first[a.nprob] * (state_only ? a.nseg - 1 : a.nseg);
  if (grid > (1LL << 31) - 1) return cudaErrorInvalidConfiguration;
  // Where SMs hold one or two CTAs, for want of CTAs or of shared memory, 256
  // threads of two rows a step shorten a chunk (B2 H4 N300 48 x 80: 24.3 us with
  // 128, 21.4 with 256; B4 H16 N2048 d128 771 and 713); where four of 128 threads
  // fit and there are enough, those read less of shared memory per product (B8
  // H16 N2048 d64 396 us, and 478 with 256).
  auto go = [&](auto kern, int threads) {
    if (cudaError_t e = allow_smem(kern, bytes); e != cudaSuccess) return e;
    return launch_after(kern, static_cast<unsigned>(grid), threads, bytes, st, a.nseg > 1 && !state_only, a);
  };
  if (grid <= 2LL * num_sms() || bytes > 56 * 1024)
    return state_only ? go(lin_simt_kernel<BF16, true, 256>, 256) : go(lin_simt_kernel<BF16, false, 256>, 256);
  return state_only ? go(lin_simt_kernel<BF16, true, 128>, 128) : go(lin_simt_kernel<BF16, false, 128>, 128);
}

}  // namespace

cudaError_t launch_lin_simt(const LinArgs& a, bool bf16, bool state_only, cudaStream_t st) {
  int dx = 0;
  for (int i = 0; i < a.nprob; ++i) dx = std::max(dx, a.p[i].dx);
  return bf16 ? simt_launch<true>(a, dx, state_only, st) : simt_launch<false>(a, dx, state_only, st);
}

cudaError_t launch_lin_carry(const LinArgs& a, int chunk, cudaStream_t st) {
  long long per = 0;
  for (int i = 0; i < a.nprob; ++i) per = std::max(per, static_cast<long long>(a.p[i].dx) * a.p[i].dz);
  const dim3 grid(static_cast<unsigned>(a.BH), static_cast<unsigned>((per + kThreads - 1) / kThreads),
                  static_cast<unsigned>(a.nprob));
  return launch_after(lin_carry_kernel, grid, kThreads, 0, st, true, a, chunk);
}

namespace {

constexpr int kMaxWidth = 256;

bool valid_linear(const ia_linear_shape_t* s, bool need_n) {
  if (!s) return false;
  if (s->B <= 0 || s->H <= 0 || s->d_k <= 0 || s->d_v <= 0) return false;
  if (need_n && s->N <= 0) return false;
  if (s->in_dtype != IA_F32 && s->in_dtype != IA_BF16) return false;
  // four problems x blocks of columns of streams in one int
  if (static_cast<long long>(s->B) * s->H > (1LL << 31) / 64) return false;
  return true;
}
bool widths_ok(const ia_linear_shape_t& s) { return s.d_k <= kMaxWidth && s.d_v <= kMaxWidth; }
bool overlap(const void* a, const void* b, size_t na, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

struct LinPlan {
  bool tc;
  int chunk, nch, nseg, cps;
};

// Segments per sequence.  A CTA runs its chunks one after the other, so a call
// with fewer streams than CTA slots leaves SMs idle; cutting each sequence
// into segments fills them, at the price of a first pass that builds the
// segments' end states (about `f` of a chunk's full cost each) and of two more
// launches.  The plan takes the count with the least time in units of one
// chunk on one slot.
LinPlan lin_plan(const ia_linear_shape_t& s, bool train) {
  LinPlan p;
  p.tc = lin_tc_supported(s);
  p.chunk = p.tc ? kLinTcChunk : C;
  p.nch = (s.N - 1) / p.chunk + 1;
  const long long bh = static_cast<long long>(s.B) * s.H;
  const long long streams = train ? bh * (2LL * lin_zblocks(s.d_v) + 2LL * lin_zblocks(s.d_k)) : bh * lin_zblocks(s.d_v);
  const int width = std::max(s.d_k, s.d_v);
  const long long slots = static_cast<long long>(num_sms()) * (p.tc || width > 128 ? 1 : width > 64 ? 2 : 4);
  // In microseconds on a B200: a chunk of the full pass and of the state-only
  // pass, what a wave of CTAs costs beside its chunks, the launch of the
  // state-only pass, and the carry over n segments.  Measured with the state
  // out: 56 chunks of d = 64 and 16 heads take 97.5 us whole, 78.5 in 2 segments,
  // 46.2 in 4, 30.9 in 8 (planned), 43.7 in 12; 55 of d = 128 take 131.7, 98.2, 63.1
  // in 4 (planned), 83.3 in 5, 72.1 in 8; 8 chunks of d = 64 and one head 17.9
  // whole, 17.6, 13.9, 11.4 in 8 (planned); of 16 heads 18.0 whole, 16.1 in 4, 15.1
  // in 8 (planned); 16 chunks of 64 heads 31.9 whole, 29.6 in 2 (planned); training
  // over 32 chunks of 16 heads 56.9 whole, 46.9 in 2 (planned).
  // On CUDA cores B2 H4 N300 48 x 80 takes 64.4 us whole, 33.0 in 5, 21.4 in 10
  // (planned), B8 H16 N2048 d64 468, 397 in 4 (planned), 391 in 10.
  const bool wide = (p.tc && !train ? s.d_k : width) > 64;   // the tensor-core pass: x and y alone
  const double full = p.tc ? (wide ? 2.2 : 1.45) : (wide ? 40.0 : 20.0);
  const double state = p.tc ? (wide ? 0.8 : 0.75) : 0.45 * full;
  const double wave = 4.5, state_wave = 3.0, extra = 1.5, carry = 2.0, carry_each = 0.04;
  if (const char* env = std::getenv("IA_LINEAR_SEGMENTS")) {   // forced count (tuning and tests)
    const int want = std::atoi(env);
    if (want >= 1) {
      p.cps = (p.nch + std::min(want, p.nch) - 1) / std::min(want, p.nch);
      p.nseg = (p.nch + p.cps - 1) / p.cps;
      return p;
    }
  }
  double best = 0.0;
  p.nseg = 1;
  p.cps = p.nch;
  // (more segments than fill the slots twice only add chunks' waves)
  const int most = static_cast<int>(std::min<long long>({p.nch, 64, 2 * slots / streams + 1}));
  for (int n = 1; n <= most; ++n) {
    const int cps = (p.nch + n - 1) / n, nseg = (p.nch + cps - 1) / cps;
    if (nseg != n) continue;
    auto waves = [&](long long ctas) { return static_cast<double>((ctas + slots - 1) / slots); };
    double t = waves(streams * n) * (cps * full + wave);
    if (n > 1) t += waves(streams * (n - 1)) * (cps * state + state_wave) + extra;
    if (n > 2) t += carry + n * carry_each;
    if (n == 1 || t < best) {
      best = t;
      p.nseg = n;
      p.cps = cps;
    }
  }
  return p;
}

size_t seg_floats(const ia_linear_shape_t& s, const LinPlan& p) {
  return static_cast<size_t>(s.B) * s.H * (p.nseg - 1) * s.d_k * s.d_v;
}

// Runs the problems in a: the segments' states first when there are several.
cudaError_t run_problems(LinArgs& a, const LinPlan& p, bool bf16, cudaStream_t st) {
  a.first[0] = 0;
  for (int i = 0; i < a.nprob; ++i) a.first[i + 1] = a.first[i] + lin_zblocks(a.p[i].dz);
  auto pass = [&](bool state_only) {
    return p.tc ? launch_lin_tc(a, state_only, st) : launch_lin_simt(a, bf16, state_only, st);
  };
  mark_launch_begin(st);
  cudaError_t e = cudaSuccess;
  if (p.nseg > 1) {
    e = pass(true);
    if (e == cudaSuccess && p.nseg > 2) e = launch_lin_carry(a, p.chunk, st);
  }
  if (e == cudaSuccess) e = pass(false);
  mark_launch_end(st);
  return e;
}

LinArgs base_args(const ia_linear_shape_t& s, const LinPlan& p, const float* log_decay, float scale, int* err) {
  LinArgs a = {};
  a.BH = s.B * s.H;
  a.H = s.H;
  a.N = s.N;
  a.nch = p.nch;
  a.nseg = p.nseg;
  a.cps = p.cps;
  a.scale = scale;
  a.log_decay = log_decay;
  a.err = err;
  return a;
}

}  // namespace
}  // namespace ia

using namespace ia;

extern "C" {

size_t ia_linear_state_bytes(const ia_linear_shape_t* s) {
  if (!valid_linear(s, false) || !widths_ok(*s)) return 0;
  return sizeof(float) * static_cast<size_t>(s->B) * s->H * s->d_k * s->d_v;
}

ia_path_t ia_linear_path(const ia_linear_shape_t* s) {
  if (!valid_linear(s, true) || !widths_ok(*s)) return IA_PATH_NONE;
  return lin_tc_supported(*s) ? IA_PATH_TENSOR_CORE : IA_PATH_SEQUENTIAL;
}

int ia_linear_prefill_segments(const ia_linear_shape_t* s) {
  return valid_linear(s, true) && widths_ok(*s) ? lin_plan(*s, false).nseg : 0;
}

int ia_linear_fwd_bwd_segments(const ia_linear_shape_t* s) {
  return valid_linear(s, true) && widths_ok(*s) ? lin_plan(*s, true).nseg : 0;
}

size_t ia_linear_prefill_workspace_bytes(const ia_linear_shape_t* s) {
  if (!valid_linear(s, true) || !widths_ok(*s)) return 0;
  return sizeof(float) * seg_floats(*s, lin_plan(*s, false));
}

size_t ia_linear_fwd_bwd_workspace_bytes(const ia_linear_shape_t* s) {
  if (!valid_linear(s, true) || !widths_ok(*s)) return 0;
  return 4 * sizeof(float) * seg_floats(*s, lin_plan(*s, true));
}

ia_status_t ia_linear_prefill_fwd(const ia_linear_shape_t* s, const void* q, const void* k, const void* v,
                                  const float* log_decay, float scale, const float* state_in, void* o,
                                  float* state_out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_linear(s, true)) return IA_ERR_INVALID_ARG;
  if (!q || !k || !v || !log_decay || !o || !std::isfinite(scale)) return IA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, log_decay, state_in, o, state_out, workspace};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return IA_ERR_INVALID_ARG;
  if (!widths_ok(*s)) return IA_ERR_UNSUPPORTED;
  const size_t sb = ia_linear_state_bytes(s);
  if (state_in && state_out && overlap(state_in, state_out, sb, sb)) return IA_ERR_INVALID_ARG;
  const LinPlan p = lin_plan(*s, false);
  const size_t need = sizeof(float) * seg_floats(*s, p);
  if (need > 0 && (!workspace || workspace_bytes < need)) return IA_ERR_WORKSPACE;
  if (inject_launch_failure()) return IA_ERR_CUDA;
  int* err = device_error_ptr();
  if (!err) return map_cuda(cudaGetLastError() == cudaSuccess ? cudaErrorUnknown : cudaErrorInvalidDevice);
  LinArgs a = base_args(*s, p, log_decay, scale, err);
  a.nprob = 1;
  a.p[0] = {q, k, v, o, state_in, state_out, static_cast<float*>(workspace), s->d_k, s->d_v, 0};
  return map_cuda(run_problems(a, p, s->in_dtype == IA_BF16, static_cast<cudaStream_t>(stream)));
}

ia_status_t ia_linear_fwd_bwd(const ia_linear_shape_t* s, const void* q, const void* k, const void* v,
                              const float* log_decay, float scale, const void* dO, void* o, void* dq, void* dk,
                              void* dv, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_linear(s, true)) return IA_ERR_INVALID_ARG;
  if (!q || !k || !v || !log_decay || !dO || !o || !dq || !dk || !dv || !std::isfinite(scale))
    return IA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, log_decay, dO, o, dq, dk, dv, workspace};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return IA_ERR_INVALID_ARG;
  if (!widths_ok(*s)) return IA_ERR_UNSUPPORTED;
  const LinPlan p = lin_plan(*s, true);
  const size_t per = seg_floats(*s, p), need = 4 * sizeof(float) * per;
  if (need > 0 && (!workspace || workspace_bytes < need)) return IA_ERR_WORKSPACE;
  if (inject_launch_failure()) return IA_ERR_CUDA;
  int* err = device_error_ptr();
  if (!err) return map_cuda(cudaGetLastError() == cudaSuccess ? cudaErrorUnknown : cudaErrorInvalidDevice);
  LinArgs a = base_args(*s, p, log_decay, scale, err);
  float* ws = static_cast<float*>(workspace);
  const int K = s->d_k, V = s->d_v;
  a.nprob = 4;
  a.p[0] = {q, k, v, o, nullptr, nullptr, ws, K, V, 0};
  a.p[1] = {dO, v, k, dq, nullptr, nullptr, ws + per, V, K, 0};
  a.p[2] = {v, dO, q, dk, nullptr, nullptr, ws + 2 * per, V, K, 1};
  a.p[3] = {k, q, dO, dv, nullptr, nullptr, ws + 3 * per, K, V, 1};
  return map_cuda(run_problems(a, p, s->in_dtype == IA_BF16, static_cast<cudaStream_t>(stream)));
}

ia_status_t ia_linear_decode_step(const ia_linear_shape_t* s, const void* q, const void* k, const void* v,
                                  const float* log_decay, float scale, const float* state_in, const int* parents,
                                  int beams, float* state_out, void* o, void* stream) {
  if (!valid_linear(s, false)) return IA_ERR_INVALID_ARG;
  if (!q || !k || !v || !log_decay || !state_in || !state_out || !o || !std::isfinite(scale))
    return IA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, log_decay, state_in, state_out, o};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return IA_ERR_INVALID_ARG;
  if (!widths_ok(*s)) return IA_ERR_UNSUPPORTED;
  const size_t sb = ia_linear_state_bytes(s);
  if (parents) {
    if (beams <= 0 || s->B % beams != 0 || (reinterpret_cast<uintptr_t>(parents) & 3u)) return IA_ERR_INVALID_ARG;
    if (overlap(state_in, state_out, sb, sb)) return IA_ERR_INVALID_ARG;
  } else if (state_in != state_out && overlap(state_in, state_out, sb, sb)) {
    return IA_ERR_INVALID_ARG;
  }
  if (inject_launch_failure()) return IA_ERR_CUDA;
  int* err = device_error_ptr();
  if (!err) return map_cuda(cudaGetLastError() == cudaSuccess ? cudaErrorUnknown : cudaErrorInvalidDevice);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return map_cuda(launch_lin_decode(*s, q, k, v, log_decay, scale, state_in, parents, beams, state_out, o, err, st));
}

}  // extern "C"
