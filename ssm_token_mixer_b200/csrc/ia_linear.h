// Internal launch interface of the linear-attention kernels.
//
// All of it is one operation.  With x, y of width dx and z of width dz,
//   out_t = scale * sum_{s <= t} lambda^(t-s) (x_t . y_s) z_s        ("forward")
// or the sum over s >= t of lambda^(s-t) ... ("reverse"), gives
//   o  : x, y, z = q, k, v        dq : x, y, z = dO, v, k
//   dk : v, dO, q in reverse      dv : k, q, dO in reverse,
// so the training step is four problems of one kernel in one launch.
#pragma once

#include <cuda_runtime.h>

#include "../../include/ia.h"

namespace ia {

struct LinProblem {
  const void* x;
  const void* y;
  const void* z;
  void* out;                // not written by a pass for the end states alone
  const float* state_in;    // [BH][dx][dz] or null
  float* state_out;         // same or null
  float* seg;               // [BH][nseg - 1][dx][dz]: end states of the segments but the last
  int dx, dz, reverse;
};

struct LinArgs {
  LinProblem p[4];
  int nprob;
  int first[5];             // prefix counts over the problems of a (b,h)'s blocks of 64 columns of z
  int BH, H, N;
  int nch;                  // chunks per sequence
  int nseg, cps;            // segments per sequence, chunks per segment
  float scale;
  const float* log_decay;
  int* err;
};

constexpr int kLinZB = 64;  // columns of z per CTA

inline int lin_zblocks(int dz) { return (dz + kLinZB - 1) / kLinZB; }

// The decay exponent a kernel works with: -inf becomes a finite value whose
// multiples still give lambda^0 = 1 and lambda^n = 0 (0 * -inf would be NaN).
__host__ __device__ inline float lin_log_decay(float g) { return g > -1e30f ? g : -1e30f; }

// Decays above 1/2 are taken from expm1, so that those near 1 keep their bits;
// below, where 1 + expm1 would cancel, from exp.  Exponents above this are the
// former's.
constexpr float kLinSlow = -0.693147f;
#ifdef __CUDACC__
// exp(e) - 1 or exp(e), by that rule: what S is multiplied with, beside S or alone.
__device__ __forceinline__ float lin_decay(float e) { return e > kLinSlow ? expm1f(e) : expf(e); }
#endif

bool lin_tc_supported(const ia_linear_shape_t& s);
constexpr int kLinTcChunk = 128;

// state_only: run every segment but the last from its start for its end state.
cudaError_t launch_lin_simt(const LinArgs& a, bool bf16, bool state_only, cudaStream_t st);
cudaError_t launch_lin_tc(const LinArgs& a, bool state_only, cudaStream_t st);
// Composes the segments' end states into running ones, in place.
cudaError_t launch_lin_carry(const LinArgs& a, int chunk, cudaStream_t st);

cudaError_t launch_lin_decode(const ia_linear_shape_t& s, const void* q, const void* k, const void* v,
                              const float* log_decay, float scale, const float* state_in, const int* parents,
                              int beams, float* state_out, void* o, int* err, cudaStream_t st);

}  // namespace ia
