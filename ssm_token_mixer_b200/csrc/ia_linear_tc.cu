// Linear attention with one decay per head on the tensor cores: the chunk
// algebra of ia_linear.cu with C = 128 tokens per chunk, for bf16 inputs with
// widths 64 and 128.
//
// One CTA carries one (b,h), one block of 64 columns of z and one segment of
// the sequence, chunk after chunk.  Four contractions per chunk (tcgen05, bf16
// operands, fp32 accumulators in TMEM):
//   G1  A  = X Y^T            128 x 128 x dx   operands straight from TMA
//   G2  O2 = P Z              128 x 64 x 256   P = decayed, masked A, from TMEM
//   G3  O1 = X S              128 x 64 x 2 dx  S = the entering state
//   G4  K  = Y^T (w Z)        dx x 64 x 256    w z in two bf16 parts, or three
//   out = scale (O2 + lambda^(p+1) O1),  S <- lambda^L S + K in fp32 registers
//
// Rounding.  Decays multiply fp32 accumulators wherever they can: A before it
// becomes P, O1 after the product, S in registers.  What has to be an operand
// although it is no input (P, S, and w z with the weights w = lambda^(L-1-p) of
// G4) goes in as bf16 parts.  P and S have two, which leave 2^-16 of a value,
// and so have w z where the state only feeds outputs of 8 bits: an output is off
// by its own rounding (1.66e-3 of the outputs' norm; 2.34e-3 with P and S rounded
// to bf16 once, where training of B8 H16 N2048 d64 took 103 us and not 121, of B4
// H16 N2048 d128 131 and not 158, and prompts a tenth less).  Where the caller
// takes the final state in fp32, w z has three (2^-24 of a value): the state is
// off by 1.4e-7 (N = 2048, d = 64) to 3.8e-7 (d = 128), less than token by token in
// fp32 (6e-7).
//
// Roles (448 threads, four warps at most on a quarter of the registers: 128 a
// thread; or 576, five warps: 96):
//   warps 0-3   P: A from TMEM, decayed, back to TMEM as the A operand of G2.
//               lambda^(t-s) = lambda^(t - e) lambda^(e - s) over groups of 32
//               columns that end at e <= t: both factors <= 1 and constant per
//               thread.  Groups on the other side of the diagonal are zero and
//               not read.
//   warps 4-7   O: O1, O2 from TMEM, out through shared memory and TMA stores,
//               each warp its 32 rows by itself (stores straight from the
//               registers, 32 bytes a lane, were 5 % slower).  With d = 64 the
//               rows are staged in z's own tile, which G2 was the last to read
//   warps 8-11  S: K from TMEM, S in registers, its parts to shared memory for
//               the next chunk's G3
//   warps 12-15 W: w z for G4 (where there are none, O does it; a pass for the
//               states alone has nothing else for P and O to do)
//   then a warp for the TMA loads and one that issues G1-G4
// Per chunk G4, G1 of the next chunk, G3 (or G3 first) and G2 are issued, so
// that P and the state work while the products of the other roles run.  The
// loops of the roles are kept short on purpose: with everything unrolled the
// warps spent six of seven issue slots waiting for instructions (three roles
// of straight-line code do not fit an SM's instruction caches; ncu, B8 H16
// N2048 d64).  Only the warp that issues the products runs straight-line code:
// its issuing is on the chunk's path (training of B4 H16 N2048 d128 137.4 us with
// four products a turn, 132.0 with all).  Letting G4 wait for K alone and not for
// the operand of S as well changed nothing (training of B8 H16 N2048 d64 122.7 us
// with, 121.0 without).  Waits are bounded mbarrier waits with a CTA-wide abort
// flag.
//
// Pairs of times in these comments that are below the present ones were taken
// before P and S had second parts.
//
// Measured: prefill with the state of B8 H16 N2048 d64 36.0 us, of B4 H16 N2048
// d128 48.4; training 122 and 157.  Tensor pipe 44 to 48 % active, issue slots 45
// to 54 %: what bounds a chunk is the chain of its four roles, P's above all.
#include <algorithm>
#include <cuda.h>

#include "ia_device.cuh"
#include "ia_internal.h"
#include "ia_launch.h"
#include "ia_linear.h"

namespace ia {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled();   // ia_prefill_tc.cu

namespace {

constexpr int C = kLinTcChunk;
constexpr int kBox = C * 128;           // 64 bf16 columns x 128 tokens, 128-byte swizzled: 16 KB
constexpr int kRoleThreads = 128;
// With d = 64 and outputs to write, z is weighed by warps of its own (at 96
// registers a thread), else by the output warps.
constexpr bool has_w(int maxdx, bool state_only) { return maxdx == 64 && !state_only; }
constexpr int threads(int maxdx, bool state_only) { return (has_w(maxdx, state_only) ? 4 : 3) * kRoleThreads + 64; }
constexpr int kBad = 8;                 // chunks whose marks of NaN are kept apart
constexpr uint32_t kAtom = 1024;        // 8 rows of 128 bytes

template <int MAXDX, bool STATE_ONLY, int PARTS>
struct Cfg {
  // Stages.  X is released late (by G3), Y by G4; Z is needed first and released
  // last.  The second part of S and the third of w z leave X two stages at d = 64
  // when the state is taken (three with outputs staged in z's tile) and one at
  // d = 128, where outputs keep a tile of their own: staged in z's, with four and
  // three of those, training of B4 H16 N2048 d128 takes 161 us, and 158.
  static constexpr bool kFull3 = PARTS == 3 && !STATE_ONLY;
  static constexpr bool kOutInZ = MAXDX == 64;
  static constexpr int NX = STATE_ONLY ? 0 : MAXDX == 64 ? (kFull3 ? 2 : 3) : 1;
  static constexpr int NY = STATE_ONLY && PARTS == 2 ? 3 : 2;
  static constexpr int NT = STATE_ONLY ? 3 : MAXDX == 64 ? (kFull3 ? 3 : 4) : kFull3 ? 2 : 3;
  static constexpr int NZ = MAXDX == 64 || STATE_ONLY ? 2 : 1;         // buffers of w z
  // TMEM columns (A twice, with P in its place).  With wide X a second O1 lets
  // G3 go first, so that X's stage is loaded again early: its stages alone do
  // not hide the load (forward of B4 H16 N2048 d128 44.6 us without, 41.5 with).
  // That leaves 64 columns for K, whose parts are then contracted one after the
  // other (16 products instead of 8 twice as wide); with d = 64 and three stages
  // this costs more than it gives (B8 H12 N2048: 27.1 us, and 27.8).
  static constexpr bool kO1Twice = MAXDX == 128 && !STATE_ONLY;
  static constexpr uint32_t kTA = 0, kTO1 = 256, kTO2 = kO1Twice ? 384 : 320, kTK = kO1Twice ? 448 : 384;
  // Every problem has dx = 64, and K 64 rows: a third less of shared memory is
  // read for G4 than with 128 rows of which half mean nothing.
  static constexpr bool kHalf = MAXDX == 64;
  static constexpr int TX = MAXDX / 64 * kBox;
  static constexpr int S_Y = NX * TX;
  static constexpr int S_Z = S_Y + NY * TX;
  static constexpr int S_ZW = S_Z + NT * kBox;          // each: its parts
  static constexpr int kSPart = MAXDX * 128;            // [dx][64] bf16, 128-byte swizzled
  static constexpr int S_SB = S_ZW + NZ * PARTS * kBox; // S in two parts
  static constexpr int S_OUT = S_SB + (STATE_ONLY ? 0 : 2 * kSPart);
  static constexpr int S_BAR = S_OUT + (STATE_ONLY || kOutInZ ? 0 : kBox);
  static constexpr int S_POW = S_BAR + 320;             // lambda^n, n = 0 .. C - 1
  static constexpr int SMEM = S_POW + C * 4 + 1024;     // + alignment of the base
  static_assert(NX <= 3 && NY <= 3 && NT <= 4 && NZ <= 2, "their barriers");
  static_assert(SMEM <= 232448, "what a CTA may have");
};

enum Bar {
  kFullX = 0, kFullY = 3, kFullZ = 6, kFreeX = 10, kFreeY = 13, kFreeZ = 16, kAFull = 20, kPReady = 22, kZReady = 24,
  kZFree = 26, kSReady = 28, kSFree, kKFull, kOFull, kOFree, kDrain, kBars
};

struct Maps {
  CUtensorMap in[4];    // q, k, v, dO
  CUtensorMap out[4];   // by problem
};
struct MapIdx {
  int x, y, z;
};
struct TcParams {
  LinArgs a;
  MapIdx mi[4];
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return pack_bf16(lo, hi);
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// What a pair has left beside its bf16 part w (exact).
__device__ __forceinline__ uint64_t rest2(uint64_t v, uint32_t w) {
  return f2_fma(f2_pack(bf_lo(w), bf_hi(w)), f2_pack(-1.f, -1.f), v);
}

// True in one lane of the (converged) warp.  Unlike a test of the lane number
// it tells the compiler that a single thread runs the branch, so the operands
// of the tensor-core and copy instructions in it go to uniform registers at
// once instead of through a loop over the active lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// The products and commits of the MMA warp: its lanes run the same code, so that
// descriptors and addresses stay in uniform registers, and `lead` lets one
// lane issue.
__device__ __forceinline__ void mma_ss(bool lead, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(static_cast<uint32_t>(lead))
      : "memory");
}
__device__ __forceinline__ void mma_ts(bool lead, uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc), "r"(static_cast<uint32_t>(lead))
      : "memory");
}
__device__ __forceinline__ void commit_to(bool lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(static_cast<uint32_t>(lead))
      : "memory");
}

// kind::f16 instruction descriptor with bf16 A and B, fp32 D.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int a_mn, int b_mn) {
  return idesc_f16(M, N, a_mn, b_mn) | (1u << 7) | (1u << 10);
}

template <int MAXDX, bool STATE_ONLY, int PARTS>
__global__ void __launch_bounds__(has_w(MAXDX, STATE_ONLY) ? 640 : 512, 1) lin_tc_kernel(const __grid_constant__ TcParams prm,
                                                        const __grid_constant__ Maps maps) {
  using K = Cfg<MAXDX, STATE_ONLY, PARTS>;
  constexpr int kNX = K::NX ? K::NX : 1, NY = K::NY, NT = K::NT;
  constexpr bool kW = has_w(MAXDX, STATE_ONLY);
  // The state-only pass has room for two K, so that one is contracted while the
  // state takes the other (its barriers: those of A and P, which it has no other
  // use for), and its P and O warps weigh half of z each: a chunk of d = 128
  // takes 0.8 us, and 1.4 with one K, weighed by four warps.
  auto k_full = [](int c) { return STATE_ONLY ? kAFull + (c & 1) : static_cast<int>(kKFull); };
  auto k_col = [](int c) { return K::kTK - (STATE_ONLY ? 128 * (c & 1) : 0); };
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const LinArgs& a = prm.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  // (b,h), problem, block of z columns, segment
  const int nseg = STATE_ONLY ? a.nseg - 1 : a.nseg;
  const long long stream = blockIdx.x / nseg;
  const int seg = static_cast<int>(blockIdx.x - stream * nseg);
  const int per = a.first[a.nprob];
  const int bh = static_cast<int>(stream / per);
  const int r = static_cast<int>(stream - static_cast<long long>(bh) * per);
  int pi = 0;
  while (pi + 1 < a.nprob && r >= a.first[pi + 1]) ++pi;
  const LinProblem& pr = a.p[pi];
  const int z0 = (r - a.first[pi]) * kLinZB;
  const int dx = pr.dx, dz = pr.dz, nbx = dx / 64;
  const bool rev = pr.reverse != 0;
  const int h = bh % a.H;
  const int c0 = seg * a.cps, n = min(a.nch, c0 + a.cps) - c0;
  auto chunk_at = [&](int c) { return rev ? a.nch - 1 - (c0 + c) : c0 + c; };

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + K::S_BAR);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + K::S_BAR + 8 * kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + K::S_BAR + 8 * kBars + 4);
  int* bad = reinterpret_cast<int*>(smem + K::S_BAR + 8 * kBars + 8);   // [kBad]
  static_assert(8 * kBars + 8 + 4 * kBad <= 320, "barriers and flags fit their slot");
  const uint32_t sbase = smem_u32(smem);
  auto sX = [&](int c) { return (c % kNX) * K::TX; };
  auto sY = [&](int c) { return K::S_Y + (c % NY) * K::TX; };
  auto sZ = [&](int c) { return K::S_Z + (c % NT) * kBox; };

  if (warp == 0) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < kBars; ++i) {   // arrivals: one, or one per warp of the roles that fill the buffer
      const bool warps4 = i == kPReady || i == kPReady + 1 || i == kSReady || i == kOFree ||
                          i == kZReady || i == kZReady + 1;
      const bool warps8 = STATE_ONLY && (i == kZReady || i == kZReady + 1);
      const bool stored = K::kOutInZ && !STATE_ONLY && i >= kFreeZ && i < kFreeZ + NT;   // by O's warps
      mbar_init(bars + i, warps8 ? 8 : warps4 || stored ? 4 : 1);
    }
    for (int i = 0; i < kBad; ++i) bad[i] = C;
    *abort_flag = 0;
    fence_barrier_init();
  }
  const float graw = a.log_decay[h];
  if (tid == 0 && !(graw <= 0.f)) atomicOr(a.err, kErrParamRange);
  const float g = lin_log_decay(graw);
  float* pw = reinterpret_cast<float*>(smem + K::S_POW);
  if (tid < C) pw[tid] = expf(g * tid);
  griddep_launch_dependents();
  griddep_wait();   // the segments' states, when a pass before this one built them
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  auto wait = [&](int bar, uint32_t parity) {
    return mbar_wait_or_abort(bars + bar, parity & 1u, a.err, abort_flag);
  };
  // one outcome for a warp: what follows is warp-wide
  auto warp_wait = [&](int bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };

  // w z of chunk c (of a half in the state-only pass) in bf16 parts, at z's own
  // offsets (row = token); u: the thread among its role's 128
  auto weigh = [&](int c, int u, int half) -> bool {
    constexpr int kIter = STATE_ONLY ? 4 : 8;
    const int L = min(C, a.N - chunk_at(c) * C);
    uint8_t* zw = smem + K::S_ZW + (c % K::NZ) * PARTS * kBox;
    const uint8_t* zs = smem + sZ(c);
    if (c >= K::NZ && !warp_wait(kZFree + c % K::NZ, c / K::NZ - 1)) return false;   // G4 has read the buffer
    if (!warp_wait(kFullZ + c % NT, c / NT)) return false;
    // (two turns at a time: training of B8 H16 N2048 d64 104.3 us with one, 102.0)
    const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
    __nv_bfloat162 probe = zero;   // 0 * z: NaN if any z is not finite
    uint32_t off = (4 * half * kRoleThreads + u) * 16;
    int t = 64 * half + (u >> 3);
    uint4 zn = *reinterpret_cast<const uint4*>(zs + off);
#pragma unroll 2
    for (int i = 0; i < kIter; ++i) {
      const uint32_t zz[4] = {zn.x, zn.y, zn.z, zn.w};
      if (i + 1 < kIter) zn = *reinterpret_cast<const uint4*>(zs + off + 16 * kRoleThreads);
      const float wt = t < L ? pw[rev ? t : L - 1 - t] : 0.f;
      const uint64_t w2 = f2_pack(wt, wt);
      uint32_t part[PARTS][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        probe = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&zz[e]), zero, probe);
        uint64_t v = f2_mul(f2_pack(bf_lo(zz[e]), bf_hi(zz[e])), w2);
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
          part[k][e] = pack2(v);
          if (k + 1 < PARTS) v = rest2(v, part[k][e]);
        }
      }
#pragma unroll
      for (int k = 0; k < PARTS; ++k)
        *reinterpret_cast<uint4*>(zw + k * kBox + off) = make_uint4(part[k][0], part[k][1], part[k][2], part[k][3]);
      off += 16 * kRoleThreads;
      t += 16;
    }
    if (!STATE_ONLY && !__hbeq2(probe, zero)) {
      // A NaN or infinity in z: 0 * z of the masked half would reach the
      // tokens before it.  G2 reads a zero instead and the output warps write
      // NaN from its token on.
#pragma unroll 1
      for (int i = 0; i < 32; ++i) {
        const int it = i >> 2, tt = 16 * it + (u >> 3);
        uint32_t* z = reinterpret_cast<uint32_t*>(smem + sZ(c) + (it * kRoleThreads + u) * 16) + (i & 3);
        uint32_t x = *z;
        if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
        if ((x & 0x7f800000u) == 0x7f800000u) x &= 0x0000ffffu;
        if (x != *z) {
          *z = x;
          atomicMin(bad + c % kBad, rev ? C - 1 - tt : tt);
        }
      }
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + kZReady + c % K::NZ);
    return true;
  };

  if (warp < 4) {
    // ------------------------------------------------------------------- P
    if (STATE_ONLY) {
#pragma unroll 1
      for (int c = 0; c < n; ++c)
        if (!weigh(c, tid, 0)) break;
    } else {
      const int t = tid;   // row of the chunk
      uint64_t e[16];      // lambda^(distance of column 32 gr + j from its group's near end), pairs
#pragma unroll
      for (int i = 0; i < 16; ++i)
        e[i] = rev ? f2_pack(pw[2 * i], pw[2 * i + 1]) : f2_pack(pw[31 - 2 * i], pw[30 - 2 * i]);
      for (int c = 0; c < n; ++c) {
        const int b = c & 1;
        if (!warp_wait(kAFull + b, c >> 1)) break;
        tc_fence_after();
        const uint32_t ta = tmem + (static_cast<uint32_t>(warp) << 21) + K::kTA + 128 * b;
#pragma unroll 1
        for (int gr = 0; gr < 4; ++gr) {
          const int side = rev ? gr - warp : warp - gr;   // > 0: whole group, 0: the diagonal one, < 0: nothing
          const float f = pw[side > 0 ? (rev ? 32 * gr - t : t - 32 * gr - 31) : 0];
          const uint64_t ff = f2_pack(f, f);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {   // 16 columns at a time
            uint32_t w[16];   // of 16 columns: the first parts of their 8 pairs, then the second ones
            auto split = [&](int i, uint64_t pair) {
              w[i] = pack2(pair);
              w[8 + i] = pack2(rest2(pair, w[i]));
            };
            if (side < 0) {
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = 0u;
            } else {
              uint32_t v[16];
              tmem_ld16(ta + 32 * gr + 16 * hf, v);
              tmem_ld_wait16(v);
              if (side > 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  split(i, f2_mul(f2_mul(f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), e[8 * hf + i]), ff));
              } else {
                // select, not multiply: a masked score may be infinite or NaN
                auto val = [&](int j) {
                  const int d = rev ? 16 * hf + j - lane : lane - 16 * hf - j;
                  return d >= 0 ? __uint_as_float(v[j]) * pw[max(d, 0)] : 0.f;
                };
#pragma unroll
                for (int i = 0; i < 8; ++i) split(i, f2_pack(val(2 * i), val(2 * i + 1)));
                __syncwarp();   // d >= 0 differs between lanes, and the store is the whole warp's
              }
            }
            tmem_st16(ta + 32 * gr + 16 * hf, w);   // the columns of A that it came from
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kPReady + b);
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------- O
    const int u = tid - kRoleThreads;
    bool alive = true;
    const int p = rev ? C - 1 - u : u;
    const float hd = a.scale * expf(g * (p + 1));
    const uint64_t scale2 = f2_pack(a.scale, a.scale), hd2 = f2_pack(hd, hd);
    const CUtensorMap* mo = &maps.out[pi];
#pragma unroll 1
    for (int c = -1; c < n; ++c) {
      if (!kW && c + 1 < n) alive = alive && weigh(c + 1, u, STATE_ONLY);
      if (c < 0) continue;           // the first chunk is weighed before the first output
      if (STATE_ONLY) {
        if (!alive) break;
        continue;
      }
      if (!alive || !warp_wait(kOFull, c)) break;
      tc_fence_after();
      const int from = *reinterpret_cast<volatile int*>(bad + c % kBad);
      if (u == 0) bad[(c + kBad - 1) % kBad] = C;   // the last chunk's: every warp has read it before this kOFull
      const uint32_t to = tmem + (static_cast<uint32_t>(warp - 4) << 21);
      const int off = (K::kOutInZ ? sZ(c) : K::S_OUT) + 128 * u;   // this thread's row, 128-byte swizzled like z
      if (!K::kOutInZ) {   // the warp's last store has left its rows
        if (lane == 0) bulk_wait_read_0();
        __syncwarp();
      }
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t v1[16], v2[16], w[8];
        tmem_ld16(to + K::kTO1 + (K::kO1Twice ? 64 * (c & 1) : 0) + 16 * q, v1);
        tmem_ld16(to + K::kTO2 + 16 * q, v2);
        tmem_ld_wait16(v1);
        tmem_ld_wait16(v2);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float lo, hi;
          f2_unpack(f2_fma(hd2, f2_pack(__uint_as_float(v1[2 * i]), __uint_as_float(v1[2 * i + 1])),
                           f2_mul(scale2, f2_pack(__uint_as_float(v2[2 * i]), __uint_as_float(v2[2 * i + 1])))), lo, hi);
          w[i] = pack_bf16(lo, hi);
        }
        if (p >= from)
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = 0x7fc07fc0u;   // NaN
        __syncwarp();   // p >= from differs between lanes, and the next loads from TMEM are the whole warp's
        *reinterpret_cast<uint4*>(smem + off + (((2 * q) ^ (u & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(smem + off + (((2 * q + 1) ^ (u & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bars + kOFree);
        const int t = chunk_at(c) * C + u;   // of the warp's first row
        if (t < a.N) {
          tma_store_3d(mo, sbase + off, z0, t, bh);
          bulk_commit();
        }
        if (K::kOutInZ) {
          bulk_wait_read_0();
          mbar_arrive(bars + kFreeZ + c % NT);
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  } else if (warp < 12) {
    // ------------------------------------------------------------------- S
    // The accumulator K of dx = 64 has M = 64 rows, in lanes 0-15 of each warp's
    // quadrant: a lane takes half a row.  Else thread u takes row u.
    constexpr int kCols = K::kHalf ? 32 : 64;
    const int u = tid - 2 * kRoleThreads;
    const int row = K::kHalf ? 16 * (warp - 8) + (lane & 15) : u, col = K::kHalf ? 32 * (lane >> 4) : 0;
    const bool holds = row < dx;
    const long long per_state = static_cast<long long>(dx) * dz;
    const long long at_state = static_cast<long long>(row) * dz + z0 + col;
    uint64_t S[kCols / 2];       // its columns in pairs
    const float dec_full = lin_decay(g * C);
    {
      const float* s0 = seg == 0 ? (pr.state_in ? pr.state_in + bh * per_state : nullptr)
                                 : STATE_ONLY ? nullptr : pr.seg + (static_cast<long long>(bh) * (a.nseg - 1) + seg - 1) * per_state;
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s0 && holds) v = *reinterpret_cast<const float4*>(s0 + at_state + 4 * i);
        S[2 * i] = f2_pack(v.x, v.y), S[2 * i + 1] = f2_pack(v.z, v.w);
      }
    }
    auto write_operand = [&]() {   // and K has been read: the next G4 may overwrite it
      if (holds)
#pragma unroll
        for (int j = 0; j < kCols / 8; ++j) {
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            w[k] = pack2(S[4 * j + k]);
            w[4 + k] = pack2(rest2(S[4 * j + k], w[k]));
          }
          uint8_t* dst = smem + K::S_SB + row * 128 + (((col / 8 + j) ^ (row & 7)) << 4);
          *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(dst + K::kSPart) = make_uint4(w[4], w[5], w[6], w[7]);
        }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + kSReady);
    };
#pragma unroll 1
    for (int c = -1; c < n; ++c) {
      if (c >= 0) {
      const int L = min(C, a.N - chunk_at(c) * C);
      const bool whole = L == C || rev;
      const float dec = whole ? dec_full : lin_decay(g * L);
      const uint64_t dec2 = f2_pack(dec, dec);
      if (g * (whole ? C : L) > kLinSlow) {   // before K is there, and two loops rather than a choice per entry
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) S[i] = f2_fma(dec2, S[i], S[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) S[i] = f2_mul(dec2, S[i]);
      }
      if (STATE_ONLY ? !warp_wait(k_full(c), c >> 1) : !warp_wait(kKFull, c)) break;
      tc_fence_after();
      const uint32_t tk = tmem + (static_cast<uint32_t>(warp - 8) << 21) + k_col(c);
      if (K::kHalf || 32 * (warp - 8) < dx) {
#pragma unroll
        for (int i = 0; i < kCols / 16; ++i) {
          uint32_t v[16], w[16];
          auto load = [&](uint32_t from, uint32_t (&r)[16]) {
            if (K::kHalf) tmem_ld16_halves<32>(from, r);
            else tmem_ld16(from, r);
          };
          load(tk + 16 * i, v);
          if (!K::kO1Twice) load(tk + 64 + 16 * i, w);
          tmem_ld_wait16(v);
          if (!K::kO1Twice) tmem_ld_wait16(w);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint64_t add = f2_pack(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
            if (!K::kO1Twice) add = f2_add(add, f2_pack(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1])));
            S[8 * i + k] = f2_add(S[8 * i + k], add);
          }
        }
      }
      tc_fence_before();
      }
      if (STATE_ONLY) {
        __syncwarp();
        if (c >= 0 && lane == 0) mbar_arrive(bars + kPReady + (c & 1));   // K's buffer is free
      } else if (c + 1 < n) {
        if (c >= 0 && !warp_wait(kSFree, c)) break;   // G3 has read the old operand
        write_operand();
      }
    }
    float* dst = STATE_ONLY ? pr.seg + (static_cast<long long>(bh) * (a.nseg - 1) + seg) * per_state
                            : (pr.state_out && seg == a.nseg - 1) ? pr.state_out + bh * per_state : nullptr;
    if (dst && holds)
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) {
        float4 v;
        f2_unpack(S[2 * i], v.x, v.y);
        f2_unpack(S[2 * i + 1], v.z, v.w);
        *reinterpret_cast<float4*>(dst + at_state + 4 * i) = v;
      }
  } else if (kW && warp < 16) {
    // ------------------------------------------------------------------- W
    const int u = tid - 3 * kRoleThreads;
#pragma unroll 1
    for (int c = 0; c < n; ++c)
      if (!weigh(c, u, 0)) break;
  } else if (warp == (kW ? 16 : 12)) {
    // ---------------------------------------------------------------- loads
    if (elect_one()) {
      const CUtensorMap *mx = &maps.in[prm.mi[pi].x], *my = &maps.in[prm.mi[pi].y], *mz = &maps.in[prm.mi[pi].z];
      int issued_z = 0, issued_y = 0, issued_x = 0;
      auto fetch = [&](int bar, int dst, const CUtensorMap* m, int boxes, int col, int t0) {
        mbar_arrive_expect_tx(bars + bar, boxes * kBox);
#pragma unroll 1
        for (int x = 0; x < boxes; ++x) tma_load_3d(sbase + dst + x * kBox, m, col + 64 * x, t0, bh, bars + bar);
      };
#pragma unroll 1
      for (int c = 0; c < n; ++c) {
        const int t0 = chunk_at(c) * C;
        if (c >= NT && !wait(kFreeZ + c % NT, c / NT - 1)) break;
        fetch(kFullZ + c % NT, sZ(c), mz, 1, z0, t0);
        issued_z = c + 1;
        if (c >= NY && !wait(kFreeY + c % NY, c / NY - 1)) break;
        fetch(kFullY + c % NY, sY(c), my, nbx, 0, t0);
        issued_y = c + 1;
        if (STATE_ONLY) continue;
        if (c >= kNX && !wait(kFreeX + c % kNX, c / kNX - 1)) break;
        fetch(kFullX + c % kNX, sX(c), mx, nbx, 0, t0);
        issued_x = c + 1;
      }
      // no copy lands after the block exits
#pragma unroll 1
      for (int c = max(0, issued_z - NT); c < issued_z; ++c) mbar_wait(bars + kFullZ + c % NT, (c / NT) & 1, a.err);
#pragma unroll 1
      for (int c = max(0, issued_y - NY); c < issued_y; ++c) mbar_wait(bars + kFullY + c % NY, (c / NY) & 1, a.err);
#pragma unroll 1
      for (int c = max(0, issued_x - kNX); c < issued_x; ++c) mbar_wait(bars + kFullX + c % kNX, (c / kNX) & 1, a.err);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ MMA
    {
      const bool lead = elect_one();
      bool issued = false;
      // descriptors of a stage's tiles: K-major for G1 and G3's X, MN-major
      // (the token index contracted) for G2 and G4
      auto kmajor = [&](int off) { return smem_desc_sw128(sbase + off, 16, kAtom); };
      auto mnmajor = [&](int off) { return smem_desc_sw128(sbase + off, kBox, kAtom); };
      constexpr uint64_t kTok = (2 * kAtom) >> 4;   // 16 tokens (or rows of S) further
      auto g1 = [&](int c) {
        const uint64_t x = kmajor(sX(c)), y = kmajor(sY(c));
#pragma unroll
        for (int b = 0; b < MAXDX / 64; ++b)
#pragma unroll
          for (int kk = 0; b < nbx && kk < 4; ++kk) {
            const uint64_t step = (b * kBox + kk * 32) >> 4;
            mma_ss(lead, tmem + K::kTA + 128 * (c & 1), x + step, y + step, idesc_bf16(128, 128, 0, 0), b + kk > 0);
          }
        commit_to(lead, bars + kAFull + (c & 1));
      };
      auto g3 = [&](int c) {
        const uint64_t x = kmajor(sX(c)), sb = mnmajor(K::S_SB);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int b = 0; b < MAXDX / 64; ++b)
#pragma unroll
            for (int kk = 0; b < nbx && kk < 4; ++kk)
              mma_ss(lead, tmem + K::kTO1 + (K::kO1Twice ? 64 * (c & 1) : 0), x + ((b * kBox + kk * 32) >> 4),
                     sb + (part * K::kSPart >> 4) + (4 * b + kk) * kTok, idesc_bf16(128, 64, 0, 1), part + b + kk > 0);
        commit_to(lead, bars + kSFree);
        commit_to(lead, bars + kFreeX + c % kNX);
      };
      auto g4 = [&](int c) {
        // (beside wider problems, the rows of K past dx = 64 are taken from the
        // next tile in shared memory and never read)
        const int zb = c % K::NZ;
        const uint64_t y = mnmajor(sY(c)), zw = mnmajor(K::S_ZW + zb * PARTS * kBox);
        if (K::kO1Twice) {   // the parts one after the other
#pragma unroll
          for (int kk = 0; kk < 8 * PARTS; ++kk)
            mma_ss(lead, tmem + k_col(c), y + (kk & 7) * kTok, zw + kk * kTok, idesc_bf16(128, 64, 1, 1), kk > 0);
        } else {             // the first two side by side, the third into the second's columns
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss(lead, tmem + k_col(c), y + kk * kTok, zw + kk * kTok, idesc_bf16(K::kHalf ? 64 : 128, 128, 1, 1), kk > 0);
          if (PARTS == 3)
#pragma unroll 4
            for (int kk = 0; kk < 8; ++kk)
              mma_ss(lead, tmem + k_col(c) + 64, y + kk * kTok, zw + ((2 * kBox) >> 4) + kk * kTok,
                     idesc_bf16(K::kHalf ? 64 : 128, 64, 1, 1), 1);
        }
        commit_to(lead, bars + k_full(c));
        commit_to(lead, bars + kZFree + zb);
        commit_to(lead, bars + kFreeY + c % NY);   // G1 of this chunk came before
        if (STATE_ONLY) commit_to(lead, bars + kFreeZ + c % NT);
      };
      auto g2 = [&](int c) {
        const uint64_t z = mnmajor(sZ(c));
#pragma unroll
        for (int kk = 0; kk < 16; ++kk)   // 16 tokens of P's first part, then of its second
          mma_ts(lead, tmem + K::kTO2, tmem + K::kTA + 128 * (c & 1) + 8 * kk, z + (kk >> 1) * kTok, idesc_bf16(128, 64, 0, 1), kk > 0);
        commit_to(lead, bars + kOFull);
        if (!K::kOutInZ) commit_to(lead, bars + kFreeZ + c % NT);
      };
      bool ok = true;
      if (!STATE_ONLY) {
        ok = warp_wait(kFullX, 0) && warp_wait(kFullY, 0);
        if (ok) {
          tc_fence_after();
          g1(0);
          issued = true;
        }
      }
#pragma unroll 1
      for (int c = 0; ok && c < n; ++c) {
        // S's operand is made, and K taken
        if (STATE_ONLY ? c >= 2 && !warp_wait(kPReady + (c & 1), (c >> 1) - 1) : !warp_wait(kSReady, c)) break;
        if (K::kO1Twice) {
          tc_fence_after();
          g3(c);
        }
        if (!warp_wait(kZReady + c % K::NZ, c / K::NZ)) break;
        if (STATE_ONLY && !warp_wait(kFullY + c % NY, c / NY)) break;   // (else G1 has waited for Y)
        tc_fence_after();
        g4(c);
        issued = true;
        if (!STATE_ONLY) {
          if (c + 1 < n) {
            if (!warp_wait(kFullX + (c + 1) % kNX, (c + 1) / kNX) || !warp_wait(kFullY + (c + 1) % NY, (c + 1) / NY)) break;
            tc_fence_after();
            g1(c + 1);
          }
          if (c > 0 && !warp_wait(kOFree, c - 1)) break;
          if (!K::kO1Twice) {
            tc_fence_after();
            g3(c);
          }
          if (!warp_wait(kPReady + (c & 1), c >> 1)) break;
          tc_fence_after();
          g2(c);
        }
      }
      if (issued) {   // every product is done before TMEM and shared memory go
        commit_to(lead, bars + kDrain);
        mbar_wait(bars + kDrain, 0, a.err);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// [BH][N][W] bf16 as boxes of 64 columns x `rows` tokens of one (b,h), 128-byte
// swizzled; tokens past N read as zero and are not written.
bool encode_map(CUtensorMap* m, const void* x, int BH, int N, int W, int rows) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(W), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(BH)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(W) * 2, static_cast<cuuint64_t>(N) * W * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MAXDX, bool STATE_ONLY, int PARTS>
cudaError_t launch(const TcParams& prm, const Maps& maps, cudaStream_t st) {
  const LinArgs& a = prm.a;
  const long long grid = static_cast<long long>(a.BH) * a.first[a.nprob] * (STATE_ONLY ? a.nseg - 1 : a.nseg);
  if (grid > (1LL << 31) - 1) return cudaErrorInvalidConfiguration;
  constexpr int kSmem = Cfg<MAXDX, STATE_ONLY, PARTS>::SMEM;
  auto kern = lin_tc_kernel<MAXDX, STATE_ONLY, PARTS>;
  if (cudaError_t e = allow_smem(kern, kSmem); e != cudaSuccess) return e;
  return launch_after(kern, static_cast<unsigned>(grid), threads(MAXDX, STATE_ONLY), kSmem, st, a.nseg > 1 && !STATE_ONLY, prm, maps);
}
template <int MAXDX>
cudaError_t launch(const TcParams& prm, const Maps& maps, bool state_only, bool keep_state, cudaStream_t st) {
  if (state_only) return keep_state ? launch<MAXDX, true, 3>(prm, maps, st) : launch<MAXDX, true, 2>(prm, maps, st);
  return keep_state ? launch<MAXDX, false, 3>(prm, maps, st) : launch<MAXDX, false, 2>(prm, maps, st);
}

}  // namespace

bool lin_tc_supported(const ia_linear_shape_t& s) {
  return s.in_dtype == IA_BF16 && (s.d_k == 64 || s.d_k == 128) && (s.d_v == 64 || s.d_v == 128);
}

cudaError_t launch_lin_tc(const LinArgs& a, bool state_only, cudaStream_t st) {
  TcParams prm = {};
  prm.a = a;
  Maps maps;
  int maxdx = 0;
  bool keep_state = false;
  for (int i = 0; i < a.nprob; ++i) {
    maxdx = std::max(maxdx, a.p[i].dx);
    keep_state = keep_state || a.p[i].state_out;
  }
  const void* seen[4] = {};
  int width[4] = {}, count = 0;
  auto input = [&](const void* x, int W) {   // one map per tensor, whichever roles it has
    for (int i = 0; i < count; ++i)
      if (seen[i] == x && width[i] == W) return i;
    if (count == 4 || !encode_map(&maps.in[count], x, a.BH, a.N, W, C)) return -1;
    seen[count] = x;
    width[count] = W;
    return count++;
  };
  for (int i = 0; i < a.nprob; ++i) {
    const LinProblem& p = a.p[i];
    prm.mi[i] = {input(p.x, p.dx), input(p.y, p.dx), input(p.z, p.dz)};
    if (prm.mi[i].x < 0 || prm.mi[i].y < 0 || prm.mi[i].z < 0) return cudaErrorNotSupported;
    if (!state_only && !encode_map(&maps.out[i], p.out, a.BH, a.N, p.dz, 32)) return cudaErrorNotSupported;
  }
  return maxdx == 64 ? launch<64>(prm, maps, state_only, keep_state, st) : launch<128>(prm, maps, state_only, keep_state, st);
}

}  // namespace ia
