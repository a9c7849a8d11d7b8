// Index arithmetic of the row kernels (ia_norm.cu) that must hold for every row
// length, kept apart so that a host compiler can check it too.
#pragma once

#ifdef __CUDACC__
#define IA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define IA_HOST_DEVICE inline
#endif

namespace ia {

// Column, counted from the row's start, that a 16-byte copy of the vector of
// columns c .. c + V - 1 reads from.  Past the row's end (c >= D) the copy has
// size 0, but its source must be aligned to 16 bytes all the same: `mis`
// columns before the row's start lies a vector's boundary, and inside the
// tensor, as mis is the row's first element modulo V.
IA_HOST_DEVICE constexpr int copy_column(int c, int D, int mis) { return c < D ? c : -mis; }

// Bytes of it that are copied: up to the row's end, the rest of the 16 becomes zero.
IA_HOST_DEVICE constexpr int copy_bytes(int c, int D, int size) {
  return D - c <= 0 ? 0 : (D - c) * size >= 16 ? 16 : (D - c) * size;
}

}  // namespace ia
