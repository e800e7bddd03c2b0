// Rules of the grouped products that need no GPU: plain C++, for the kernels'
// host and device code and for any other compiler.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define OMNI_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define OMNI_HOST_DEVICE inline
#endif

namespace omni {

// How long a wait of dW's zeroing warp may last, in wait limits (a second
// each).  The warp waits only at the blocks it has to zero rows of, and takes
// no part in the tiles between them: a wait spans all that its CTA has summed
// since the one before, the blocks (64 rows) of every tile on the way and
// their ways out (4500 cycles, a few blocks' time).  2^18 blocks take a tenth
// of a second at 740 cycles each, two tenths where the loads bound them.
struct WaitSpan {
  uint32_t blocks = 0;
  OMNI_HOST_DEVICE void tile(int32_t n) { blocks += static_cast<uint32_t>(n) + 8; }
  OMNI_HOST_DEVICE uint32_t limits() const { return 1 + (blocks >> 18); }
  OMNI_HOST_DEVICE void waited() { blocks = 0; }
};

// Results leave through shared memory in chunks of 16 columns of 128.
constexpr int kOutCols = 16;

// How a warp's chunks of a tile of n columns leave.  They lie gap columns
// apart and go two at a time; those that go through shared memory take the
// barrier of the four warps of a half twice.
struct DrainRule {
  bool clipped;  // columns end with the matrix, not with a group: TMA cuts them
  bool pairs;    // two whole chunks may share the barriers of one
  int gap;
  OMNI_HOST_DEVICE bool whole(int left) const { return clipped || left >= kOutCols; }
  OMNI_HOST_DEVICE bool two(int left) const { return pairs && left >= gap + kOutCols; }
  // the barriers of a tile, for a warp whose first chunk is at column c
  OMNI_HOST_DEVICE int barriers(int n, int c) const {
    int b = 0;
    for (; c < n; c += 2 * gap) {
      if (two(n - c)) b += 2;
      else b += 2 * (whole(n - c) ? 1 : 0) + 2 * (c + gap < n && whole(n - c - gap) ? 1 : 0);
    }
    return b;
  }
};

}  // namespace omni
