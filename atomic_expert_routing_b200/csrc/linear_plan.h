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

}  // namespace omni
