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

constexpr int kBM = 128;  // i per CTA

// Which tiles a product takes.  Measured on 16384 rows, 2048 to 4096 wide, a
// k-block of 128 bytes costs a slot (an SM, or a pair) about
//   32 wide 305 cycles, 64: 374, 128: 540, pairs of 256: 740;
// a tile with fewer columns costs in proportion, down to what loading its A
// and turning a stage over cost.  The estimate is the rounds the slots need
// times the cost of the tiles; the cheapest is taken.  A
// batch with many rows per group ends up with pairs of 256 (1550 TFLOP/s
// against 1090 at 128), a decode batch with 32, and a product with few tiles
// with narrower ones than its rows would fill, so that more SMs have one
// (300 rows, 2048 to 512: 40 tiles of 32 in 305 cycles a block against 4
// pairs in 740).
struct Shape {
  int ctas, bn, cycles, least;
};
constexpr Shape kShapes[] = {
    {1, 32, 305, 305}, {1, 64, 374, 330}, {1, 128, 540, 420}, {2, 256, 740, 480}};

inline int64_t round_cost(const Shape& sh, int64_t I, int64_t rows, int64_t live, int sms) {
  const int64_t each = (rows + live - 1) / live;
  // the tiles of one group exactly; of many, half a tile more for each group's end
  int64_t per = live == 1 ? (rows + sh.bn - 1) / sh.bn : (2 * rows / sh.bn + live) / 2;
  if (per < live) per = live;
  // groups are uneven: where the mean one fills half a tile, some fill all of it
  int64_t cost = sh.cycles;
  if (2 * each < sh.bn) {
    cost = sh.cycles * each / sh.bn;
    if (cost < sh.least) cost = sh.least;
  }
  const int64_t tiles = per * ((I + kBM * sh.ctas - 1) / (kBM * sh.ctas)), slots = sms / sh.ctas;
  return (tiles + slots - 1) / slots * cost;
}

// The place in kShapes of the tiles for I columns of results and `rows` rows in G groups.
inline int pick_shape(int64_t I, int64_t rows, int64_t G, int sms) {
  const int64_t live = G < rows ? G : rows;
  int best = 0;
  int64_t least = 0;
  for (int q = 0; q < 4; ++q) {
    const int64_t c = round_cost(kShapes[q], I, rows, live, sms);
    if (q == 0 || c < least) {
      best = q;
      least = c;
    }
  }
  return best;
}

// dW: pairs of 256 x 256, or single CTAs of 128 x 128 where those leave a
// third or more of a pair's columns idle or give the SMs fewer rounds.  A tile
// costs its products (740 or 540 cycles per 64 rows) or its way out (4500 or
// 2300), whichever is more.
inline bool grad_w_pairs(int64_t in, int64_t out, int64_t rows, int64_t G, int sms) {
  const int64_t blocks = (rows / G + 63) / 64;
  auto cost = [&](int64_t m, int64_t n, int64_t slots, int64_t block, int64_t way_out) {
    const int64_t tiles = (in + m - 1) / m * ((out + n - 1) / n) * G;
    return (tiles + slots - 1) / slots * (blocks * block > way_out ? blocks * block : way_out);
  };
  return cost(256, 256, sms / 2, 740, 4500) <= cost(128, 128, sms, 540, 2300);
}

}  // namespace omni
