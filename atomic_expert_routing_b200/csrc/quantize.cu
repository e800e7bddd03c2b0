// Rows to 8-bit integers with one scale each:
//   scale = fp32(max|x| / 127),  q = the integer nearest to x / scale.
// One warp per row: the row's maximum in a first pass, its integers in a
// second (the row is in L1 or L2 by then).
//
// The quotient is rounded exactly, as if formed in infinite precision: the
// fp32 quotient can land on the middle between two integers when the true
// one lies beside it, so the candidate is checked against x with fused
// multiply-adds, whose sign is that of the exact difference.
#include "linear.cuh"

namespace omni {
namespace {

constexpr int kWarps = 8;

// |v|'s bits, monotone in |v|, with every NaN above infinity
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The integer nearest to x / s (ties to even), |x| <= 127.5 s, s > 0 normal.
__device__ __forceinline__ int nearest_quotient(float x, float s, float inv) {
  float q = rintf(x * inv);  // at most one off
  const float up = fmaf(-(q + 0.5f), s, x), down = fmaf(-(q - 0.5f), s, x);
  const bool odd = (static_cast<int>(q) & 1) != 0;
  if (up > 0.0f || (up == 0.0f && odd)) q += 1.0f;
  else if (down < 0.0f || (down == 0.0f && odd)) q -= 1.0f;
  return static_cast<int>(fminf(fmaxf(q, -127.0f), 127.0f));
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
    k_quantize_rows(int64_t n, int width, const T* __restrict__ src, int8_t* __restrict__ q,
                    float* __restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= n) return;
  const T* p = src + row * width;
  uint32_t m = 0;
  for (int c = lane * 8; c < width; c += 256) {
    float f[8];
    load8(p + c, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(f[i]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  const bool fine = m < 0x7f800000u;
  float s = fine ? __fdiv_rn(__uint_as_float(m), 127.0f) : __uint_as_float(0x7fc00000u);
  if (lane == 0) scale[row] = s;
  const bool zero = !fine || s == 0.0f;
  // tiny rows are scaled up (exactly) so that the differences stay normal
  const float lift = s < 0x1p-80f ? 0x1p100f : 1.0f;
  s *= lift;
  const float inv = __fdiv_rn(1.0f, s);
  for (int c = lane * 8; c < width; c += 256) {
    uint32_t w[2] = {0u, 0u};
    if (!zero) {
      float f[8];
      load8(p + c, f);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i >> 2] |= (static_cast<uint32_t>(nearest_quotient(f[i] * lift, s, inv)) & 0xffu)
                     << (8 * (i & 3));
    }
    *reinterpret_cast<uint2*>(q + row * width + c) = make_uint2(w[0], w[1]);
  }
}

}  // namespace

cudaError_t launch_quantize_rows(int64_t n, int64_t width, bool f32, const void* src, int8_t* q,
                                 float* scale, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((n + kWarps - 1) / kWarps);
  const int w = static_cast<int>(width);
  if (f32)
    OMNI_TRY(launch_k(k_quantize_rows<float>, grid, kWarps * 32, 0, s, n, w,
                      static_cast<const float*>(src), q, scale));
  else
    OMNI_TRY(launch_k(k_quantize_rows<__nv_bfloat16>, grid, kWarps * 32, 0, s, n, w,
                      static_cast<const __nv_bfloat16*>(src), q, scale));
  return cudaGetLastError();
}

}  // namespace omni
