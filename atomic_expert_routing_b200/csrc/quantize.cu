// Rows to 8-bit integers with one scale each:
//   scale = fp32(max|x| / 127),  q = the integer nearest to x / scale.
// A row is read once and kept in registers between its maximum and its
// integers, by a warp (rows of up to 2048 values, when there are many) or by
// a CTA of eight warps (up to 16384 values; a decode batch's few rows would
// leave most of the GPU idle with a warp each); longer rows are read twice.
//
// The quotient is rounded exactly, as if formed in infinite precision: the
// fp32 quotient can land on the middle between two integers when the true
// one lies beside it, so a quotient that comes within 10^-4 of a middle is
// checked against x with fused multiply-adds, whose sign is that of the
// exact difference.
#include "linear.cuh"

namespace omni {
namespace {

constexpr int kThreads = 256;
constexpr int kHeld = 8;  // vectors of 8 values a thread keeps

// |v|'s bits, monotone in |v|, with every NaN above infinity
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The integer nearest to x / s (ties to even), clamped to [-127, 127];
// |x| <= 191 s, s normal.  x * inv is off by less than 10^-4 from x / s.
__device__ __forceinline__ int nearest_quotient(float x, float s, float inv) {
  const float t = x * inv;
  float q = rintf(t);
  if (fabsf(t - q) > 0.4999f) {
    const float up = fmaf(-(q + 0.5f), s, x), down = fmaf(-(q - 0.5f), s, x);
    const bool odd = (static_cast<int>(q) & 1) != 0;
    if (up > 0.0f || (up == 0.0f && odd)) q += 1.0f;
    else if (down < 0.0f || (down == 0.0f && odd)) q -= 1.0f;
  }
  return static_cast<int>(fminf(fmaxf(q, -127.0f), 127.0f));
}

struct RowScale {
  float s, inv, lift;
  bool zero;  // every integer of the row is 0
};

// The scale of a row whose largest |value| has the bits m; stored by one thread.
__device__ __forceinline__ RowScale row_scale(uint32_t m, float* scale, bool store) {
  RowScale r;
  const bool fine = m < 0x7f800000u;
  const float s = fine ? __fdiv_rn(__uint_as_float(m), 127.0f) : __uint_as_float(0x7fc00000u);
  if (store) *scale = s;
  r.zero = !fine || s == 0.0f;
  // tiny rows are scaled up (exactly) so that the differences stay normal
  r.lift = s < 0x1p-80f ? 0x1p100f : 1.0f;
  r.s = s * r.lift;
  r.inv = __fdiv_rn(1.0f, r.s);
  return r;
}

__device__ __forceinline__ uint2 quantize8(const float* f, const RowScale& r) {
  uint32_t w[2] = {0u, 0u};
  if (!r.zero) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i >> 2] |= (static_cast<uint32_t>(nearest_quotient(f[i] * r.lift, r.s, r.inv)) & 0xffu)
                   << (8 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
}

// eight values as loaded
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
    f[4] = bf16lo(u.z); f[5] = bf16hi(u.z); f[6] = bf16lo(u.w); f[7] = bf16hi(u.w);
  }
};
template <> struct Eight<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) { load8(p, v); }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = v[i];
  }
};

// TPR threads per row (32 or the CTA); HELD: the row fits their registers
template <typename T, int TPR, bool HELD>
__global__ void __launch_bounds__(kThreads)
    k_quantize_rows(int64_t n, int width, const T* __restrict__ src, int8_t* __restrict__ q,
                    float* __restrict__ scale) {
  __shared__ uint32_t part[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  if (row >= n) return;
  const T* p = src + row * width;
  int8_t* o = q + row * width;
  Eight<T> held[HELD ? kHeld : 1];
  uint32_t m = 0;
  auto largest = [&](const Eight<T>& e) {
    float f[8];
    e.get(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(f[i]));
  };
  if constexpr (HELD) {
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if ((h * TPR + lane) * 8 < width) held[h].load(p + (h * TPR + lane) * 8);
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if ((h * TPR + lane) * 8 < width) largest(held[h]);
  } else {
    for (int c = lane * 8; c < width; c += TPR * 8) {
      held[0].load(p + c);
      largest(held[0]);
    }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, part[w]);
  }
  const RowScale r = row_scale(m, scale + row, lane == 0);
  float f[8];
  if constexpr (HELD) {
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      const int c = (h * TPR + lane) * 8;
      if (c < width) {
        held[h].get(f);
        *reinterpret_cast<uint2*>(o + c) = quantize8(f, r);
      }
    }
  } else {
    for (int c = lane * 8; c < width; c += TPR * 8) {
      held[0].load(p + c);
      held[0].get(f);
      *reinterpret_cast<uint2*>(o + c) = quantize8(f, r);
    }
  }
}

template <typename T>
cudaError_t launch(int64_t n, int width, const void* src, int8_t* q, float* scale,
                   cudaStream_t s) {
  // a warp per row once that gives every SM a few CTAs
  const bool warps = width <= 32 * 8 * kHeld && n >= 148 * 4 * (kThreads / 32);
  const bool held = width <= kThreads * 8 * kHeld;
  const unsigned grid = static_cast<unsigned>(warps ? (n + kThreads / 32 - 1) / (kThreads / 32) : n);
  const T* p = static_cast<const T*>(src);
  if (warps)
    OMNI_TRY(launch_k(k_quantize_rows<T, 32, true>, grid, kThreads, 0, s, n, width, p, q, scale));
  else if (held)
    OMNI_TRY(launch_k(k_quantize_rows<T, kThreads, true>, grid, kThreads, 0, s, n, width, p, q, scale));
  else
    OMNI_TRY(launch_k(k_quantize_rows<T, kThreads, false>, grid, kThreads, 0, s, n, width, p, q, scale));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_rows(int64_t n, int64_t width, bool f32, const void* src, int8_t* q,
                                 float* scale, cudaStream_t s) {
  const int w = static_cast<int>(width);
  return f32 ? launch<float>(n, w, src, q, scale, s)
             : launch<__nv_bfloat16>(n, w, src, q, scale, s);
}

}  // namespace omni
