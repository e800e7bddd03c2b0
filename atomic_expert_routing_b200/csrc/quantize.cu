// Rows to 8-bit integers with one scale each:
//   scale = fp32(max|x| / 127),  q = the integer nearest to x / scale.
// A row is read once and kept in registers between its maximum and its
// integers, by two warps (rows of up to 2048 values, when there are many) or
// by a CTA of eight (up to 16384 values; a decode batch's few rows would leave
// most of the GPU idle with a warp each); longer rows are read twice.
//
// 16384 x 2048 in fp32 take 27 us, at the memory's rate (6.2 TB/s); in bf16,
// half the bytes read, 28 (15 at the copy rate; 2.4 TB/s and 54% of the issue
// slots, so neither of the two bounds it, and what does was not found); 64
// rows 2.7.
//
// The quotient is rounded exactly, as if formed in infinite precision: the
// fp32 quotient can land on the middle between two integers when the true
// one lies beside it, so quotients within 3e-5 of a middle are checked
// against x with fused multiply-adds, whose sign is that of the exact
// difference.
#include "linear.cuh"

namespace omni {
namespace {

constexpr int kThreads = 256;

// |v|'s bits, monotone in |v|, with every NaN above infinity
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The integer nearest to x / s (ties to even), clamped to [-127, 127];
// |x| <= 191 s, s normal.
__device__ __forceinline__ int nearest_quotient(float x, float s, float inv) {
  float q = rintf(x * inv);  // at most one off
  const float up = fmaf(-(q + 0.5f), s, x), down = fmaf(-(q - 0.5f), s, x);
  const bool odd = (static_cast<int>(q) & 1) != 0;
  if (up > 0.0f || (up == 0.0f && odd)) q += 1.0f;
  else if (down < 0.0f || (down == 0.0f && odd)) q -= 1.0f;
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
  asm("rcp.approx.f32 %0, %1;" : "=f"(r.inv) : "f"(r.s));  // within 2^-23
  return r;
}

// eight values as loaded
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = *reinterpret_cast<const uint4*>(p);
  }
  // the largest |value|'s bits as a float's; m is of the same kind
  __device__ __forceinline__ uint32_t largest(uint32_t m) const {
    const uint32_t k = 0x7fff7fffu;
    const uint32_t w = __vmaxu2(__vmaxu2(u.x & k, u.y & k), __vmaxu2(u.z & k, u.w & k));
    return max(m, max(w << 16, w & 0xffff0000u));
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
    f[4] = bf16lo(u.z); f[5] = bf16hi(u.z); f[6] = bf16lo(u.w); f[7] = bf16hi(u.w);
  }
};
template <> struct Eight<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) { load8(p, v); }
  __device__ __forceinline__ uint32_t largest(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    return m;
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = v[i];
  }
};

constexpr float kRound = 12582912.0f;  // 1.5 * 2^23
constexpr float kNear = 0.49997f;

__device__ __forceinline__ uint2 pack8(const uint32_t* q) {
  return make_uint2(
      __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410),
      __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410));
}

// The same with every doubtful value done exactly.  One copy of it, not one per
// vector a thread holds: inlined, the kernel waited on its instructions (36 us
// for 16384 x 2048 bf16).
template <typename T>
__device__ __noinline__ uint2 quantize8_exact(Eight<T> e, float s, float inv, float lift) {
  float f[8];
  e.get(f);
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = f[i] * inv;
    q[i] = __float_as_uint(__fadd_rn(t, kRound));
    if (lift != 1.0f || fabsf(t - rintf(t)) > kNear)
      q[i] = static_cast<uint32_t>(nearest_quotient(f[i] * lift, s, inv));
  }
  return pack8(q);
}

// Adding 1.5 * 2^23 rounds a small value to the nearest integer (ties to even)
// and leaves the integer in the low bits.  x * inv, a value up to 127.5, is off
// by at most 127.5 * (2^-23 + 2^-24) < 2.3e-5 from x / s, so a rounding that is
// 3e-5 or more from the middle stands.  Nearer ones (among
// bf16 values, all those of half the largest: some of a row of 2048) and
// those of a scaled-up row (whose quotients may pass 127) are done exactly.
template <typename T>
__device__ __forceinline__ uint2 quantize8(const Eight<T>& e, const RowScale& r) {
  float f[8];
  e.get(f);
  uint32_t q[8];
  bool near = r.lift != 1.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = f[i] * r.inv;
    const float m = __fadd_rn(t, kRound);
    near |= fabsf(t - __fsub_rn(m, kRound)) > kNear;
    q[i] = __float_as_uint(m);
  }
  if (r.zero) return make_uint2(0u, 0u);
  return near ? quantize8_exact(e, r.s, r.inv, r.lift) : pack8(q);
}

// TPR threads per row, HELD vectors of 8 values of it in each thread's
// registers (0: the row does not fit)
template <typename T, int TPR, int HELD>
__global__ void __launch_bounds__(kThreads)
    k_quantize_rows(int64_t n, int width, const T* __restrict__ src, int8_t* __restrict__ q,
                    float* __restrict__ scale) {
  __shared__ uint32_t part[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  const bool there = row < n;
  if (!there) width = 0;
  const T* p = src + row * width;
  int8_t* o = q + row * width;
  Eight<T> held[HELD > 0 ? HELD : 1];
  uint32_t m = 0;
  if constexpr (HELD > 0) {
#pragma unroll
    for (int h = 0; h < HELD; ++h)
      if ((h * TPR + lane) * 8 < width) held[h].load(p + (h * TPR + lane) * 8);
#pragma unroll
    for (int h = 0; h < HELD; ++h)
      if ((h * TPR + lane) * 8 < width) m = held[h].largest(m);
  } else {
    for (int c = lane * 8; c < width; c += TPR * 8) {
      held[0].load(p + c);
      m = held[0].largest(m);
    }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < TPR / 32; ++w) m = max(m, part[threadIdx.x / TPR * (TPR / 32) + w]);
  const RowScale r = row_scale(m, scale + row, there && lane == 0);
  if constexpr (HELD > 0) {
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      const int c = (h * TPR + lane) * 8;
      if (c < width) *reinterpret_cast<uint2*>(o + c) = quantize8(held[h], r);
    }
  } else {
    for (int c = lane * 8; c < width; c += TPR * 8) {
      held[0].load(p + c);
      *reinterpret_cast<uint2*>(o + c) = quantize8(held[0], r);
    }
  }
}

template <typename T>
cudaError_t launch(int64_t n, int width, const void* src, int8_t* q, float* scale,
                   cudaStream_t s) {
  const T* p = static_cast<const T*>(src);
  auto go = [&](auto kernel, int rows_per_cta) -> cudaError_t {
    const unsigned grid = static_cast<unsigned>((n + rows_per_cta - 1) / rows_per_cta);
    return launch_k(kernel, grid, kThreads, 0, s, n, width, p, q, scale);
  };
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // two warps per row once that gives every SM a few CTAs
  if (width <= 64 * 8 * 4 && n >= int64_t(4) * sms * (kThreads / 64))
    OMNI_TRY(go(k_quantize_rows<T, 64, 4>, kThreads / 64));
  else if (width <= kThreads * 8 * 8)
    OMNI_TRY(go(k_quantize_rows<T, kThreads, 8>, 1));
  else
    OMNI_TRY(go(k_quantize_rows<T, kThreads, 0>, 1));
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
