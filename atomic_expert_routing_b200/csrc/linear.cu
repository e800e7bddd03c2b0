// The products of wide experts and of 8-bit integers: entry points
// (include/omnimoe.h) and kernels.
//
// Every product is D[j, i] = sum_k B[j, k] A[i, k] over the tiles of a group:
//   forward, 8-bit: j a product row, i an output channel, k an input channel;
//   dx:             j a product row, i an input channel, k an output channel;
//   dW:             j an output channel, i an input channel, k a product row.
// A CTA takes 64 x 64 tiles of all groups in turn, 16 of k at a time through
// shared memory, 4 x 4 sums per thread, in pieces of 512 products (a long sum's
// rounding then grows with the pieces, not with the products).
#include "linear.cuh"

namespace omni {
namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;
constexpr int kPiece = 512;  // products summed before they join the running sum

template <Product P>
__global__ void __launch_bounds__(kThreads) k_linear(const LinearArgs a) {
  extern __shared__ GroupTab tab[];
  __shared__ GroupScratch sh;
  __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
  __shared__ int32_t src_row[kTile];
  pdl_wait();
  constexpr bool kGradW = P == Product::kGradW;
  constexpr bool kGradX = P == Product::kGradX;
  const int I = kGradX || kGradW ? a.in : a.out;
  const int mt = (I + kTile - 1) / kTile;
  int32_t* status = blockIdx.x == 0 ? a.status : nullptr;
  build_groups(
      a.g,
      [&](int rows) {
        if (kGradW)
          return rows > 0 || !a.accumulate ? mt * ((a.out + kTile - 1) / kTile) : 0;
        return mt * ((rows + kTile - 1) / kTile);
      },
      tab, &sh, status);
  const int tiles = sh.total_tiles;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  int c = 0;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    while (c + 1 < sh.total_groups && tab[c + 1].begin <= t) ++c;
    const GroupTab gr = tab[c];
    const int local = t - gr.begin;
    const int i0 = (local % mt) * kTile, j0 = (local / mt) * kTile;
    const int J = kGradW ? a.out : gr.rows;
    const int K = kGradW ? gr.rows : kGradX ? a.out : a.in;
    const int64_t wbase = static_cast<int64_t>(gr.id) * a.out * a.in;
    auto token = [&](int r) -> int64_t {  // product row (of this group) -> row of x
      const int64_t m = gr.row0 + r;
      if (a.rows == nullptr) return m;
      const int32_t v = a.rows[m];
      if (v < 0 || v >= a.T) {
        raise_status(a.status, OMNI_DEV_BAD_INDEX);
        return 0;
      }
      return v;
    };
    if constexpr (!kGradW && !kGradX) {
      if (tid < kTile) src_row[tid] = j0 + tid < J ? static_cast<int32_t>(token(j0 + tid)) : 0;
      __syncthreads();
    }
    float acc[4][4] = {}, sum[4][4] = {};
    int isum[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += kStep) {
      for (int q = tid; q < kStep * kTile; q += kThreads) {
        // k fastest where it is contiguous in memory
        const int kk = kGradW ? q / kTile : q % kStep, u = kGradW ? q % kTile : q / kStep;
        const int k = k0 + kk, i = i0 + u, j = j0 + u;
        float va = 0.0f, vb = 0.0f;
        if (k < K) {
          if constexpr (P == Product::kForward) {
            if (i < I) va = to_float(static_cast<const __nv_bfloat16*>(a.W)[wbase + int64_t(i) * a.in + k]);
            if (j < J) vb = to_float(static_cast<const __nv_bfloat16*>(a.x)[int64_t(src_row[u]) * a.in + k]);
          } else if constexpr (P == Product::kInt8) {
            if (i < I) va = static_cast<const int8_t*>(a.W)[wbase + int64_t(i) * a.in + k];
            if (j < J) vb = static_cast<const int8_t*>(a.x)[int64_t(src_row[u]) * a.in + k];
          } else if constexpr (kGradX) {
            if (i < I) va = to_float(static_cast<const __nv_bfloat16*>(a.W)[wbase + int64_t(k) * a.in + i]);
            if (j < J) vb = to_float(static_cast<const __nv_bfloat16*>(a.dy)[int64_t(gr.row0 + j) * a.out + k]);
          } else {
            if (i < I) va = to_float(static_cast<const __nv_bfloat16*>(a.x)[token(k) * a.in + i]);
            if (j < J) vb = to_float(static_cast<const __nv_bfloat16*>(a.dy)[int64_t(gr.row0 + k) * a.out + j]);
          }
        }
        sa[kk][u] = va;
        sb[kk][u] = vb;
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < kStep; ++kk) {
        float fa[4], fb[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          fa[u] = sa[kk][tx + 16 * u];
          fb[u] = sb[kk][ty + 16 * u];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(fb[u], fa[v], acc[u][v]);
      }
      __syncthreads();
      if constexpr (P == Product::kInt8) {
        // a step's sum is exact in fp32 (16 * 127^2 < 2^24); the whole sum needs integers
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            isum[u][v] += static_cast<int>(acc[u][v]);
            acc[u][v] = 0.0f;
          }
      } else if ((k0 + kStep) % kPiece == 0 || k0 + kStep >= K) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            sum[u][v] += acc[u][v];
            acc[u][v] = 0.0f;
          }
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + ty + 16 * u;
      if (j >= J) continue;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int i = i0 + tx + 16 * v;
        if (i >= I) continue;
        if constexpr (kGradW) {
          float* o = static_cast<float*>(a.o) + wbase + int64_t(j) * a.in + i;
          *o = a.accumulate ? *o + sum[u][v] : sum[u][v];
        } else {
          float z = sum[u][v];
          if constexpr (P == Product::kInt8)
            z = static_cast<float>(isum[u][v]) * a.xs[src_row[ty + 16 * u]] *
                a.Ws[int64_t(gr.id) * a.out + i];
          if (a.silu) z = silu(z);
          const int64_t at = int64_t(gr.row0 + j) * I + i;
          if (a.out_f32) static_cast<float*>(a.o)[at] = z;
          else static_cast<__nv_bfloat16*>(a.o)[at] = __float2bfloat16_rn(z);
        }
      }
    }
    if constexpr (!kGradW && !kGradX) __syncthreads();  // src_row is the next tile's
  }
}

}  // namespace

cudaError_t launch_linear(Product p, const LinearArgs& a, cudaStream_t s) {
  auto go = [&](auto kernel) -> cudaError_t {
    const size_t smem = sizeof(GroupTab) * static_cast<size_t>(a.g.G);
    OMNI_TRY(launch_k(kernel, 148 * 4, kThreads, smem, s, a));
    return cudaGetLastError();
  };
  switch (p) {
    case Product::kForward: return go(k_linear<Product::kForward>);
    case Product::kGradX: return go(k_linear<Product::kGradX>);
    case Product::kGradW: return go(k_linear<Product::kGradW>);
    default: return go(k_linear<Product::kInt8>);
  }
}

namespace {

bool aligned(const void* p, uintptr_t a) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
bool aligned_or_null(const void* p, uintptr_t a) { return p == nullptr || aligned(p, a); }

// The host checks of include/omnimoe.h that every call makes.
int check_linear(const omni_linear_dims* d, const int32_t* group_off, const int32_t* ids,
                 const int32_t* n_groups, const int32_t* rows, int32_t* counts, int in_step,
                 LinearArgs* a) {
  if (d == nullptr) return OMNI_ERR_INVALID_ARG;
  if (d->M < 0 || d->T < 0 || (d->T < 1 && d->M > 0) || d->in < 1 || d->out < 1 || d->E < 1 ||
      d->G < 1 || d->G > d->E || (rows == nullptr && d->T != d->M) ||
      (d->out_dtype != OMNI_F32 && d->out_dtype != OMNI_BF16) ||
      (d->flags & ~OMNI_LINEAR_SILU) != 0)
    return OMNI_ERR_INVALID_ARG;
  const int64_t lim = int64_t(1) << 30;
  if (d->G > OMNI_MAX_GROUPS || d->in > 65536 || d->out > 65536 || d->in % in_step != 0 ||
      d->out % 8 != 0 || d->M >= lim || d->T >= lim || d->E >= lim)
    return OMNI_ERR_UNSUPPORTED;
  if (!aligned_or_null(group_off, 4) || !aligned_or_null(ids, 4) ||
      !aligned_or_null(n_groups, 4) || !aligned_or_null(rows, 4) || !aligned_or_null(counts, 4))
    return OMNI_ERR_INVALID_ARG;
  *a = LinearArgs{};
  a->g = Groups{d->M, static_cast<int32_t>(d->E), static_cast<int32_t>(d->G), group_off, ids,
                n_groups};
  a->T = d->T;
  a->in = static_cast<int32_t>(d->in);
  a->out = static_cast<int32_t>(d->out);
  a->out_f32 = d->out_dtype == OMNI_F32;
  a->silu = (d->flags & OMNI_LINEAR_SILU) != 0;
  a->rows = rows;
  a->status = counts != nullptr ? counts + 2 : nullptr;
  return OMNI_OK;
}

}  // namespace
}  // namespace omni

using omni::aligned;
using omni::aligned_or_null;
using omni::cuda_status;
using omni::LinearArgs;
using omni::Product;

extern "C" {

int omni_grouped_linear(const omni_linear_dims* dims, const void* x, const void* W,
                        const int32_t* group_off, const int32_t* ids, const int32_t* n_groups,
                        const int32_t* rows, void* y, int32_t* counts, void* stream) {
  omni::CallRange range("omni_grouped_linear");
  LinearArgs a;
  const int rc = omni::check_linear(dims, group_off, ids, n_groups, rows, counts, 8, &a);
  if (rc != OMNI_OK) return rc;
  if (dims->M == 0) return OMNI_OK;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(y, 16) || group_off == nullptr)
    return OMNI_ERR_INVALID_ARG;
  a.x = x;
  a.W = W;
  a.o = y;
  return cuda_status(omni::launch_linear(Product::kForward, a, static_cast<cudaStream_t>(stream)));
}

int omni_grouped_linear_backward(const omni_linear_dims* dims, const void* x, const void* W,
                                 const void* dy, const int32_t* group_off, const int32_t* ids,
                                 const int32_t* n_groups, const int32_t* rows, void* dx,
                                 float* dW, int accumulate, int32_t* counts, void* stream) {
  omni::CallRange range("omni_grouped_linear_backward");
  LinearArgs a;
  const int rc = omni::check_linear(dims, group_off, ids, n_groups, rows, counts, 8, &a);
  if (rc != OMNI_OK) return rc;
  if (a.silu) return OMNI_ERR_UNSUPPORTED;
  if (group_off == nullptr || (dx == nullptr && dW == nullptr) || !aligned_or_null(dx, 16) ||
      !aligned_or_null(dW, 16))
    return OMNI_ERR_INVALID_ARG;
  if (dims->M > 0 && (!aligned(dy, 16) || (dx != nullptr && !aligned(W, 16)) ||
                      (dW != nullptr && !aligned(x, 16))))
    return OMNI_ERR_INVALID_ARG;
  a.x = x;
  a.W = W;
  a.dy = dy;
  a.accumulate = accumulate != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dx != nullptr && dims->M > 0) {
    a.o = dx;
    const int e = cuda_status(omni::launch_linear(Product::kGradX, a, s));
    if (e != OMNI_OK) return e;
  }
  if (dW != nullptr && (dims->M > 0 || !a.accumulate)) {
    a.o = dW;
    return cuda_status(omni::launch_linear(Product::kGradW, a, s));
  }
  return OMNI_OK;
}

int omni_quantize_rows(int64_t n, int64_t width, int dtype, const void* src, int8_t* q,
                       float* scale, void* stream) {
  omni::CallRange range("omni_quantize_rows");
  if (n < 0 || width < 1 || (dtype != OMNI_F32 && dtype != OMNI_BF16)) return OMNI_ERR_INVALID_ARG;
  if (width % 16 != 0 || width > 65536 || n >= (int64_t(1) << 30)) return OMNI_ERR_UNSUPPORTED;
  if (n == 0) return OMNI_OK;
  if (!aligned(src, 16) || !aligned(q, 16) || !aligned(scale, 4)) return OMNI_ERR_INVALID_ARG;
  return cuda_status(omni::launch_quantize_rows(n, width, dtype == OMNI_F32, src, q, scale,
                                                static_cast<cudaStream_t>(stream)));
}

int omni_quantized_linear(const omni_linear_dims* dims, const int8_t* xq, const float* xs,
                          const int8_t* Wq, const float* Ws, const int32_t* group_off,
                          const int32_t* ids, const int32_t* n_groups, const int32_t* rows,
                          void* y, int32_t* counts, void* stream) {
  omni::CallRange range("omni_quantized_linear");
  LinearArgs a;
  const int rc = omni::check_linear(dims, group_off, ids, n_groups, rows, counts, 16, &a);
  if (rc != OMNI_OK) return rc;
  if (group_off == nullptr &&
      (dims->E != 1 || ids != nullptr || n_groups != nullptr))
    return OMNI_ERR_INVALID_ARG;
  if (dims->M == 0) return OMNI_OK;
  if (!aligned(xq, 16) || !aligned(Wq, 16) || !aligned(y, 16) || !aligned(xs, 4) ||
      !aligned(Ws, 4))
    return OMNI_ERR_INVALID_ARG;
  a.x = xq;
  a.W = Wq;
  a.xs = xs;
  a.Ws = Ws;
  a.o = y;
  return cuda_status(omni::launch_linear(Product::kInt8, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
