// The products of wide experts and of 8-bit integers: the entry points of
// include/omnimoe.h and their host checks (kernels: linear_tc.cu, quantize.cu).
#include "linear.cuh"

namespace omni {
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
  const bool form_dx = dx != nullptr && dims->M > 0;
  const bool form_dW = dW != nullptr && (dims->M > 0 || !a.accumulate);
  if (form_dx) {
    LinearArgs b = a;
    b.o = dx;
    b.leads = form_dW;
    const int e = cuda_status(omni::launch_linear(Product::kGradX, b, s));
    if (e != OMNI_OK) return e;
  }
  if (form_dW) {
    a.o = dW;
    a.follows = form_dx;
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
