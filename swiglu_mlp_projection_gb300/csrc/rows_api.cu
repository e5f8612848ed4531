// C ABI of the row operators: the RMS norm and its gradient, rows sorted by
// expert and back.  See include/swiglu.h for the contract of each entry point.
#include "api_checks.h"
#include "grouped.h"
#include "internal.h"
#include "rows.h"
#include "swiglu.h"

namespace swg {
namespace {

size_t elem_bytes(int dtype) {
  return dtype == SWIGLU_F32 ? 4 : dtype == SWIGLU_BF16 ? 2 : 1;
}

int check_float(int dtype) {
  if (dtype != SWIGLU_F32 && dtype != SWIGLU_BF16)
    return api_fail(SWIGLU_ERR_INVALID_ARG, "unknown dtype");
  return SWIGLU_OK;
}

int check_norm(int64_t M, int64_t d, float eps, int dtype, int weight_dtype) {
  int v = check_float(dtype);
  if (v == SWIGLU_OK) v = check_float(weight_dtype);
  if (v != SWIGLU_OK) return v;
  if (M < 0 || d < 0) return api_fail(SWIGLU_ERR_INVALID_ARG, "negative size");
  if (!(eps > 0.f) || eps > 3.0e38f)
    return api_fail(SWIGLU_ERR_INVALID_ARG, "eps must be positive and finite");
  // (1024 threads hold 32 elements each; a row that starts inside 16 bytes has
  // up to two pieces more)
  if (d > kMaxNormWidth - (d % (dtype == SWIGLU_F32 ? 4 : 8) ? 16 : 0))
    return api_fail(SWIGLU_ERR_UNSUPPORTED, "a row of more than 32768 elements");
  if (M > (int64_t)1 << 30) return api_fail(SWIGLU_ERR_UNSUPPORTED, "a size exceeds 2^30");
  return SWIGLU_OK;
}

int check_pairs(int64_t T, int64_t k, int64_t d) {
  if (T < 0 || k < 0 || d < 0) return api_fail(SWIGLU_ERR_INVALID_ARG, "negative size");
  if (k > kMaxTopK) return api_fail(SWIGLU_ERR_UNSUPPORTED, "more than 32 choices per token");
  if (T > (int64_t)1 << 30 || T * k > (int64_t)1 << 30)
    return api_fail(SWIGLU_ERR_UNSUPPORTED, "a size exceeds 2^30");
  if (d > (int64_t)1 << 28)   // (a row's bytes are counted in 32 bits)
    return api_fail(SWIGLU_ERR_UNSUPPORTED, "a row of more than 2^28 elements");
  return SWIGLU_OK;
}

int check_experts(int64_t E) {
  if (E < 1) return api_fail(SWIGLU_ERR_INVALID_ARG, "no experts");
  if (E > kMaxExperts) return api_fail(SWIGLU_ERR_UNSUPPORTED, "more than 1024 experts");
  return SWIGLU_OK;
}

int finish(cudaError_t e) {
  if (e != cudaSuccess) return api_cuda_fail(e, "kernel launch");
  api_clear_error();
  return SWIGLU_OK;
}

// The norm's forward call; scales: null, or the 8-bit form.
int rms_norm(const void* x, const void* residual, const void* weight, void* out, float* scales,
             void* sum, int64_t M, int64_t d, float eps, int dtype, int weight_dtype, bool fp8,
             cudaStream_t st) {
  int v = check_norm(M, d, eps, dtype, weight_dtype);
  if (v != SWIGLU_OK) return v;
  if ((residual != nullptr) != (sum != nullptr) && M > 0 && d > 0)
    return api_fail(SWIGLU_ERR_INVALID_ARG, "residual and sum go together");
  const size_t n = (size_t)M * d, e = elem_bytes(dtype);
  const Span in[] = {{"x", x, n * e}, {"residual", residual, residual ? n * e : 0},
                     {"weight", weight, (size_t)d * elem_bytes(weight_dtype)}};
  const Span out_s = {fp8 ? "codes" : "y", out, n * (fp8 ? 1 : e)};
  const Span sum_s = {"sum", sum, sum ? n * e : 0};
  const Span scale_s = {"scales", scales, fp8 ? (size_t)M * 4 : 0, 4};
  if ((v = check_spans(in, 3)) != SWIGLU_OK || (v = check_spans(&out_s, 1)) != SWIGLU_OK ||
      (v = check_spans(&sum_s, 1)) != SWIGLU_OK || (v = check_spans(&scale_s, 1)) != SWIGLU_OK)
    return v;
  // y and sum may each be x or residual themselves: a thread reads what it overwrites
  if ((v = fp8 ? check_apart(out_s, in, 3) : check_apart_or_same(out_s, in, 2)) != SWIGLU_OK ||
      (v = check_apart(out_s, in + 2, 1)) != SWIGLU_OK ||
      (v = check_apart_or_same(sum_s, in, 2)) != SWIGLU_OK ||
      (v = check_apart(sum_s, in + 2, 1)) != SWIGLU_OK ||
      (v = check_apart(sum_s, &out_s, 1)) != SWIGLU_OK ||
      (v = check_apart(scale_s, in, 3)) != SWIGLU_OK ||
      (v = check_apart(scale_s, &out_s, 1)) != SWIGLU_OK ||
      (v = check_apart(scale_s, &sum_s, 1)) != SWIGLU_OK)
    return v;
  int dev, num_sms;
  if ((v = api_current_device(&dev, &num_sms)) != SWIGLU_OK) return v;
  if (fp8 && d == 0 && M > 0) {   // rows of nothing: scale 0
    const cudaError_t err = cudaMemsetAsync(scales, 0, (size_t)M * 4, st);
    if (err != cudaSuccess) return api_cuda_fail(err, "cudaMemsetAsync(scales)");
  }
  return finish(launch_rms_norm(NormCall{x, residual, weight, out, fp8 ? scales : nullptr, sum, M,
                                         d, eps, dtype == SWIGLU_F32, weight_dtype == SWIGLU_F32},
                                num_sms, st));
}

}  // namespace
}  // namespace swg

using namespace swg;

extern "C" {

int swiglu_rms_norm(const void* x, const void* residual, const void* weight, void* y, void* sum,
                    int64_t M, int64_t d, float eps, int dtype, int weight_dtype, void* stream) {
  return rms_norm(x, residual, weight, y, nullptr, sum, M, d, eps, dtype, weight_dtype, false,
                  (cudaStream_t)stream);
}

int swiglu_rms_norm_fp8(const void* x, const void* residual, const void* weight, void* codes,
                        float* scales, void* sum, int64_t M, int64_t d, float eps, int dtype,
                        int weight_dtype, void* stream) {
  return rms_norm(x, residual, weight, codes, scales, sum, M, d, eps, dtype, weight_dtype, true,
                  (cudaStream_t)stream);
}

size_t swiglu_rms_norm_backward_workspace_bytes(int64_t M, int64_t d, int dtype) {
  if (check_norm(M, d, 1.f, dtype, dtype) != SWIGLU_OK) return 0;
  int dev, num_sms;
  if (api_current_device(&dev, &num_sms) != SWIGLU_OK) return 0;
  api_clear_error();
  return round256(rms_norm_backward_bytes(M, d, dtype == SWIGLU_F32, num_sms));
}

int swiglu_rms_norm_backward(const void* dy, const void* s, const void* weight, const void* ds,
                             void* dx, void* dweight, int64_t M, int64_t d, float eps, int dtype,
                             int weight_dtype, void* workspace, size_t workspace_bytes,
                             void* stream) {
  int v = check_norm(M, d, eps, dtype, weight_dtype);
  if (v != SWIGLU_OK) return v;
  const size_t n = (size_t)M * d * elem_bytes(dtype), nw = (size_t)d * elem_bytes(weight_dtype);
  const Span in[] = {{"dy", dy, n}, {"s", s, n}, {"ds", ds, ds ? n : 0}, {"weight", weight, nw},
                     {"workspace", workspace, workspace ? workspace_bytes : 0}};
  const Span out[] = {{"dx", dx, n}, {"dweight", dweight, nw}};
  if ((v = check_spans(in, 4)) != SWIGLU_OK || (v = check_spans(out, 2)) != SWIGLU_OK) return v;
  // dx may be dy, s or ds itself: a thread reads what it overwrites
  if ((v = check_apart_or_same(out[0], in, 3)) != SWIGLU_OK ||
      (v = check_apart(out[0], in + 3, 2)) != SWIGLU_OK ||
      (v = check_apart(out[1], in, 5)) != SWIGLU_OK ||
      (v = check_apart(out[1], out, 1)) != SWIGLU_OK ||
      // (CTAs write their partial sums while others read)
      (v = check_apart(in[4], in, 4)) != SWIGLU_OK)
    return v;
  int dev, num_sms;
  if ((v = api_current_device(&dev, &num_sms)) != SWIGLU_OK) return v;
  if (d == 0) {
    api_clear_error();
    return SWIGLU_OK;
  }
  const cudaStream_t st = (cudaStream_t)stream;
  const std::unique_lock<std::mutex> lock =
      workspace ? std::unique_lock<std::mutex>() : api_lock_enqueue(dev, st);
  Workspace ws;
  const size_t body = round256(rms_norm_backward_bytes(M, d, dtype == SWIGLU_F32, num_sms));
  if (body && (v = api_take_workspace(dev, st, workspace, workspace_bytes, 0, body, &ws)) != SWIGLU_OK)
    return v;
  cudaError_t e = launch_rms_norm_backward(
      NormBackwardCall{dy, s, weight, ds, dx, dweight, M, d, eps, dtype == SWIGLU_F32,
                       weight_dtype == SWIGLU_F32},
      (float*)ws.body, num_sms, st);
  if (ws.pooled) {
    const cudaError_t ef = cudaFreeAsync(ws.pooled, st);
    if (e == cudaSuccess) e = ef;
  }
  return finish(e);
}

int swiglu_permute(const void* x, const float* scales, const int32_t* position,
                   const int32_t* offsets, void* out, float* out_scales, int64_t T, int64_t k,
                   int64_t E, int64_t d, int dtype, void* stream) {
  int v = check_pairs(T, k, d);
  if (v != SWIGLU_OK) return v;
  if ((v = check_experts(E)) != SWIGLU_OK) return v;
  const bool e4m3 = dtype == SWIGLU_E4M3;
  if (!e4m3 && (v = check_float(dtype)) != SWIGLU_OK) return v;
  if (!e4m3 && (scales || out_scales))
    return api_fail(SWIGLU_ERR_INVALID_ARG, "scales go with e4m3 rows only");
  const size_t e = elem_bytes(dtype), rows = (size_t)T * k;
  const Span in[] = {{"x", x, (size_t)T * d * e}, {"scales", scales, e4m3 ? (size_t)T * 4 : 0, 4},
                     {"position", position, rows * 4, 4},
                     {"offsets", offsets, (size_t)(E + 1) * 4, 4}};
  const Span out_s[] = {{"out", out, rows * d * e},
                        {"out_scales", out_scales, e4m3 ? rows * 4 : 0, 4}};
  if ((v = check_spans(in, 4)) != SWIGLU_OK || (v = check_spans(out_s, 2)) != SWIGLU_OK ||
      (v = check_apart(out_s[0], in, 4)) != SWIGLU_OK ||
      (v = check_apart(out_s[1], in, 4)) != SWIGLU_OK ||
      (v = check_apart(out_s[1], out_s, 1)) != SWIGLU_OK)
    return v;
  int dev, num_sms;
  if ((v = api_current_device(&dev, &num_sms)) != SWIGLU_OK) return v;
  return finish(launch_permute(PermuteCall{x, e4m3 ? scales : nullptr, position, offsets, out,
                                           out_scales, T, k, E, d, (int)e},
                               num_sms, (cudaStream_t)stream));
}

int swiglu_unpermute(const void* z, const int32_t* position, const float* weights,
                     const void* residual, void* y, int64_t T, int64_t k, int64_t d, int dtype,
                     void* stream) {
  int v = check_pairs(T, k, d);
  if (v != SWIGLU_OK) return v;
  if ((v = check_float(dtype)) != SWIGLU_OK) return v;
  const size_t e = elem_bytes(dtype), rows = (size_t)T * k;
  const Span in[] = {{"z", z, rows * d * e}, {"position", position, rows * 4, 4},
                     {"weights", weights, weights ? rows * 4 : 0, 4},
                     {"residual", residual, residual ? (size_t)T * d * e : 0}};
  const Span out = {"y", y, (size_t)T * d * e};
  if ((v = check_spans(in, 4)) != SWIGLU_OK || (v = check_spans(&out, 1)) != SWIGLU_OK ||
      (v = check_apart(out, in, 3)) != SWIGLU_OK ||
      (v = check_apart_or_same(out, in + 3, 1)) != SWIGLU_OK)
    return v;
  int dev, num_sms;
  if ((v = api_current_device(&dev, &num_sms)) != SWIGLU_OK) return v;
  return finish(launch_unpermute(UnpermuteCall{z, position, weights, residual, y, T, k, d,
                                               dtype == SWIGLU_F32},
                                 num_sms, (cudaStream_t)stream));
}

int swiglu_unpermute_backward(const void* dy, const void* z, const int32_t* position,
                              const int32_t* offsets, const float* weights, void* dz,
                              float* dweights, int64_t T, int64_t k, int64_t E, int64_t d,
                              int dtype, void* stream) {
  int v = check_pairs(T, k, d);
  if (v != SWIGLU_OK) return v;
  if ((v = check_experts(E)) != SWIGLU_OK) return v;
  if ((v = check_float(dtype)) != SWIGLU_OK) return v;
  const size_t e = elem_bytes(dtype), rows = (size_t)T * k;
  const Span in[] = {{"dy", dy, (size_t)T * d * e}, {"z", z, rows * d * e},
                     {"position", position, rows * 4, 4},
                     {"offsets", offsets, (size_t)(E + 1) * 4, 4},
                     {"weights", weights, rows * 4, 4}};
  const Span out[] = {{"dz", dz, rows * d * e}, {"dweights", dweights, rows * 4, 4}};
  if ((v = check_spans(in, 5)) != SWIGLU_OK || (v = check_spans(out, 2)) != SWIGLU_OK ||
      (v = check_apart(out[0], in, 5)) != SWIGLU_OK ||
      (v = check_apart(out[1], in, 5)) != SWIGLU_OK || (v = check_apart(out[1], out, 1)) != SWIGLU_OK)
    return v;
  int dev, num_sms;
  if ((v = api_current_device(&dev, &num_sms)) != SWIGLU_OK) return v;
  return finish(launch_unpermute_backward(
      UnpermuteBackwardCall{dy, z, position, offsets, weights, dz, dweights, T, k, E, d,
                            dtype == SWIGLU_F32},
      num_sms, (cudaStream_t)stream));
}

}  // extern "C"
