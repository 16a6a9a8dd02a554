// Host side of dropout and of the RMS norm with the residual's addition:
// argument checks, workspace size and launches behind the C ABI declared in
// include/ckl.h.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/ckl.h"
#include "ckl_host.hpp"
#include "ckl_ops.hpp"

using namespace ckl::host;

namespace {

constexpr int64_t kMaxElements = (int64_t)1 << 36;  // (2^31 threads; a launch takes fewer than 2^32)

ckl_status drop_args(double p, uint64_t seed, uint64_t offset, const int64_t* state, ckl::DropArgs* a) {
  if (!(p >= 0.0 && p <= 1.0)) return fail(CKL_ERR_INVALID_ARG, "p must be from 0 to 1");
  if ((uintptr_t)state & 7u) return fail(CKL_ERR_INVALID_ARG, "state must be 8-byte aligned");
  a->threshold = (uint32_t)std::nearbyint(p * 65536.0);
  a->scale = a->threshold < 65536 ? 65536.f / (float)(65536 - a->threshold) : 0.f;
  a->seed = seed;
  a->offset = offset;
  a->state = state;
  return CKL_OK;
}

ckl_status check_norm(int64_t T, int64_t d, int32_t x_dtype, int32_t r_dtype, int32_t weight_dtype) {
  ckl_status s = check_rows(T);
  if (s == CKL_OK) s = check_hidden(d);
  if (s != CKL_OK) return s;
  if (!dtype_ok(x_dtype) || !dtype_ok(r_dtype) || !dtype_ok(weight_dtype))
    return fail(CKL_ERR_INVALID_ARG, "dtype codes must be CKL_F32 (0) or CKL_BF16 (1)");
  if (x_dtype == CKL_F32 && r_dtype == CKL_BF16)
    return fail(CKL_ERR_UNSUPPORTED, "a residual in bf16 goes with x in bf16");
  return CKL_OK;
}
ckl_status check_eps(float eps) {
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(CKL_ERR_INVALID_ARG, "eps must be finite and >= 0");
  return CKL_OK;
}

}  // namespace

extern "C" {

ckl_status ckl_dropout(const void* x, int32_t dtype, int64_t n, double p, uint64_t seed, uint64_t offset,
                       const int64_t* state, void* out, void* stream) {
  if (n < 0) return fail(CKL_ERR_INVALID_ARG, "n=%lld must be >= 0", (long long)n);
  if (n > kMaxElements) return fail(CKL_ERR_UNSUPPORTED, "n=%lld: at most 2^36 elements", (long long)n);
  if (!dtype_ok(dtype)) return fail(CKL_ERR_INVALID_ARG, "dtype must be CKL_F32 (0) or CKL_BF16 (1)");
  ckl::DropArgs a;
  ckl_status s = drop_args(p, seed, offset, state, &a);
  if (s != CKL_OK) return s;
  if (n == 0) return CKL_OK;
  if (!x || !out) return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(x) || !aligned16(out)) return fail(CKL_ERR_INVALID_ARG, "x and out must be 16-byte aligned");
  s = check_disjoint({{out, (size_t)n * esize(dtype), "out"}},
                     {{x, (size_t)n * esize(dtype), "x"}, {state, 16, "state"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  HIP_TRY(timed(CKL_KERNEL_ACTIVATION, st,
                [&] { return ckl::launch_dropout(x, dtype == CKL_BF16, n, a, out, st); }),
          "dropout");
  return CKL_OK;
}

ckl_status ckl_add_norm_forward(const void* x, int32_t x_dtype, const void* residual, int32_t r_dtype, int64_t T,
                                int64_t d, const void* weight, int32_t weight_dtype, float eps, double p,
                                uint64_t seed, uint64_t offset, const int64_t* state, void* h, void* y, float* rstd,
                                void* stream) {
  ckl_status s = check_norm(T, d, x_dtype, r_dtype, weight_dtype);
  if (s == CKL_OK) s = check_eps(eps);
  if (s != CKL_OK) return s;
  ckl::DropArgs a;
  s = drop_args(p, seed, offset, state, &a);
  if (s != CKL_OK) return s;
  if (T == 0) return CKL_OK;
  if (!x || !residual || !weight || !h || !y) return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(h) || !aligned16(y))
    return fail(CKL_ERR_INVALID_ARG, "x, residual, weight, h and y must be 16-byte aligned");
  if ((uintptr_t)rstd & 3u) return fail(CKL_ERR_INVALID_ARG, "rstd must be 4-byte aligned");
  const size_t n = (size_t)T * d;
  s = check_disjoint({{h, n * esize(r_dtype), "h"}, {y, n * esize(x_dtype), "y"}, {rstd, (size_t)T * 4, "rstd"}},
                     {{x, n * esize(x_dtype), "x"}, {residual, n * esize(r_dtype), "residual"},
                      {weight, (size_t)d * esize(weight_dtype), "weight"}, {state, 16, "state"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  HIP_TRY(timed(CKL_KERNEL_ACTIVATION, st,
                [&] {
                  return ckl::launch_add_norm(x, x_dtype == CKL_BF16, residual, r_dtype == CKL_BF16, T, (int)d, weight,
                                              weight_dtype == CKL_BF16, eps, a, h, 0, y, nullptr, rstd, st);
                }),
          "add_norm_forward");
  return CKL_OK;
}

ckl_status ckl_add_norm_quant(const void* x, int32_t x_dtype, const void* residual, int32_t r_dtype, int64_t T,
                              int64_t d, const void* weight, int32_t weight_dtype, float eps, int32_t form, void* h,
                              void* codes, void* scales, void* stream) {
  ckl_status s = check_norm(T, d, x_dtype, r_dtype, weight_dtype);
  if (s == CKL_OK) s = check_eps(eps);
  if (s != CKL_OK) return s;
  if (form != CKL_QUANT_INT8 && form != CKL_QUANT_E4M3)
    return fail(CKL_ERR_INVALID_ARG, "form must be CKL_QUANT_INT8 (1) or CKL_QUANT_E4M3 (2)");
  if (T == 0) return CKL_OK;
  if (!x || !residual || !weight || !h || !codes || !scales)
    return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(h) || !aligned16(codes))
    return fail(CKL_ERR_INVALID_ARG, "x, residual, weight, h and codes must be 16-byte aligned");
  if (form == CKL_QUANT_E4M3 && ((uintptr_t)scales & 3u))
    return fail(CKL_ERR_INVALID_ARG, "the rows' scales must be 4-byte aligned");
  const size_t n = (size_t)T * d;
  s = check_disjoint({{h, n * esize(r_dtype), "h"}, {codes, n, "codes"},
                      {scales, form == CKL_QUANT_INT8 ? T * exp_cols(d) : (size_t)T * 4, "scales"}},
                     {{x, n * esize(x_dtype), "x"}, {residual, n * esize(r_dtype), "residual"},
                      {weight, (size_t)d * esize(weight_dtype), "weight"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  const ckl::DropArgs none{0, 1.f, 0, 0, nullptr};
  HIP_TRY(timed(CKL_KERNEL_ACTIVATION, st,
                [&] {
                  return ckl::launch_add_norm(x, x_dtype == CKL_BF16, residual, r_dtype == CKL_BF16, T, (int)d, weight,
                                              weight_dtype == CKL_BF16, eps, none, h, form, codes, scales, nullptr, st);
                }),
          "add_norm_quant");
  return CKL_OK;
}

ckl_status ckl_add_norm_workspace_size(int64_t T, int64_t d, size_t* bytes) {
  ckl_status s = check_rows(T);
  if (s == CKL_OK) s = check_hidden(d);
  if (s != CKL_OK) return s;
  if (!bytes) return fail(CKL_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = (size_t)ckl::add_norm_backward_groups(T, d) * d * 4;
  return CKL_OK;
}

ckl_status ckl_add_norm_backward(const void* dy, int32_t x_dtype, const void* dh, int32_t r_dtype, int64_t T,
                                 int64_t d, const void* h, const float* rstd, const void* weight,
                                 int32_t weight_dtype, double p, uint64_t seed, uint64_t offset, const int64_t* state,
                                 void* dx, void* dresidual, void* dweight, void* ws, size_t ws_bytes, void* stream) {
  ckl_status s = check_norm(T, d, x_dtype, r_dtype, weight_dtype);
  if (s != CKL_OK) return s;
  ckl::DropArgs a;
  s = drop_args(p, seed, offset, state, &a);
  if (s != CKL_OK) return s;
  if (!weight || !dweight || (T > 0 && (!dy || !h || !rstd || !dresidual)))
    return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (T > 0 && !dx && (a.threshold != 0 || x_dtype != r_dtype))
    return fail(CKL_ERR_INVALID_ARG, "dx may be NULL only where it equals dresidual: no dropout, one type");
  if (!aligned16(dy) || !aligned16(dh) || !aligned16(h) || !aligned16(weight) || !aligned16(dx) ||
      !aligned16(dresidual) || !aligned16(dweight) || !aligned16(ws))
    return fail(CKL_ERR_INVALID_ARG, "dy, dh, h, weight, dx, dresidual, dweight and ws must be 16-byte aligned");
  if ((uintptr_t)rstd & 3u) return fail(CKL_ERR_INVALID_ARG, "rstd must be 4-byte aligned");
  const size_t need = (size_t)ckl::add_norm_backward_groups(T, d) * d * 4;
  if (need && (!ws || ws_bytes < need))
    return fail(CKL_ERR_WORKSPACE, "norm workspace needs %zu bytes, got %zu", need, ws ? ws_bytes : (size_t)0);
  const size_t n = (size_t)T * d;
  s = check_disjoint({{dx, n * esize(x_dtype), "dx"}, {dresidual, n * esize(r_dtype), "dresidual"},
                      {dweight, (size_t)d * esize(weight_dtype), "dweight"}, {ws, need, "ws"}},
                     {{dy, n * esize(x_dtype), "dy"}, {dh, n * esize(r_dtype), "dh"}, {h, n * esize(r_dtype), "h"},
                      {rstd, (size_t)T * 4, "rstd"}, {weight, (size_t)d * esize(weight_dtype), "weight"},
                      {state, 16, "state"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  HIP_TRY(timed(CKL_KERNEL_ACTIVATION, st,
                [&] {
                  return ckl::launch_add_norm_backward(dy, x_dtype == CKL_BF16, dh, r_dtype == CKL_BF16, T, (int)d, h,
                                                       rstd, weight, weight_dtype == CKL_BF16, a, dx, dresidual,
                                                       dweight, (float*)ws, st);
                }),
          "add_norm_backward");
  return CKL_OK;
}

}  // extern "C"
