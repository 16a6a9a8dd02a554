// Host side of the operators around the loss (teacher top-K, embedding, 8-bit
// activations and their norm): argument checks, workspace sizes and launches
// behind the C ABI declared in include/ckl.h.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/ckl.h"
#include "ckl_host.hpp"
#include "ckl_ops.hpp"

using namespace ckl::host;

namespace {

ckl_status check_topk(int64_t T, int64_t V, int64_t K) {
  ckl_status s = check_rows(T);
  if (s == CKL_OK) s = check_vocab(V);
  if (s != CKL_OK) return s;
  if (K < 1 || K > V) return fail(CKL_ERR_INVALID_ARG, "K=%lld must satisfy 1 <= K <= V", (long long)K);
  if (K > kMaxK) return fail(CKL_ERR_UNSUPPORTED, "K=%lld exceeds %lld", (long long)K, (long long)kMaxK);
  if (T * K >= ((int64_t)1 << 31)) return fail(CKL_ERR_UNSUPPORTED, "T*K must stay below 2^31");
  return CKL_OK;
}

// Words and states of the row segments.
struct TopkWs {
  size_t cand, state, total;
};
TopkWs topk_layout(int64_t T, int64_t V, int64_t K) {
  TopkWs w{};
  int segments = 1;
  int64_t cols = 0;
  if (T > 0) ckl::topk_plan(T, V, &segments, &cols);
  if (segments > 1) {
    w.state = align256((size_t)T * segments * ckl::topk_segment_words(K) * 8);
    w.total = w.state + align256((size_t)T * segments * 8);
  }
  return w;
}

ckl_status check_embedding(int64_t T, int64_t d, int64_t V, int64_t v_offset) {
  ckl_status s = check_rows(T);
  if (s == CKL_OK) s = check_hidden(d);
  if (s == CKL_OK) s = check_vocab(V);
  if (s != CKL_OK) return s;
  if (v_offset < 0 || v_offset > INT64_MAX - V)
    return fail(CKL_ERR_INVALID_ARG, "v_offset must be >= 0 and v_offset + V at most 2^63 - 1");
  return CKL_OK;
}

}  // namespace

extern "C" {

ckl_status ckl_topk_workspace_size(int64_t T, int64_t V, int64_t K, size_t* bytes) {
  ckl_status s = check_topk(T, V, K);
  if (s != CKL_OK) return s;
  if (!bytes) return fail(CKL_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = topk_layout(T, V, K).total;
  return CKL_OK;
}

ckl_status ckl_teacher_topk(const void* logits, int32_t dtype, int64_t T, int64_t V, int64_t K, int32_t teacher_form,
                            const uint8_t* mask, int32_t* idx, float* values, float* lse, void* ws, size_t ws_bytes,
                            void* stream) {
  ckl_status s = check_topk(T, V, K);
  if (s != CKL_OK) return s;
  if (!dtype_ok(dtype)) return fail(CKL_ERR_INVALID_ARG, "dtype must be CKL_F32 (0) or CKL_BF16 (1)");
  if (teacher_form != CKL_TEACHER_LOGITS && teacher_form != CKL_TEACHER_LOGPROBS)
    return fail(CKL_ERR_INVALID_ARG, "teacher_form must be CKL_TEACHER_LOGITS (0) or CKL_TEACHER_LOGPROBS (1)");
  if (T == 0) return CKL_OK;
  if (!logits || !idx || !values || !lse) return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(logits) || !aligned16(idx) || !aligned16(values) || !aligned16(ws))
    return fail(CKL_ERR_INVALID_ARG, "logits, idx, values and ws must be 16-byte aligned");
  if ((uintptr_t)lse & 3u) return fail(CKL_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  const TopkWs w = topk_layout(T, V, K);
  if (w.total && (!ws || ws_bytes < w.total))
    return fail(CKL_ERR_WORKSPACE, "top-K workspace needs %zu bytes, got %zu", w.total, ws ? ws_bytes : (size_t)0);
  s = check_disjoint({{idx, (size_t)(T * K) * 4, "idx"}, {values, (size_t)(T * K) * 4, "values"},
                      {lse, (size_t)T * 4, "lse"}, {ws, w.total, "ws"}},
                     {{logits, (size_t)T * V * esize(dtype), "logits"}, {mask, (size_t)T, "mask"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  char* b = (char*)ws;
  HIP_TRY(timed(CKL_KERNEL_TOPK, st,
                [&] {
                  return ckl::launch_teacher_topk(logits, dtype == CKL_BF16, T, V, (int)K,
                                                  teacher_form == CKL_TEACHER_LOGPROBS, mask, idx, values, lse,
                                                  (uint64_t*)(b + w.cand), (float2*)(b + w.state), st);
                }),
          "teacher_topk");
  return CKL_OK;
}

ckl_status ckl_embedding_forward(const void* W, int32_t dtype, int64_t V, int64_t d, int64_t v_offset,
                                 const void* tokens, int32_t token_bytes, int64_t T, float scale, void* out,
                                 void* stream) {
  ckl_status s = check_embedding(T, d, V, v_offset);
  if (s != CKL_OK) return s;
  // (32 elements a thread, and a launch keeps the low 32 bits of its number of threads)
  if (ceil_div(T * (d / 8), 1024) >= ((int64_t)1 << 24)) return fail(CKL_ERR_UNSUPPORTED, "T*d: at most 2^37 - 8192");
  if (!dtype_ok(dtype)) return fail(CKL_ERR_INVALID_ARG, "dtype must be CKL_F32 (0) or CKL_BF16 (1)");
  if (token_bytes != 4 && token_bytes != 8) return fail(CKL_ERR_INVALID_ARG, "token_bytes must be 4 or 8");
  if (T == 0) return CKL_OK;
  if (!W || !tokens || !out) return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(W) || !aligned16(out)) return fail(CKL_ERR_INVALID_ARG, "W and out must be 16-byte aligned");
  if ((uintptr_t)tokens & (uintptr_t)(token_bytes - 1))
    return fail(CKL_ERR_INVALID_ARG, "tokens must be aligned to their size");
  s = check_disjoint({{out, (size_t)T * d * esize(dtype), "out"}},
                     {{W, (size_t)V * d * esize(dtype), "W"}, {tokens, (size_t)T * token_bytes, "tokens"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  HIP_TRY(timed(CKL_KERNEL_EMBEDDING, st,
                [&] {
                  return ckl::launch_embedding_forward(W, dtype == CKL_BF16, V, (int)d, v_offset, tokens,
                                                       token_bytes == 8, T, scale, out, st);
                }),
          "embedding_forward");
  return CKL_OK;
}

ckl_status ckl_embedding_workspace_size(int64_t T, int64_t d, int64_t V, size_t* bytes) {
  ckl_status s = check_embedding(T, d, V, 0);
  if (s != CKL_OK) return s;
  if (!bytes) return fail(CKL_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = T > 0 ? ckl::embed_ws(T, V, d).total : 0;
  return CKL_OK;
}

ckl_status ckl_embedding_backward(const void* dY, int32_t dtype, int64_t T, int64_t d, const void* tokens,
                                  int32_t token_bytes, int64_t V, int64_t v_offset, float scale, void* dW,
                                  int32_t dw_dtype, int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  ckl_status s = check_embedding(T, d, V, v_offset);
  if (s != CKL_OK) return s;
  if (!dtype_ok(dtype) || !dtype_ok(dw_dtype))
    return fail(CKL_ERR_INVALID_ARG, "dtype codes must be CKL_F32 (0) or CKL_BF16 (1)");
  if (token_bytes != 4 && token_bytes != 8) return fail(CKL_ERR_INVALID_ARG, "token_bytes must be 4 or 8");
  if (accumulate != 0 && accumulate != 1) return fail(CKL_ERR_INVALID_ARG, "accumulate must be 0 or 1");
  if (!dW || (T > 0 && (!dY || !tokens))) return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(dY) || !aligned16(dW) || !aligned16(ws))
    return fail(CKL_ERR_INVALID_ARG, "dY, dW and ws must be 16-byte aligned");
  if ((uintptr_t)tokens & (uintptr_t)(token_bytes - 1))
    return fail(CKL_ERR_INVALID_ARG, "tokens must be aligned to their size");
  const size_t need = T > 0 ? ckl::embed_ws(T, V, d).total : 0;
  if (need && (!ws || ws_bytes < need))
    return fail(CKL_ERR_WORKSPACE, "embedding workspace needs %zu bytes, got %zu", need, ws ? ws_bytes : (size_t)0);
  s = check_disjoint({{dW, (size_t)V * d * esize(dw_dtype), "dW"}, {ws, need, "ws"}},
                     {{dY, (size_t)T * d * esize(dtype), "dY"}, {tokens, (size_t)T * token_bytes, "tokens"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  HIP_TRY(timed(CKL_KERNEL_EMBEDDING, st,
                [&] {
                  return ckl::launch_embedding_backward(dY, dtype == CKL_BF16, T, (int)d, tokens, token_bytes == 8, V,
                                                        v_offset, scale, dW, dw_dtype == CKL_BF16, accumulate,
                                                        (char*)ws, st);
                }),
          "embedding_backward");
  return CKL_OK;
}

ckl_status ckl_act_encode(const void* x, int32_t dtype, int64_t T, int64_t d, int8_t* codes, uint8_t* exps,
                          void* stream) {
  ckl_status s = check_rows(T);
  if (s == CKL_OK) s = check_hidden(d);
  if (s != CKL_OK) return s;
  if (!dtype_ok(dtype)) return fail(CKL_ERR_INVALID_ARG, "dtype must be CKL_F32 (0) or CKL_BF16 (1)");
  if (T == 0) return CKL_OK;
  if (!x || !codes || !exps) return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(x) || !aligned16(codes)) return fail(CKL_ERR_INVALID_ARG, "x and codes must be 16-byte aligned");
  s = check_disjoint({{codes, (size_t)T * d, "codes"}, {exps, T * exp_cols(d), "exps"}},
                     {{x, (size_t)T * d * esize(dtype), "x"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  HIP_TRY(timed(CKL_KERNEL_ACTIVATION, st,
                [&] { return ckl::launch_act_encode(x, dtype == CKL_BF16, T, (int)d, codes, exps, st); }),
          "act_encode");
  return CKL_OK;
}

ckl_status ckl_act_decode(const int8_t* codes, const uint8_t* exps, int64_t T, int64_t d, const float* rstd,
                          const void* weight, int32_t weight_dtype, void* out, int32_t out_dtype, void* stream) {
  ckl_status s = check_rows(T);
  if (s == CKL_OK) s = check_hidden(d);
  if (s != CKL_OK) return s;
  if (!dtype_ok(weight_dtype) || !dtype_ok(out_dtype))
    return fail(CKL_ERR_INVALID_ARG, "dtype codes must be CKL_F32 (0) or CKL_BF16 (1)");
  if (T == 0) return CKL_OK;
  if (!codes || !exps || !out) return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((rstd == nullptr) != (weight == nullptr))
    return fail(CKL_ERR_INVALID_ARG, "rstd and weight go together: both or neither");
  if (!aligned16(codes) || !aligned16(weight) || !aligned16(out))
    return fail(CKL_ERR_INVALID_ARG, "codes, weight and out must be 16-byte aligned");
  if ((uintptr_t)rstd & 3u) return fail(CKL_ERR_INVALID_ARG, "rstd must be 4-byte aligned");
  s = check_disjoint({{out, (size_t)T * d * esize(out_dtype), "out"}},
                     {{codes, (size_t)T * d, "codes"}, {exps, T * exp_cols(d), "exps"}, {rstd, (size_t)T * 4, "rstd"},
                      {weight, (size_t)d * esize(weight_dtype), "weight"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  HIP_TRY(timed(CKL_KERNEL_ACTIVATION, st,
                [&] {
                  return ckl::launch_act_decode(codes, exps, T, (int)d, rstd, weight, weight_dtype == CKL_BF16, out,
                                                out_dtype == CKL_BF16, st);
                }),
          "act_decode");
  return CKL_OK;
}

ckl_status ckl_norm_forward(const void* x, int32_t dtype, int64_t T, int64_t d, const void* weight,
                            int32_t weight_dtype, float eps, void* y, int8_t* codes, uint8_t* exps, float* rstd,
                            void* stream) {
  ckl_status s = check_rows(T);
  if (s == CKL_OK) s = check_hidden(d);
  if (s != CKL_OK) return s;
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype))
    return fail(CKL_ERR_INVALID_ARG, "dtype codes must be CKL_F32 (0) or CKL_BF16 (1)");
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(CKL_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (T == 0) return CKL_OK;
  if (!x || !weight || !y) return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if ((codes == nullptr) != (exps == nullptr) || (codes == nullptr) != (rstd == nullptr))
    return fail(CKL_ERR_INVALID_ARG, "codes, exps and rstd go together: all or none");
  if (!aligned16(x) || !aligned16(weight) || !aligned16(y) || !aligned16(codes))
    return fail(CKL_ERR_INVALID_ARG, "x, weight, y and codes must be 16-byte aligned");
  if ((uintptr_t)rstd & 3u) return fail(CKL_ERR_INVALID_ARG, "rstd must be 4-byte aligned");
  s = check_disjoint({{y, (size_t)T * d * esize(dtype), "y"}, {codes, (size_t)T * d, "codes"},
                      {exps, T * exp_cols(d), "exps"}, {rstd, (size_t)T * 4, "rstd"}},
                     {{x, (size_t)T * d * esize(dtype), "x"}, {weight, (size_t)d * esize(weight_dtype), "weight"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  HIP_TRY(timed(CKL_KERNEL_ACTIVATION, st,
                [&] {
                  return ckl::launch_norm_forward(x, dtype == CKL_BF16, T, (int)d, weight, weight_dtype == CKL_BF16,
                                                  eps, y, codes, exps, rstd, st);
                }),
          "norm_forward");
  return CKL_OK;
}

ckl_status ckl_norm_workspace_size(int64_t T, int64_t d, size_t* bytes) {
  ckl_status s = check_rows(T);
  if (s == CKL_OK) s = check_hidden(d);
  if (s != CKL_OK) return s;
  if (!bytes) return fail(CKL_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = (size_t)ckl::norm_backward_groups(T, d) * d * 4;
  return CKL_OK;
}

ckl_status ckl_norm_backward(const void* dy, int32_t dtype, int64_t T, int64_t d, const int8_t* codes,
                             const uint8_t* exps, const float* rstd, const void* weight, int32_t weight_dtype,
                             void* dx, void* dweight, void* ws, size_t ws_bytes, void* stream) {
  ckl_status s = check_rows(T);
  if (s == CKL_OK) s = check_hidden(d);
  if (s != CKL_OK) return s;
  if (!dtype_ok(dtype) || !dtype_ok(weight_dtype))
    return fail(CKL_ERR_INVALID_ARG, "dtype codes must be CKL_F32 (0) or CKL_BF16 (1)");
  if (!weight || !dweight || (T > 0 && (!dy || !codes || !exps || !rstd || !dx)))
    return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(dy) || !aligned16(codes) || !aligned16(weight) || !aligned16(dx) || !aligned16(dweight) ||
      !aligned16(ws))
    return fail(CKL_ERR_INVALID_ARG, "dy, codes, weight, dx, dweight and ws must be 16-byte aligned");
  if ((uintptr_t)rstd & 3u) return fail(CKL_ERR_INVALID_ARG, "rstd must be 4-byte aligned");
  const size_t need = (size_t)ckl::norm_backward_groups(T, d) * d * 4;
  if (need && (!ws || ws_bytes < need))
    return fail(CKL_ERR_WORKSPACE, "norm workspace needs %zu bytes, got %zu", need, ws ? ws_bytes : (size_t)0);
  s = check_disjoint({{dx, (size_t)T * d * esize(dtype), "dx"}, {dweight, (size_t)d * esize(weight_dtype), "dweight"},
                      {ws, need, "ws"}},
                     {{dy, (size_t)T * d * esize(dtype), "dy"}, {codes, (size_t)T * d, "codes"},
                      {exps, T * exp_cols(d), "exps"}, {rstd, (size_t)T * 4, "rstd"},
                      {weight, (size_t)d * esize(weight_dtype), "weight"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  HIP_TRY(timed(CKL_KERNEL_ACTIVATION, st,
                [&] {
                  return ckl::launch_norm_backward(dy, dtype == CKL_BF16, T, (int)d, codes, exps, rstd, weight,
                                                   weight_dtype == CKL_BF16, dx, dweight, (float*)ws, st);
                }),
          "norm_backward");
  return CKL_OK;
}

}  // extern "C"
