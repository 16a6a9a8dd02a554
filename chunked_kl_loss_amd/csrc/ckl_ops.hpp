// Host-side launchers of the operators around the loss: teacher top-K,
// embedding, 8-bit activations and the RMS norm that reads them (internal; not
// part of the ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ckl {

// ------------------------------------------------------------ teacher top-K --
// Segments a row of V logits is cut into when there are `rows` of them, and
// the shifted columns of a segment.
void topk_plan(int64_t rows, int64_t V, int* segments, int64_t* seg_cols);
// cand [rows][segments][words of a segment] and state [rows][segments] are used
// when the plan has more than one segment.
int64_t topk_segment_words(int64_t K);
hipError_t launch_teacher_topk(const void* logits, int bf16, int64_t rows, int64_t V, int K, int logprob,
                               const uint8_t* mask, int* idx, float* val, float* lse, uint64_t* cand, float2* state,
                               hipStream_t st);

// ---------------------------------------------------------------- embedding --
hipError_t launch_embedding_forward(const void* W, int bf16, int64_t V, int d, int64_t v_offset, const void* tokens,
                                    int tokens64, int64_t T, float scale, void* out, hipStream_t st);
// Workspace of the backward pass, in bytes from its start.
struct EmbedWs {
  size_t key0, key1, pos0, pos1, hist, joins, part, total;
  int64_t chunk, chunks;    // positions a reducing thread walks, and their number
  int passes, digit_bits;   // radix passes (0: the positions are ranked directly)
  int64_t sort_rounds, sort_blocks;  // a sorting workgroup's keys / 1024, and their number
};
EmbedWs embed_ws(int64_t T, int64_t V, int64_t d);
hipError_t launch_embedding_backward(const void* dY, int bf16, int64_t T, int d, const void* tokens, int tokens64,
                                     int64_t V, int64_t v_offset, float scale, void* dW, int dw_bf16, int accumulate,
                                     char* ws, hipStream_t st);

// -------------------------------------------------- 8-bit activations, norm --
hipError_t launch_act_encode(const void* x, int bf16, int64_t T, int d, int8_t* codes, uint8_t* exps, hipStream_t st);
// rstd and weight not NULL: the normalised, weighted rows instead of x.
hipError_t launch_act_decode(const int8_t* codes, const uint8_t* exps, int64_t T, int d, const float* rstd,
                             const void* weight, int weight_bf16, void* out, int out_bf16, hipStream_t st);
hipError_t launch_norm_forward(const void* x, int bf16, int64_t T, int d, const void* weight, int weight_bf16,
                               float eps, void* y, int8_t* codes, uint8_t* exps, float* rstd, hipStream_t st);
// Workgroups of the backward pass; each leaves one fp32 row of d in `part`.
int64_t norm_backward_groups(int64_t T, int64_t d);
hipError_t launch_norm_backward(const void* dy, int bf16, int64_t T, int d, const int8_t* codes, const uint8_t* exps,
                                const float* rstd, const void* weight, int weight_bf16, void* dx, void* dweight,
                                float* part, hipStream_t st);

}  // namespace ckl
