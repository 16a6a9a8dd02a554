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

// ------------------------------------------------ log probabilities of tokens --
struct TokenRows {
  const void* tokens;
  int tokens64;
  const uint8_t* mask;
  float* logprob;
  float* entropy;  // (the backward pass reads it)
};
// Whether a row's alternatives are kept in the waves' registers (row_top_kernel); if
// not, rows are cut as launch_teacher_topk cuts them, with cand and state as there
// and state_e [rows][segments].  A word that comes costs a wave of the former about
// 0.15 us, a row of the latter about 8 us.  (us, registers / buffer: 60000 x 1500 bf16,
// top 5 / 20 / 64: 97 / 164 / 333 against 690 to 760; 8192 x 12000 bf16, top 5 / 20 / 64:
// 81 / 99 / 154 against 122 / 122 / 127, fp32 99 / 134 / 196 against 134 to 137; 2000 x 32000
// bf16, top 5 / 20: 40 / 57 against 44 / 50; 2048 x 201088, top 10 / 20: 179 / 199 against 170.  The border
// in words is where 20 alternatives cost about the same; 5 of them are cheaper in registers up to 32000 words: 2000 x
// 16384 28, x 16385 by the buffer 41.)
inline bool logprob_in_registers(int64_t V, int64_t top) { return V <= 2048 ? top <= 64 : V <= 16384 && top <= 24; }
hipError_t launch_token_logprobs(const void* logits, int bf16, int64_t rows, int64_t V, int top, const TokenRows& t,
                                 float* lse, int* idx, float* val, uint64_t* cand, float2* state, float* state_e,
                                 hipStream_t st);
// dlogprob or dentropy may be NULL (zero).
hipError_t launch_token_logprobs_backward(const void* logits, int bf16, int64_t rows, int64_t V, const TokenRows& t,
                                          const float* lse, const float* dlogprob, const float* dentropy,
                                          void* dlogits, hipStream_t st);

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
// dweight = the sum of `groups` fp32 rows of d, in their order by slices.
hipError_t launch_norm_dweight(const float* part, int groups, int d, int weight_bf16, void* dweight, hipStream_t st);

// -------------------------------------- dropout, norm behind a residual's sum --
// threshold of 65536: the share dropped (0: none).  state not NULL: {seed, offset}
// in device memory instead of seed, its offset added to the call's.
struct DropArgs {
  uint32_t threshold;
  float scale;
  uint64_t seed, offset;
  const int64_t* state;
};
hipError_t launch_dropout(const void* x, int bf16, int64_t n, const DropArgs& a, void* out, hipStream_t st);
// form 0: y in x's type, with dropout; 1: int8 and block exponents, 2: e4m3 and
// row scales, without.
hipError_t launch_add_norm(const void* x, int x_bf16, const void* residual, int r_bf16, int64_t T, int d,
                           const void* weight, int weight_bf16, float eps, const DropArgs& a, void* h, int form,
                           void* y, void* scales, float* rstd, hipStream_t st);
// Workgroups of the backward pass; each leaves one fp32 row of d in `part`.
int64_t add_norm_backward_groups(int64_t T, int64_t d);
// dx NULL: it is dres (no dropout, one type).
hipError_t launch_add_norm_backward(const void* dy, int x_bf16, const void* dh, int r_bf16, int64_t T, int d,
                                    const void* h, const float* rstd, const void* weight, int weight_bf16,
                                    const DropArgs& a, void* dx, void* dres, void* dweight, float* part,
                                    hipStream_t st);

}  // namespace ckl
