// Host-side launchers of the log probabilities from states and head (internal;
// not part of the ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ckl {

// The forward's tile: vocabulary rows, token rows, and the workgroups that run at
// once on the GPU.
struct HeadTile {
  int kind, BM, BN, slots;
};
HeadTile head_tile(int in_bf16, int64_t rows);

// perm, n (NULL: all rows, as they are): row i is row perm[i] of the call, i < *n.
hipError_t launch_head_tokens(const void* tokens, int tokens64, int T, int Tp, int V, const int* perm, const int* n,
                              int* tok, hipStream_t st);
// T rows from H on; nrows not NULL: rows past *nrows - row0 are padding.
hipError_t launch_head_rows(const HeadTile& k, const void* H, const void* W, int T, int d, int V, const int* tok,
                            float* ztok, float4* part, int n_splits, int tiles_per_split, const int* nrows, int row0,
                            hipStream_t st);
// Rows row0 .. row0 + rows of the (packed) rows into the call's results; part [S][rows], ztok and tok of row0 on.
hipError_t launch_head_finish(const float4* part, int S, int rows, int row0, const float* ztok, const int* tok,
                              const int* perm, const int* n, float* logprob, float* entropy, float* lse,
                              hipStream_t st);
hipError_t launch_head_masked(const int* rank, int T, float* logprob, float* entropy, float* lse, hipStream_t st);
// dlogprob or dentropy may be NULL (zero).
hipError_t launch_head_consts(const void* tokens, int tokens64, int T, int Tp, int V, const int* perm, const int* n,
                              const float* lse, const float* entropy, const float* dlogprob, const float* dentropy,
                              float4* consts, int* tok, hipStream_t st);
hipError_t launch_head_grad(int in_bf16, const void* H, const void* W, int T, int d, int V, const float4* consts,
                            const int* tok, int tb0, int t_rows, int vb0, int v_rows, int n_splits,
                            int tiles_per_split, void* G, int64_t ldG, void* Gt, int64_t ldGt, const int* nrows,
                            hipStream_t st);

}  // namespace ckl
