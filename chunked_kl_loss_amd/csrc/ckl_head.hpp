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
HeadTile head_tile(int in_bf16, int64_t rows, int64_t V);

// The rows of a call, and those that are worked on: all of them (perm, rank and n
// NULL), or the kept rows of a mask one after another: row i is row perm[i] of the
// call, i < *n, and rank[t] < 0 where row t is masked.
struct HeadRows {
  const void* tokens;
  int tokens64;
  const int *perm, *rank, *n;
};
// Rows row0 .. row0 + T of them, from H on; ztok and part [S][T] are this launch's.
hipError_t launch_head_rows(const HeadTile& k, const void* H, const void* W, int T, int d, int V, const HeadRows& rows,
                            int row0, float* ztok, float4* part, int n_splits, int tiles_per_split, hipStream_t st);
// Their results, and zeros for the masked ones of the call's rows row0 .. row0 + count.
hipError_t launch_head_finish(const float4* part, int S, int count, int V, const HeadRows& rows, int row0,
                              const float* ztok, float* logprob, float* entropy, float* lse, hipStream_t st);
// dlogprob or dentropy may be NULL (zero).
hipError_t launch_head_consts(const HeadRows& rows, int T, int Tp, int V, const float* lse, const float* entropy,
                              const float* dlogprob, const float* dentropy, float4* consts, int* tok, hipStream_t st);
// Each block of Tc of the rows below T (or *n) by the 64 words that hold their token:
// order, ascending in each group, and start [blocks][4 tiles + 1] of `tiles` times 256
// words; rows without a token are in none.
hipError_t launch_head_buckets(const int* tok, int T, int Tc, const int* n, int tiles, int* order, int* start,
                               hipStream_t st);
// dH's rows row0 .. row0 + count: the sum of S parts, [count][d] each, and of `sums` [rows][d] where it is not NULL (S may
// then be 0), + gtok W[tok] where gtok is not NULL (W in bf16).  Packed row i goes to row perm[i] (perm NULL: i),
// and those of the call's rows row0 .. row0 + count that are masked (rank not NULL) get zeros.  out may be `sums`.
hipError_t launch_head_dh(const float* part, int64_t stride, int S, const float* sums, int row0, int count, int d,
                          const int* tok, const float* gtok, const void* W, const HeadRows& rows, void* out,
                          int out_bf16, hipStream_t st);
// All T rows from parts of the transpose, [d][ldt] each (bf16: gtok is not NULL).
hipError_t launch_head_dh_t(const float* part, int64_t stride, int64_t ldt, int S, int T, int d, const int* tok,
                            const float* gtok, const void* W, const HeadRows& rows, void* dH, int dh_bf16,
                            hipStream_t st);
// bf16: the tokens' own entries go to gtok in fp32, and are 0 in G.  nrows: G is formed in blocks of
// 256 rows (fp32: 64) up to the one that holds the last row below it.
hipError_t launch_head_grad(int in_bf16, const void* H, const void* W, int T, int d, int V, const float4* consts,
                            const int* tok, float* gtok, int tb0, int t_rows, int vb0, int v_rows, int tiles_per_split,
                            void* G, int64_t ldG, void* Gt, int64_t ldGt, const int* nrows, hipStream_t st);

}  // namespace ckl
