// gfx950 kernels on rows of logits in memory: log probabilities of given tokens
// with entropy and top alternatives, and the gradient of the first two.
#include <algorithm>
#include <type_traits>

#include "ckl_ops.hpp"
#include "ckl_topk.hpp"

namespace ckl {

namespace {

// ---------------------------------------------------- without alternatives --
// One workgroup a row, in one pass: sums of 2^a and a 2^a behind a running
// reference (RowAcc).  Rows begin at any column of an odd V, so vectors are
// counted from the 16-byte boundary before the row and the first and last are
// masked.  Two groups of loads are under way while one is looked at.
constexpr int kRowVecs = 4;

template <typename T, int THREADS>
__global__ __launch_bounds__(THREADS) void row_stats_kernel(const T* __restrict__ logits, int64_t rows, int V,
                                                            const uint8_t* __restrict__ mask, RowOut out,
                                                            float* __restrict__ lse) {
  __shared__ float wm[THREADS / 64], ws[THREADS / 64], we[THREADS / 64];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  if (mask != nullptr && mask[row] == 0) {
    if (tid == 0) lse[row] = out.logprob[row] = out.entropy[row] = 0.f;
    return;
  }
  const T* p = logits + row * (int64_t)V;
  const int first = (int)(((uintptr_t)p & 15u) / sizeof(T)), hi = first + V;
  const T* base = p - first;
  const int64_t rest = (rows - row) * V;  // columns that can be read: a few past the row where others follow
  const int end = first + (int)(rest < V + 8 ? rest : V + 8);
  auto fetch = [&](int j) {
    Raw8<T> r;
    if (j >= first && j + 8 <= hi) {
      r.load(base + j);
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = -INFINITY;
      if (j < hi) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = j + i >= first && j + i < hi && j + i < end ? (float)base[j + i] : -INFINITY;
      }
      r.from(f);
    }
    return r;
  };
  constexpr int kStep = THREADS * 8, kTile = kStep * kRowVecs;
  RowAcc acc;
  Raw8<T> raw[kRowVecs], next[kRowVecs];
#pragma unroll
  for (int u = 0; u < kRowVecs; ++u) raw[u] = fetch(u * kStep + tid * 8);
  for (int t0 = 0; t0 < hi; t0 += kTile) {
    if (t0 + kTile < hi) {
#pragma unroll
      for (int u = 0; u < kRowVecs; ++u) next[u] = fetch(t0 + kTile + u * kStep + tid * 8);
    }
#pragma unroll
    for (int u = 0; u < kRowVecs; ++u) {
      float vm = raw[u].get(0);
#pragma unroll
      for (int i = 1; i < 8; ++i) vm = fmaxf(vm, raw[u].get(i));
      acc.add(raw[u], vm);
    }
#pragma unroll
    for (int u = 0; u < kRowVecs; ++u) raw[u] = next[u];
  }
  acc.settle();
  float m = acc.m, s = acc.s, e = acc.e;
  ent_reduce(m, s, e, wm, ws, we);
  if (tid == 0) {
    const float l = s == s ? m + logf(s) : s;
    lse[row] = l;
    row_outputs(out, logits, row, V, l, s, e);
  }
}

// ---------------------------------------------------------------- gradient --
// dz = a (1[v = token] - q) - b q (log q + entropy), q = exp(z - lse), for a row's
// incoming gradients a (log probability) and b (entropy).  A row whose mask is 0,
// whose a and b are 0 or that has no column left (lse = -inf) gets zeros and is
// not read.  One pass; a workgroup takes kGradVecs vectors of a row a thread.
constexpr int kGradThreads = 256;

template <typename T, int VECS>
__global__ __launch_bounds__(kGradThreads) void logprob_grad_kernel(
    const T* __restrict__ logits, int V, int parts, const void* __restrict__ tokens, int tokens64,
    const uint8_t* __restrict__ mask, const float* __restrict__ lse, const float* __restrict__ entropy,
    const float* __restrict__ dlogprob, const float* __restrict__ dentropy, T* __restrict__ dlogits) {
  const int64_t row = blockIdx.x / parts;
  const int part = (int)(blockIdx.x - row * parts);
  const int64_t tok = token_at(tokens, tokens64, row);
  const bool inside = tok >= 0 && tok < V;
  const bool keep = mask == nullptr || mask[row] != 0;
  const float a = keep && inside && dlogprob != nullptr ? dlogprob[row] : 0.f;
  const float b = keep && dentropy != nullptr ? dentropy[row] : 0.f;
  const float l = lse[row];
  const bool zero = (a == 0.f && b == 0.f) || l == -INFINITY;
  const T* p = logits + row * (int64_t)V;
  // (both arrays begin on a 16-byte boundary, so their rows are shifted alike)
  const int first = (int)(((uintptr_t)p & 15u) / sizeof(T)), hi = first + V;
  const T* base = p - first;
  T* dst = dlogits + row * (int64_t)V - first;
  const int target = inside ? first + (int)tok : -1;
  const float c0 = -a - (b == 0.f ? 0.f : b * entropy[row]);
  auto grad = [&](float z, int j) {
    const float lq = z - l, q = fast_exp2(lq * kLog2e);
    // (where q is zero so is q log q: log q is kept finite; a NaN passes)
    const float lf = lq < kExpZero ? kExpZero : lq;
    return q * (c0 - b * lf) + (j == target ? a : 0.f);
  };
  const int j0 = (part * VECS * kGradThreads + (int)threadIdx.x) * 8;
  Raw8<T> raw[VECS];
#pragma unroll
  for (int u = 0; u < VECS; ++u) {
    const int j = j0 + u * kGradThreads * 8;
    if (!zero && j >= first && j + 8 <= hi) raw[u].load(base + j);
  }
#pragma unroll
  for (int u = 0; u < VECS; ++u) {
    const int j = j0 + u * kGradThreads * 8;
    if (j >= first && j + 8 <= hi) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = zero ? 0.f : grad(raw[u].get(i), j + i);
      stream8(dst + j, f);
    } else if (j < hi) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (j + i >= first && j + i < hi) dst[j + i] = (T)(zero ? 0.f : grad((float)base[j + i], j + i));
    }
  }
}

}  // namespace

// -------------------------------------------------------------- launchers --
hipError_t launch_token_logprobs(const void* logits, int bf16, int64_t rows, int64_t V, int top,
                                 const TokenRows& t, float* lse, int* idx, float* val, uint64_t* cand, float2* state,
                                 float* state_e, hipStream_t st) {
  const RowOut out{t.tokens, t.tokens64, t.logprob, t.entropy, state_e};
  if (top == 0) {
    auto go = [&](auto* p) {
      using E = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
      auto run = [&](auto threads) {
        constexpr int N = decltype(threads)::value;
        row_stats_kernel<E, N><<<(unsigned)rows, N, 0, st>>>(p, rows, (int)V, t.mask, out, lse);
      };
      if (V <= 2048)
        run(std::integral_constant<int, 64>{});
      else if (V <= 65536)
        run(std::integral_constant<int, 256>{});
      else
        run(std::integral_constant<int, 512>{});
    };
    bf16 ? go((const bf16_t*)logits) : go((const float*)logits);
    return hipGetLastError();
  }
  int segments;
  int64_t seg_cols;
  topk_plan(rows, V, &segments, &seg_cols);
  const unsigned blocks = (unsigned)(rows * segments);
  auto go = [&](auto* p, auto cap) {
    using E = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    constexpr int CAP = decltype(cap)::value;
    topk_rows_kernel<E, CAP, true><<<blocks, kTopkThreads, 0, st>>>(p, rows, (int)V, top, segments, (int)seg_cols, 1,
                                                                    t.mask, idx, val, lse, cand, state, out);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || segments == 1) return e;
    topk_merge_kernel<E, CAP, true><<<(unsigned)rows, kTopkThreads, 0, st>>>(cand, state, top, segments, 1, t.mask, idx,
                                                                            val, lse, p, (int)V, out);
    return hipGetLastError();
  };
  using Small = std::integral_constant<int, 4096>;
  using Large = std::integral_constant<int, 8192>;
  if (bf16) return top <= 1024 ? go((const bf16_t*)logits, Small{}) : go((const bf16_t*)logits, Large{});
  return top <= 1024 ? go((const float*)logits, Small{}) : go((const float*)logits, Large{});
}

hipError_t launch_token_logprobs_backward(const void* logits, int bf16, int64_t rows, int64_t V, const TokenRows& t,
                                          const float* lse, const float* dlogprob, const float* dentropy,
                                          void* dlogits, hipStream_t st) {
  auto go = [&](auto* p, auto vecs) {
    using E = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    constexpr int VECS = decltype(vecs)::value;
    const int parts = (int)cdiv(V + 7, VECS * kGradThreads * 8);
    logprob_grad_kernel<E, VECS><<<(unsigned)(rows * parts), kGradThreads, 0, st>>>(
        p, (int)V, parts, t.tokens, t.tokens64, t.mask, lse, t.entropy, dlogprob, dentropy, (E*)dlogits);
    return hipGetLastError();
  };
  using One = std::integral_constant<int, 1>;
  using Four = std::integral_constant<int, 4>;
  if (bf16) return V <= 2048 ? go((const bf16_t*)logits, One{}) : go((const bf16_t*)logits, Four{});
  return V <= 2048 ? go((const float*)logits, One{}) : go((const float*)logits, Four{});
}

}  // namespace ckl
