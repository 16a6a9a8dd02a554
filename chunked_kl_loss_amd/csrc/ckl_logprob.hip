// gfx950 kernels on rows of logits in memory: log probabilities of given tokens
// with entropy and top alternatives, and the gradient of the first two.
#include <algorithm>
#include <type_traits>

#include "ckl_ops.hpp"
#include "ckl_topk.hpp"

namespace ckl {

namespace {

// A row as vectors of eight: rows begin at any column of an odd V, so vectors are
// counted from the 16-byte boundary before the row, and what lies outside it reads
// as -infinity.
template <typename T>
struct RowVecs {
  const T* base;
  int first, hi;  // the row is [first, hi) from base on
  __device__ __forceinline__ RowVecs(const T* logits, int64_t row, int V) {
    const T* p = logits + row * (int64_t)V;
    first = (int)(((uintptr_t)p & 15u) / sizeof(T));
    hi = first + V;
    base = p - first;
  }
  __device__ __forceinline__ Raw8<T> fetch(int j) const {
    Raw8<T> r;
    if (j >= first && j + 8 <= hi) {
      r.load(base + j);
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = j + i >= first && j + i < hi ? (float)base[j + i] : -INFINITY;
      r.from(f);
    }
    return r;
  }
};
template <typename T>
__device__ __forceinline__ float vec_max(const Raw8<T>& r) {
  float m = r.get(0);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, r.get(i));
  return m;
}

// ---------------------------------------------------- without alternatives --
// One workgroup a row, in one pass: sums of 2^a and a 2^a behind a running
// reference (RowAcc), four vectors a thread under way while four are looked at.
// Bound by memory where there are many rows (2048 x 201088 bf16: 154 us, 5.4 TB/s;
// fp32 274, 6.0) and by one workgroup's way along the row where there are few: 1 to 64
// rows of 32000 words 7 to 8 us, of 201088 19 to 23 (the host's part of a call 14).
constexpr int kRowVecs = 4;

template <typename T, int THREADS>
__global__ __launch_bounds__(THREADS) void row_stats_kernel(const T* __restrict__ logits, int V,
                                                            const uint8_t* __restrict__ mask, RowOut out,
                                                            float* __restrict__ lse) {
  __shared__ float wm[THREADS / 64], ws[THREADS / 64], we[THREADS / 64];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  if (mask != nullptr && mask[row] == 0) {
    if (tid == 0) lse[row] = out.logprob[row] = out.entropy[row] = 0.f;
    return;
  }
  const RowVecs<T> in(logits, row, V);
  constexpr int kStep = THREADS * 8, kTile = kStep * kRowVecs;
  RowAcc acc;
  Raw8<T> raw[kRowVecs], next[kRowVecs];
#pragma unroll
  for (int u = 0; u < kRowVecs; ++u) raw[u] = in.fetch(u * kStep + tid * 8);
  for (int t0 = 0; t0 < in.hi; t0 += kTile) {
    if (t0 + kTile < in.hi) {
#pragma unroll
      for (int u = 0; u < kRowVecs; ++u) next[u] = in.fetch(t0 + kTile + u * kStep + tid * 8);
    }
#pragma unroll
    for (int u = 0; u < kRowVecs; ++u) acc.add(raw[u], vec_max(raw[u]));
#pragma unroll
    for (int u = 0; u < kRowVecs; ++u) raw[u] = next[u];
  }
  acc.settle();
  float m = acc.m, s = acc.s, e = acc.e;
  ent_reduce(m, s, e, wm, ws, we);
  if (tid == 0) {
    const float l = s == s ? m + logf(s) : s;
    lse[row] = l;
    row_outputs(out, logits, row, V, l, m, s, e);
  }
}

// --------------------------------------------------------- few alternatives --
// The same pass, and every wave keeps the 64 largest words (see topk_rows_kernel)
// of what it has seen, in order, one to a lane; the first K of them are exact.  A
// first bound comes from the lanes' maxima over the first group of vectors: the
// largest key (but for its low bits) that K of them reach.  From then on a vector
// is looked at where its maximum is no smaller than the K-th word's, which for a
// row in no order happens K ln(columns / K) times a wave; a word is put in its
// place by one comparison of all lanes and a shift, or, where many come at once,
// 64 are sorted and merged.  No barrier until the waves' lists are joined.  Bound by
// the latency of the words' steps: without alternatives 8192 x 12000 bf16 takes 47 us,
// with 5 of them 72 to 81, with 20 99.  Eight waves a SIMD leave 64 registers, of which 2
// or 3 (and 21 to 27 scalar ones) are spilled around the words' steps.
__device__ __forceinline__ uint64_t lane_word(uint64_t w, int lane) {
  return ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(w >> 32), lane) << 32) |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)w, lane);
}
// The word of the lane below (lane 0: its own).
__device__ __forceinline__ uint64_t word_below(uint64_t w) {
  const int hi = (int)(w >> 32), lo = (int)(uint32_t)w;
  return ((uint64_t)(uint32_t)__builtin_amdgcn_update_dpp(hi, hi, 0x138, 0xf, 0xf, false) << 32) |
         (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, 0x138, 0xf, 0xf, false);
}
__device__ __forceinline__ uint64_t word_xor(uint64_t w, int lanes) {
  return ((uint64_t)(uint32_t)__shfl_xor((int)(w >> 32), lanes) << 32) | (uint32_t)__shfl_xor((int)(uint32_t)w, lanes);
}
// Compare-exchange with the lane `lanes` away: the larger word to the lower lane,
// or to the upper one.
__device__ __forceinline__ uint64_t word_step(uint64_t w, int lanes, bool larger_up) {
  const uint64_t o = word_xor(w, lanes);
  const bool upper = (threadIdx.x & lanes) != 0;
  return (upper == larger_up) == (w > o) ? w : o;
}
// 64 words in descending order over the lanes.
__device__ __forceinline__ uint64_t word_sort(uint64_t w) {
#pragma unroll
  for (int k = 2; k <= 64; k *= 2)
#pragma unroll
    for (int j = k / 2; j > 0; j /= 2) w = word_step(w, j, (threadIdx.x & k & 63) != 0);
  return w;
}
// The 64 largest of two descending lists, descending.
__device__ __forceinline__ uint64_t word_merge(uint64_t a, uint64_t b) {
  const uint64_t turned = word_xor(b, 63);
  a = a > turned ? a : turned;
#pragma unroll
  for (int j = 32; j > 0; j /= 2) a = word_step(a, j, false);
  return a;
}

template <typename T, int THREADS>
__global__ __launch_bounds__(THREADS, 8) void row_top_kernel(const T* __restrict__ logits, int V, int K,
                                                          const uint8_t* __restrict__ mask, RowOut out,
                                                          float* __restrict__ lse, int* __restrict__ idx,
                                                          float* __restrict__ val) {
  constexpr int WAVES = THREADS / 64;
  __shared__ float wm[WAVES], ws[WAVES], we[WAVES];
  __shared__ uint64_t lists[WAVES][64];
  __shared__ uint32_t first_key[2][WAVES];
  __shared__ unsigned long long shared_cut;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x;
  idx += row * K;
  val += row * K;
  if (mask != nullptr && mask[row] == 0) {
    if (tid < K) {
      idx[tid] = tid;
      val[tid] = 0.f;
    }
    if (tid == 0) lse[row] = out.logprob[row] = out.entropy[row] = 0.f;
    return;
  }
  const RowVecs<T> in(logits, row, V);
  constexpr int VECS = sizeof(T) == 2 ? 4 : 2;
  constexpr int kStep = THREADS * 8, kTile = kStep * VECS;
  RowAcc acc;
  uint64_t best = 0, cut = 0;  // words above `cut` are wanted
  float bound = key_value(0);  // (a NaN: all are)
  Raw8<T> raw[VECS], next[VECS];
#pragma unroll
  for (int u = 0; u < VECS; ++u) raw[u] = in.fetch(u * kStep + tid * 8);
  {
    float m = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
      m = fmaxf(m, vec_max(raw[u]));
#pragma unroll
      for (int i = 0; i < 8; ++i) nan |= raw[u].get(i) != raw[u].get(i);
    }
    // (a lane that holds nothing of the row counts for none)
    const int j = tid * 8;
    const uint32_t key = nan ? kNanKey : j + 8 > in.first && j < in.hi ? order_key(m) : 0u;
    // K lanes reach the largest of the waves' K-th largest, and the least of their (K / waves)-th largest (bit by
    // bit, but for the low ones: a lower key serves as well)
    const int share = (K + WAVES - 1) / WAVES;
    uint32_t t = 0, t_share = 0;
#pragma unroll
    for (int bit = 31; bit >= 12; --bit) {
      const uint32_t up = t | (1u << bit), up_share = t_share | (1u << bit);
      if (__popcll(__ballot(key >= up)) >= K) t = up;
      if (WAVES > 1 && __popcll(__ballot(key >= up_share)) >= share) t_share = up_share;
    }
    if constexpr (WAVES > 1) {
      if (lane == 0) {
        first_key[0][wave] = t;
        first_key[1][wave] = t_share;
      }
      if (tid == 0) shared_cut = 0;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        t = first_key[0][w] > t ? first_key[0][w] : t;
        t_share = first_key[1][w] < t_share ? first_key[1][w] : t_share;
      }
      t = t_share > t ? t_share : t;
    }
    if (t != 0) {
      cut = ((uint64_t)t << 32) - 1;
      bound = key_value(t);
    }
  }
  uint64_t told = cut;  // the largest cut that the other waves know of
  // the words of the lanes `who`, each put in its place
  auto insert = [&](uint64_t word, uint64_t who) {
    if (!who) return;
    while (who) {
      const uint64_t w = lane_word(word, __builtin_ctzll(who));
      who &= who - 1;
      const int place = __popcll(__ballot(best > w));
      const uint64_t below = word_below(best);
      best = lane < place ? best : lane == place ? w : below;
    }
    const uint64_t last = lane_word(best, K - 1);
    cut = last > cut ? last : cut;
  };
  for (int t0 = 0; t0 < in.hi; t0 += kTile) {
    if (t0 + kTile < in.hi) {
#pragma unroll
      for (int u = 0; u < VECS; ++u) next[u] = in.fetch(t0 + kTile + u * kStep + tid * 8);
    }
    if constexpr (WAVES > 1) {
      // K words above a wave's cut are K of the row's: the waves share the largest (it only spares them words that
      // would be dropped at the end, whenever they learn of it)
      if (cut > told) {
        if (lane == 0) atomicMax(&shared_cut, (unsigned long long)cut);
        told = cut;
      }
      const uint64_t theirs = *(volatile unsigned long long*)&shared_cut;
      const uint64_t known = ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(theirs >> 32)) << 32) |
                             (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)theirs);
      if (known > cut) {
        cut = told = known;
        bound = key_value((uint32_t)((cut + 1) >> 32));
      }
    }
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
      const float vm = vec_max(raw[u]);
      const float sum = acc.add(raw[u], vm);
      const bool hot = !(vm < bound) || sum != sum;  // (NaN: fmaxf passes it over, the sum does not)
      uint64_t lanes = __ballot(hot);
      if (lanes) {
        const int j = t0 + u * kStep + tid * 8;
        if (__popcll(lanes) > 8) {  // (the first vectors, or rising rows)
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const bool there = hot && j + i >= in.first && j + i < in.hi;
            const uint64_t word =
                there ? ((uint64_t)order_key(raw[u].pick(i)) << 32) | ~(uint32_t)(j + i - in.first) : 0;
            const uint64_t who = __ballot(word > cut);
            if (__popcll(who) > 12) {
              best = word_merge(best, word_sort(word));
              const uint64_t last = lane_word(best, K - 1);
              cut = last > cut ? last : cut;
            } else {
              insert(word, who);
            }
          }
        } else {
          // one vector after another, an element to each of eight lanes
          while (lanes) {
            const int from = __builtin_ctzll(lanes);
            lanes &= lanes - 1;
            const int at = j - (tid - (wave * 64 + from)) * 8 + lane;  // (j of that lane, and this lane's element)
            const float x = raw[u].of_lane(from).pick(lane & 7);
            const bool there = lane < 8 && at >= in.first && at < in.hi;
            const uint64_t word = there ? ((uint64_t)order_key(x) << 32) | ~(uint32_t)(at - in.first) : 0;
            insert(word, __ballot(word > cut));
          }
        }
        bound = key_value((uint32_t)((cut + 1) >> 32));
      }
    }
#pragma unroll
    for (int u = 0; u < VECS; ++u) raw[u] = next[u];
  }
  acc.settle();
  float m = acc.m, s = acc.s, e = acc.e;
  if (wave > 0) lists[wave][lane] = best;
  ent_reduce(m, s, e, wm, ws, we);  // (its barrier is the lists')
  if (wave > 0) return;
  for (int w = 1; w < WAVES; ++w) best = word_merge(best, lists[w][lane]);
  const float top = key_value((uint32_t)(lane_word(best, 0) >> 32));
  // a NaN anywhere in the row comes first, then an infinity
  const float l = (top != top || top == INFINITY || top == -INFINITY) ? top : m + logf(s);
  if (lane < K) {
    float v = key_value((uint32_t)(best >> 32));
    if (v != -INFINITY) v = row_logprob(v, m, logf(s));  // a logit of -inf has log probability -inf in every row
    idx[lane] = (int)~(uint32_t)best;
    val[lane] = v;
  }
  if (lane == 0) {
    lse[row] = l;
    row_outputs(out, logits, row, V, l, m, s, e);
  }
}

// ---------------------------------------------------------------- gradient --
// dz = a (1[v = token] - q) - b q (log q + entropy), q = exp(z - lse) (the lse as it
// was rounded: q carries 2^-24 |lse|), for a row's incoming gradients a (log probability) and b (entropy).  A row whose mask is 0,
// whose a and b are 0 or that has no column left (lse = -inf) gets zeros and is
// not read.  One pass; a thread takes VECS vectors of a row, one for short rows.  Bound
// by memory where there are many rows: 2048 x 201088 bf16 282 us, 5.8 TB/s read and
// written (a copy of as much 5.2).
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
  if (top == 0 || logprob_in_registers(V, top)) {
    auto go = [&](auto* p) {
      using E = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
      auto run = [&](auto threads) {
        constexpr int N = decltype(threads)::value;
        if (top == 0)
          row_stats_kernel<E, N><<<(unsigned)rows, N, 0, st>>>(p, (int)V, t.mask, out, lse);
        else
          row_top_kernel<E, N><<<(unsigned)rows, N, 0, st>>>(p, (int)V, top, t.mask, out, lse, idx, val);
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
