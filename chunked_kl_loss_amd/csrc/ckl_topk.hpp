// Device code of the top-K of rows of logits (see the section's comment).
#pragma once

#include <type_traits>

#include "ckl_vec.hpp"

namespace ckl {

namespace {

// ------------------------------------------------------------ teacher top-K --
// Per row of logits: the K largest in descending order (equal values: the lower
// index first), and log sum exp of the whole row.
//
// One pass over the row.  An element is a 64-bit word: a key that orders the
// values as unsigned integers (NaN largest, -0 = +0) above the inverted index,
// so that larger words come first and no two are equal.  A workgroup walks its
// segment of the row in tiles of 8192 columns held in registers.  From the
// first it takes a key with at least K elements at or above it, found by
// counting the keys of a range in 256 bins; from then on only elements above
// that key are wanted: those with the very key come later than K others and
// lose.  A vector of eight whose maximum is wanted is put on its wave's list;
// when lists fill up, their vectors are read again, one to a lane, and what is
// wanted of them goes into a buffer in shared memory.  (Taking elements where
// they are found costs each wave three times the common path's instructions
// for one lane's sake: 245 us against 170 at 2048 x 201088.)  A filling buffer
// is cut as the first tile was, which raises the key.  Where too many elements
// share one key for a cut by keys, a radix selection over the words decides by
// index.  What remains is sorted.  The common path, per vector of eight: eight
// exponentials, one running maximum and one comparison.
//
// Bound by memory where there are many rows: 2048 x 201088 bf16, K = 100, 168 us
// or 4.9 TB/s (four workgroups to a compute unit, the next tile's loads under
// way while one is looked at).  For one row the steps' latency counts: 32000
// columns 17 us, of which 3 for the first key, 2 a tile, 2.5 for the order.
constexpr int kTopkThreads = 256;
constexpr int kTopkVecs = 4;                                 // vectors of eight a thread holds
constexpr int kTopkStep = kTopkThreads * 8;                  // columns of one vector each
constexpr int kTopkTile = kTopkVecs * kTopkStep;
constexpr int kTopkList = 64 * kTopkVecs + 64;               // vectors on a wave's list: a tile's, and 64
constexpr uint32_t kNanKey = 0xfffffffeu;                    // every key lies below 2^32 - 1
// Exponentials are taken as 2^(x log2 e + neg) with neg = -m log2 e rounded, and
// the rounding is divided out of their sum later.  Below this limit it is at
// most half of neg's last place, 4, so both factors are ordinary numbers (past 2^31
// they may overflow).  Larger references, which only masks have, take
// 2^((x - m) log2 e).
constexpr float kTopkNegLimit = 1e8f;

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return kNanKey;
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 + 0 = +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
// (keys that no number has, above that of infinity and below that of -infinity,
// give NaNs)
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <int BINS>
struct TopkShared {
  static constexpr int bins = BINS;  // of the final order; 256 serve everything else
  __attribute__((aligned(16))) uint32_t hist[BINS];
  uint32_t wave_n[4];
  uint32_t range[2][4];
  uint32_t pending[2][4];
  float wave_m[4], wave_s[4], wave_e[4];
  uint32_t count, sel, need, bin;
  uint32_t start[BINS + 1];
};

// Places for a lane's `mine` words behind those in the buffer: one addition to
// the counter a wave.
template <typename S>
__device__ __forceinline__ int topk_place(int mine, S& sh) {
  const int inc = wave_scan(mine);
  int at = 0;
  if ((threadIdx.x & 63) == 63) at = (int)atomicAdd(&sh.count, (uint32_t)inc);
  return __builtin_amdgcn_readlane(at, 63) + inc - mine;
}

// The extremes of a value over the workgroup.
template <typename S>
__device__ __forceinline__ void topk_range(uint32_t& lo, uint32_t& hi, S& sh) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t a = __shfl_xor(lo, o), b = __shfl_xor(hi, o);
    lo = a < lo ? a : lo;
    hi = b > hi ? b : hi;
  }
  if ((threadIdx.x & 63) == 0) {
    sh.range[0][threadIdx.x >> 6] = lo;
    sh.range[1][threadIdx.x >> 6] = hi;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t a = sh.range[0][w], b = sh.range[1][w];
    lo = a < lo ? a : lo;
    hi = b > hi ? b : hi;
  }
}

// A key t in [lo, hi) that at least K elements reach: count(t) >= K.  The range
// is counted in 256 bins and narrowed to one of them until count(t) <= limit or
// it holds one key only; *n = count(t).  No element reaches hi; at_lo =
// count(lo), or more.  each(f) calls f for a thread's keys.  All threads call
// it, after a barrier behind the last use of sh.
template <typename E, typename S>
__device__ __forceinline__ uint32_t topk_select(E each, uint32_t lo, uint32_t hi, int at_lo, int K, int limit, S& sh,
                                                int* n) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t above = 0;  // elements that reach hi
  while (at_lo > limit && hi - lo > 1) {
    const int bits = 32 - __clz((int)(hi - lo - 1)), shift = bits > 8 ? bits - 8 : 0;
    sh.hist[tid] = 0;
    __syncthreads();
    each([&](uint32_t k) {
      if (k >= lo && k < hi) atomicAdd(&sh.hist[(k - lo) >> shift], 1u);
    });
    __syncthreads();
    // suffix sums: thread b holds the elements that reach bin b
    const uint32_t own = sh.hist[tid];
    uint32_t suf = (uint32_t)wave_scan((int)own);
    const uint32_t in_wave = (uint32_t)__builtin_amdgcn_readlane((int)suf, 63);
    suf = in_wave - suf + own;
    if (lane == 0) sh.wave_n[wave] = in_wave;
    __syncthreads();
    suf += above;
    for (int w = wave + 1; w < 4; ++w) suf += sh.wave_n[w];
    if (suf >= (uint32_t)K && suf - own < (uint32_t)K) {
      sh.sel = (uint32_t)tid;
      sh.need = suf;
      sh.bin = own;
    }
    __syncthreads();
    lo += sh.sel << shift;
    if (hi - lo > (1u << shift)) hi = lo + (1u << shift);  // (the last bin may end past 2^32)
    at_lo = (int)sh.need;
    above = sh.need - sh.bin;
  }
  *n = at_lo;
  return lo;
}

// Cuts the n > K words of buf to exactly the K largest, by radix selection:
// where keys are equal the index decides.  In any order; begins and ends with a
// barrier.
template <typename S>
__device__ __forceinline__ void topk_cut_exact(uint64_t* buf, int n, int K, S& sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint64_t prefix = 0, pmask = 0;
  uint32_t need = (uint32_t)K;
  __syncthreads();
  for (int shift = 56; shift >= 0; shift -= 8) {
    sh.hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kTopkThreads) {
      const uint64_t c = buf[i];
      if ((c & pmask) == prefix) atomicAdd(&sh.hist[(uint32_t)(c >> shift) & 255u], 1u);
    }
    __syncthreads();
    // suffix sums over the bins: thread b holds the words in bins >= b
    const uint32_t own = sh.hist[tid];
    uint32_t suf = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t v = __shfl_down(suf, o);
      if (lane + o < 64) suf += v;
    }
    if (lane == 0) sh.wave_n[wave] = suf;
    __syncthreads();
    for (int w = wave + 1; w < 4; ++w) suf += sh.wave_n[w];
    if (suf >= need && suf - own < need) {
      sh.sel = (uint32_t)tid;
      sh.need = need - (suf - own);
      sh.bin = own;
    }
    __syncthreads();
    prefix |= (uint64_t)sh.sel << shift;
    pmask |= (uint64_t)255u << shift;
    need = sh.need;
    if (sh.bin == need) break;  // the whole bin is kept
  }
  if (tid == 0) sh.count = 0;
  // in place: the words kept so far never reach past the words read so far
  for (int i0 = 0; i0 < n; i0 += kTopkThreads) {
    const int i = i0 + tid;
    const uint64_t c = i < n ? buf[i] : 0;
    __syncthreads();
    if (i < n && (c & pmask) >= prefix) buf[atomicAdd(&sh.count, 1u)] = c;
  }
  __syncthreads();
}

// Cuts the n > limit >= K words of buf to at most `limit` of the largest, at
// least K, in any order.  Returns their number and sets *key to a key that at
// least K of them, and none but them, reach.  Begins and ends with a barrier.
// (3000 words to 1000: 5 us.)
template <int CAP, typename S>
__device__ __forceinline__ int topk_cut(uint64_t* buf, int n, int K, int limit, S& sh, uint32_t* key) {
  const int tid = threadIdx.x;
  const uint32_t* keys = reinterpret_cast<const uint32_t*>(buf) + 1;
  __syncthreads();
  uint32_t least = ~0u, most = 0;
#pragma unroll 4
  for (int i = tid; i < n; i += kTopkThreads) {
    const uint32_t k = keys[2 * i];
    most = k > most ? k : most;
    least = k < least ? k : least;
  }
  topk_range(least, most, sh);
  int kept;
  const uint32_t t = topk_select(
      [&](auto f) {
#pragma unroll 4
        for (int i = tid; i < n; i += kTopkThreads) f(keys[2 * i]);
      },
      least, most + 1, n, K, limit, sh, &kept);
  *key = t;
  if (kept > limit) {
    topk_cut_exact(buf, n, K, sh);
    return K;
  }
  constexpr int W = CAP / kTopkThreads;
  const int lane = tid & 63, wave = tid >> 6;
  uint64_t c[W];
  int mine = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    c[w] = w * kTopkThreads + tid < n ? buf[w * kTopkThreads + tid] : 0;
    mine += (uint32_t)(c[w] >> 32) >= t ? 1 : 0;
  }
  const int inc = wave_scan(mine);
  if (lane == 63) sh.wave_n[wave] = (uint32_t)inc;
  __syncthreads();  // also: all words have been read
  int at = inc - mine;
  for (int w = 0; w < wave; ++w) at += (int)sh.wave_n[w];
#pragma unroll
  for (int w = 0; w < W; ++w)
    if ((uint32_t)(c[w] >> 32) >= t) buf[at++] = c[w];
  if (tid == 0) sh.count = (uint32_t)kept;
  __syncthreads();
  return kept;
}

// The value of lane ^ LANES.
template <int LANES>
__device__ __forceinline__ uint32_t lane_xor(uint32_t x) {
  if constexpr (LANES == 1) return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xb1, 0xf, 0xf, true);  // quad 1 0 3 2
  if constexpr (LANES == 2) return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4e, 0xf, 0xf, true);  // quad 2 3 0 1
  if constexpr (LANES == 4) {  // from 4 above in banks 0 and 2 of a row, from 4 below in the others
    const int up = __builtin_amdgcn_update_dpp((int)x, (int)x, 0x104, 0xf, 0x5, false);
    return (uint32_t)__builtin_amdgcn_update_dpp(up, (int)x, 0x114, 0xf, 0xa, false);
  }
  if constexpr (LANES == 8)  // the row of 16 turned by 8
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x128, 0xf, 0xf, true);
  return (uint32_t)__shfl_xor((int)x, LANES);
}

// Descending bitonic sort of n words, W to a thread: partners are in the same
// thread, in the same wave, or (the largest distances) in another wave, where
// they meet in buf.  n <= W kTopkThreads, which fit buf.
template <int W>
__device__ __forceinline__ void topk_sort_bitonic(uint64_t* buf, int n) {
  const int tid = threadIdx.x;
  uint64_t x[W];
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) x[w] = tid * W + w < n ? buf[tid * W + w] : 0;
  __syncthreads();
#pragma unroll 1
  for (int size = 2; size <= W * kTopkThreads; size <<= 1) {
#pragma unroll 1
    for (int stride = size >> 1; stride >= W; stride >>= 1) {
      const int lanes = stride / W;
      // the larger word goes first where the block of `size` words is an even
      // one, and to the lower partner there
      const bool keep_max = ((tid & lanes) == 0) == (((tid * W) & size) == 0);
      auto exchange = [&](auto partner) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const uint64_t y = partner(w);
          if ((x[w] < y) == keep_max) x[w] = y;
        }
      };
      auto by_lane = [&](auto l) {
        exchange([&](int w) {
          return (uint64_t)lane_xor<decltype(l)::value>((uint32_t)(x[w] >> 32)) << 32 |
                 lane_xor<decltype(l)::value>((uint32_t)x[w]);
        });
      };
      switch (lanes) {
        case 1: by_lane(std::integral_constant<int, 1>{}); break;
        case 2: by_lane(std::integral_constant<int, 2>{}); break;
        case 4: by_lane(std::integral_constant<int, 4>{}); break;
        case 8: by_lane(std::integral_constant<int, 8>{}); break;
        case 16: by_lane(std::integral_constant<int, 16>{}); break;
        case 32: by_lane(std::integral_constant<int, 32>{}); break;
        default:
#pragma unroll
          for (int w = 0; w < W; ++w) buf[w * kTopkThreads + tid] = x[w];
          __syncthreads();
          exchange([&](int w) { return buf[w * kTopkThreads + (tid ^ lanes)]; });
          __syncthreads();
      }
    }
    // within the thread
#pragma unroll
    for (int b = W / 2; b > 0; b >>= 1) {
      if (b < size) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
          if ((w & b) == 0) {
            const uint64_t u = x[w], v = x[w | b];
            const bool swap = (u < v) == (((tid * W + w) & size) == 0);
            x[w] = swap ? v : u;
            x[w | b] = swap ? u : v;
          }
        }
      }
    }
  }
#pragma unroll
  for (int w = 0; w < W; ++w) buf[tid * W + w] = x[w];
  __syncthreads();
}

// Merge of two (reference m, sum of exp(x - m)) states.
__device__ __forceinline__ void exp_merge(float& m, float& s, float m2, float s2) {
  const float mn = fmaxf(m, m2);
  if (mn == -INFINITY) {
    s += s2;  // zero, or NaN
    return;
  }
  s = s * fast_exp2((m - mn) * kLog2e) + s2 * fast_exp2((m2 - mn) * kLog2e);
  m = mn;
}

// The workgroup's log-sum-exp state, in every thread.
template <typename S>
__device__ __forceinline__ void topk_reduce_state(float& m, float& s, S& sh) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float m2 = __shfl_xor(m, o), s2 = __shfl_xor(s, o);
    exp_merge(m, s, m2, s2);
  }
  if ((threadIdx.x & 63) == 0) {
    sh.wave_m[threadIdx.x >> 6] = m;
    sh.wave_s[threadIdx.x >> 6] = s;
  }
  __syncthreads();
  m = sh.wave_m[0];
  s = sh.wave_s[0];
  for (int w = 1; w < 4; ++w) exp_merge(m, s, sh.wave_m[w], sh.wave_s[w]);
}

// Log probability of a logit from its row's reference m and ln s.  (z - (m + ln s)
// would carry the rounding of a sum of m's size: 5e-4 for logits near 10^4.)
__device__ __forceinline__ float row_logprob(float z, float m, float ln_s) { return (z - m) - ln_s; }

// The K largest of a row's n words in order, and its state, as the row's
// results.  The words are put into bins over the range of their keys, and in its
// bin a word's place is the number of larger words there.  Where a bin that
// matters holds more than 256 words (keys that are mostly equal, or a far
// outlier) a bitonic sort does it.  Returns the log sum exp.  (2048 rows of 100000 bf16, K = 2048: 352 us
// a call with this, 580 with the bitonic sort.)  ENT: log probabilities are taken
// from differences (see row_logprob).
template <int CAP, bool ENT, typename S>
__device__ __forceinline__ float topk_finish(uint64_t* buf, int n, int K, float m, float s, int logprob, int* idx,
                                            float* val, float* lse, S& sh) {
  constexpr int W = CAP <= 4096 ? 10 : 24, limit = W * kTopkThreads;  // words that go into the bins
  constexpr int per = S::bins / kTopkThreads;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t key;
  if (n > limit) n = topk_cut<CAP>(buf, n, K, limit, sh, &key);
  __syncthreads();
#pragma unroll
  for (int b = 0; b < per; ++b) sh.hist[b * kTopkThreads + tid] = 0;
  if (tid == 0) sh.bin = 0;
  const uint32_t* keys = reinterpret_cast<const uint32_t*>(buf) + 1;
  uint32_t least = ~0u, most = 0;
#pragma unroll 4
  for (int i = tid; i < n; i += kTopkThreads) {
    const uint32_t k = keys[2 * i];
    most = k > most ? k : most;
    least = k < least ? k : least;
  }
  topk_range(least, most, sh);
  const float top = key_value(most);
  // a NaN anywhere in the row comes first, then an infinity
  const float l = (top != top || top == INFINITY || top == -INFINITY) ? top : m + logf(s);
  if (tid == 0) *lse = l;
  const float ln_s = ENT ? logf(s) : 0.f;
  auto put = [&](int place, uint64_t word) {
    float v = key_value((uint32_t)(word >> 32));
    if (logprob && v != -INFINITY) v = ENT ? row_logprob(v, m, ln_s) : v - l;  // a logit of -inf has log-probability -inf in every row
    idx[place] = (int)~(uint32_t)word;
    val[place] = v;
  };
  constexpr int bin_bits = S::bins == 256 ? 8 : 10;
  const int bits = 32 - __clz((int)((most - least) | 1)), shift = bits > bin_bits ? bits - bin_bits : 0;
#pragma unroll 4
  for (int i = tid; i < n; i += kTopkThreads) atomicAdd(&sh.hist[(most - keys[2 * i]) >> shift], 1u);
  __syncthreads();
  uint32_t own[per], all = 0;
#pragma unroll
  for (int b = 0; b < per; ++b) all += own[b] = sh.hist[tid * per + b];
  const uint32_t inc = (uint32_t)wave_scan((int)all);
  if (lane == 63) sh.wave_n[wave] = inc;
  __syncthreads();
  uint32_t at = inc - all;
  for (int w = 0; w < wave; ++w) at += sh.wave_n[w];
#pragma unroll
  for (int b = 0; b < per; ++b) {
    sh.start[tid * per + b] = at;
    sh.hist[tid * per + b] = at;  // the bin's next place
    if (own[b] > 256 && at < (uint32_t)K) sh.bin = 1;
    at += own[b];
  }
  if (tid == kTopkThreads - 1) sh.start[S::bins] = (uint32_t)n;
  uint64_t x[W];
#pragma unroll
  for (int w = 0; w < W; ++w) x[w] = w * kTopkThreads + tid < n ? buf[w * kTopkThreads + tid] : 0;
  __syncthreads();
  if (sh.bin) {
    if (n > 2048 && K <= 2048) n = topk_cut<CAP>(buf, n, K, 2048, sh, &key);
    if (n <= 2048)
      topk_sort_bitonic<8>(buf, n);
    else if constexpr (CAP > 4096)
      topk_sort_bitonic<CAP / kTopkThreads>(buf, n);
    for (int k = tid; k < K; k += kTopkThreads) put(k, buf[k]);
    return l;
  }
#pragma unroll
  for (int w = 0; w < W; ++w)
    if (w * kTopkThreads + tid < n) buf[atomicAdd(&sh.hist[(most - (uint32_t)(x[w] >> 32)) >> shift], 1u)] = x[w];
  if (tid < 4) buf[n + tid] = 0;
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < n; i += kTopkThreads) {
    const uint64_t word = buf[i];
    const uint32_t b = (most - (uint32_t)(word >> 32)) >> shift;
    const int from = (int)sh.start[b], to = (int)sh.start[b + 1];
    if (from >= K) break;  // (the words lie bin by bin)
    int p = from;
#pragma unroll 1
    for (int j = from; j < to; j += 4) {  // (what lies behind the bin is smaller)
#pragma unroll
      for (int k = 0; k < 4; ++k) p += buf[j + k] > word ? 1 : 0;
    }
    if (p < K) put(p, word);
  }
  return l;
}

__device__ __forceinline__ void topk_masked_row(int K, int* idx, float* val, float* lse) {
  for (int k = threadIdx.x; k < K; k += kTopkThreads) {
    idx[k] = k;
    val[k] = 0.f;
  }
  if (threadIdx.x == 0) *lse = 0.f;
}

// ------------------------------------------- a row's sums for its entropy --
// (m, s, e): a reference m, s = sum of 2^a and e = sum of a 2^a with a = (x - m)
// log2 e, of which log sum exp x = m + ln s and the entropy = ln s - ln 2 e / s.
// A shift of the reference by D (base 2) makes e' = 2^D (e + D s).
constexpr float kExpZero = -1e4f;  // 2^a is zero from here on, and its product with a too
__device__ __forceinline__ void ent_merge(float& m, float& s, float& e, float m2, float s2, float e2) {
  const float mn = fmaxf(m, m2);
  const float d1 = m == mn ? 0.f : fmaxf((m - mn) * kLog2e, kExpZero);  // (equal infinities have no difference)
  const float d2 = m2 == mn ? 0.f : fmaxf((m2 - mn) * kLog2e, kExpZero);
  const float f1 = fast_exp2(d1), f2 = fast_exp2(d2);
  e = f1 * (e + d1 * s) + f2 * (e2 + d2 * s2);
  s = f1 * s + f2 * s2;
  m = mn;
}
// What a thread gathers.  The reference moves only when it falls behind by 4 (a
// few times a row): the terms of e are then at most 6 times those of s, which
// costs the entropy at most 6 roundings of 2^-24.  Exponentials are taken with
// neg = -m log2 e rounded, as above.
struct RowAcc {
  float m = -INFINITY, neg = 0.f, s = 0.f, e = 0.f;
  // divides out the rounding of neg
  __device__ __forceinline__ void settle() {
    if (fabsf(neg) < kTopkNegLimit && m > -INFINITY) {
      const float off = fmaf(m, kLog2e, neg), f = fast_exp2(-off);
      e = f * (e - off * s);
      s *= f;
    }
  }
  // eight elements of maximum vm; returns the sum of their exponentials
  template <typename R>
  __device__ __forceinline__ float add(const R& raw, float vm) {
    if (vm > m + 4.f) {
      const float to = -vm * kLog2e;
      if (m > -INFINITY) {
        settle();
        // (what is there takes the new neg's rounding, which will be divided out of it with the rest)
        const float d = fmaxf((m - vm) * kLog2e, kExpZero) + (fabsf(to) < kTopkNegLimit ? fmaf(vm, kLog2e, to) : 0.f);
        const float f = fast_exp2(d);
        e = f * (e + d * s);
        s *= f;
      }
      m = vm;
      neg = to;
    }
    float sum = 0.f, es = 0.f;
    if (fabsf(neg) < kTopkNegLimit) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = fmaf(raw.get(i), kLog2e, neg), u = fast_exp2(a);
        sum += u;
        es = fmaf(u, a, es);
      }
      if (es != es) {  // (0 times an infinite a: -inf and masks of the lowest value; or a NaN)
        es = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = fmaf(raw.get(i), kLog2e, neg);
          es = fmaf(fast_exp2(a), fmaxf(a, kExpZero), es);
        }
      }
    } else {  // masks of a large or the lowest value, infinities
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = raw.get(i), a = x == m ? 0.f : (x - m) * kLog2e, u = fast_exp2(a);
        sum += u;
        es = fmaf(u, fmaxf(a, kExpZero), es);
      }
    }
    s += sum;
    e += es;
    return sum;
  }
};
// The sums of the whole workgroup, in every thread.
__device__ __forceinline__ void ent_reduce(float& m, float& s, float& e, float* wm, float* ws, float* we) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float m2 = __shfl_xor(m, o), s2 = __shfl_xor(s, o), e2 = __shfl_xor(e, o);
    ent_merge(m, s, e, m2, s2, e2);
  }
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    wm[wave] = m;
    ws[wave] = s;
    we[wave] = e;
  }
  __syncthreads();
  m = wm[0];
  s = ws[0];
  e = we[0];
  for (int w = 1; w < (int)(blockDim.x >> 6); ++w) ent_merge(m, s, e, wm[w], ws[w], we[w]);
}
// What a row of logits leaves besides its alternatives, by one thread: the log
// probability of its token (0 where the token is no column) and its entropy.  l:
// the row's log sum exp, with (m, s, e) its sums.
struct RowOut {
  const void* tokens;
  int tokens64;
  float* logprob;
  float* entropy;
  float* state_e;  // of row segments
};
__device__ __forceinline__ int64_t token_at(const void* tokens, int tokens64, int64_t i) {
  return tokens64 ? reinterpret_cast<const int64_t*>(tokens)[i] : (int64_t)reinterpret_cast<const int32_t*>(tokens)[i];
}
template <typename T>
__device__ __forceinline__ void row_outputs(const RowOut& o, const T* logits, int64_t row, int V, float l, float m,
                                            float s, float e) {
  const int64_t tok = token_at(o.tokens, o.tokens64, row);
  const float ln_s = logf(s);
  float lp = 0.f;
  if (tok >= 0 && tok < V) {
    const float z = (float)logits[row * (int64_t)V + tok];
    lp = z == -INFINITY && l == l ? z : row_logprob(z, m, ln_s);  // (a logit of -inf has log probability -inf in every row)
  }
  float ent = ln_s - kLn2 * (e / s);
  ent = ent < 0.f ? 0.f : ent;
  if (l == -INFINITY) ent = 0.f;             // no column is left
  if (!(l < INFINITY)) ent = __uint_as_float(0x7fc00000u);
  o.logprob[row] = lp;
  o.entropy[row] = ent;
}

// Eight columns as they are in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16_t> {
  u32x4 a;
  __device__ __forceinline__ void load(const bf16_t* p) { a = *reinterpret_cast<const u32x4*>(p); }
  __device__ __forceinline__ void clear() { a = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ void from(const float* f) {
    a = u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
  }
  __device__ __forceinline__ float get(int i) const {
    return (i & 1) ? __uint_as_float(a[i >> 1] & 0xffff0000u) : __uint_as_float(a[i >> 1] << 16);
  }
  // one lane's, in all of them
  __device__ __forceinline__ Raw8 of_lane(int lane) const {
    Raw8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.a[i] = (uint32_t)__builtin_amdgcn_readlane((int)a[i], lane);
    return r;
  }
  // (i not known at compile time)
  __device__ __forceinline__ float pick(int i) const {
    const uint32_t lo = (i & 2) ? a[1] : a[0], hi = (i & 2) ? a[3] : a[2];
    const uint32_t w = (i & 4) ? hi : lo;
    return __uint_as_float((i & 1) ? w & 0xffff0000u : w << 16);
  }
};
template <>
struct Raw8<float> {
  f32x4 a[2];
  __device__ __forceinline__ void load(const float* p) {
    a[0] = reinterpret_cast<const f32x4*>(p)[0];
    a[1] = reinterpret_cast<const f32x4*>(p)[1];
  }
  __device__ __forceinline__ void clear() { a[0] = a[1] = f32x4{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ void from(const float* f) {
    a[0] = f32x4{f[0], f[1], f[2], f[3]};
    a[1] = f32x4{f[4], f[5], f[6], f[7]};
  }
  __device__ __forceinline__ float get(int i) const { return a[i >> 2][i & 3]; }
  __device__ __forceinline__ Raw8 of_lane(int lane) const {
    Raw8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      r.a[i >> 2][i & 3] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(a[i >> 2][i & 3]), lane));
    return r;
  }
  __device__ __forceinline__ float pick(int i) const {
    const bool up = i & 4, odd = i & 1;
    const float p = up ? a[1][0] : a[0][0], q = up ? a[1][1] : a[0][1];
    const float r = up ? a[1][2] : a[0][2], t = up ? a[1][3] : a[0][3];
    return (i & 2) ? (odd ? t : r) : (odd ? q : p);
  }
};

// What a segment of a row leaves for the merge: up to `slots` words.
__host__ __device__ inline int topk_slots(int K) { return K + K / 8 + 32; }

// ENT: the rows' entropies and the log probabilities of given tokens besides.
template <typename T, int CAP, bool ENT = false>
__global__ __launch_bounds__(kTopkThreads, CAP <= 4096 ? 4 : 2) void topk_rows_kernel(
    const T* __restrict__ logits, int64_t rows, int V, int K, int segments, int seg_cols, int logprob,
    const uint8_t* __restrict__ mask, int* __restrict__ idx, float* __restrict__ val, float* __restrict__ lse,
    uint64_t* __restrict__ cand, float2* __restrict__ state, RowOut out) {
  __shared__ __attribute__((aligned(16))) uint64_t buf[CAP];
  __shared__ TopkShared<CAP <= 4096 ? 256 : 1024> sh;
  __shared__ uint32_t lists[kTopkThreads / 64][kTopkList];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x / segments;
  const int seg = (int)(blockIdx.x - row * segments);
  if (mask != nullptr && mask[row] == 0) {
    if (segments == 1) {
      topk_masked_row(K, idx + row * K, val + row * K, lse + row);
      if (ENT && tid == 0) out.logprob[row] = out.entropy[row] = 0.f;
    }
    return;
  }
  // Columns shifted so that shifted column 0 lies on a 16-byte boundary (rows
  // of an odd V begin anywhere).
  const T* p = logits + row * (int64_t)V;
  const int shift = (int)(((uintptr_t)p & 15u) / sizeof(T));
  const T* base = p - shift;
  const int lo = seg * seg_cols, first = lo > shift ? lo : shift;
  const int hi = (lo + seg_cols < V + shift) ? lo + seg_cols : V + shift;
  const int mid_limit = K + K / 4 + 64;  // what a cut on the way may leave: at most CAP - kTopkStep
  const int cut_at = 2 * mid_limit < CAP - 1024 ? 2 * mid_limit : CAP - 1024;

  // columns that can be read: a few past the row where other rows follow
  const int64_t rest = (rows - row) * V;
  const int end = shift + (int)(rest < V + 8 ? rest : V + 8);
  // The vector at shifted column j, with -infinity outside [first, hi).
  auto fetch = [&](int j) {
    Raw8<T> r;
    if (j + 8 <= hi && j >= first) {
      r.load(base + j);
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = -INFINITY;
      if (j < hi) {
        if (j + 8 <= end) {
          load8(base + j, f);  // (a row's neighbours in memory; the first row begins on a boundary)
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = j + i < end ? (float)base[j + i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = j + i >= first && j + i < hi ? f[i] : -INFINITY;
      }
      r.from(f);
    }
    return r;
  };
  uint32_t need = 0;  // keys from here on are wanted
  float need_value = key_value(0);
  // which of a vector's elements are wanted; need_value is a NaN where need is
  // no number's key, and all vectors are looked at
  auto wanted = [&](const Raw8<T>& r, int j) {
    int hits = 0;
    if (need_value != need_value) {
#pragma unroll
      for (int i = 0; i < 8; ++i) hits |= order_key(r.get(i)) >= need ? 1 << i : 0;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) hits |= !(r.get(i) < need_value) ? 1 << i : 0;
    }
    if (j < first || j + 8 > hi) {
#pragma unroll
      for (int i = 0; i < 8; ++i) hits &= j + i >= first && j + i < hi ? -1 : ~(1 << i);
    }
    return hits;
  };

  Raw8<T> raw[kTopkVecs], next[kTopkVecs];
  // sum of 2^(x log2 e + neg), neg = -m log2 e rounded, for a reference m
  float m = -INFINITY, neg = 0.f, s = 0.f;
  RowAcc acc;  // (ENT: instead of them)
  int n = 0, listed = 0, side = 0;
  uint32_t after = 0;  // what is wanted at least once all lists are read
  for (int t0 = lo - kTopkTile; t0 < hi; t0 += kTopkTile) {
    const bool last = t0 + kTopkTile >= hi;
    if (!last) {
#pragma unroll
      for (int u = 0; u < kTopkVecs; ++u) next[u] = fetch(t0 + kTopkTile + u * kTopkStep + tid * 8);
    }
    if (t0 >= lo) {
#pragma unroll
      for (int u = 0; u < kTopkVecs; ++u) {
        float vm = raw[u].get(0), sum = 0.f;
#pragma unroll
        for (int i = 1; i < 8; ++i) vm = fmaxf(vm, raw[u].get(i));
        if constexpr (ENT) {
          sum = acc.add(raw[u], vm);
        } else {
          // The reference moves only when it falls behind by 40: terms up to e^40
          // are as precise and cannot overflow.
          if (vm > m + 40.f) {
            const float to = -vm * kLog2e;
            s *= fast_exp2((m - vm) * kLog2e);
            if (fabsf(neg) < kTopkNegLimit && m > -INFINITY) s *= fast_exp2(-fmaf(m, kLog2e, neg));  // the old neg's rounding
            m = vm;
            neg = to;
          }
          if (fabsf(neg) < kTopkNegLimit) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += fast_exp2(fmaf(raw[u].get(i), kLog2e, neg));
          } else {  // masks of a large or the lowest value, infinities
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += fast_exp2((raw[u].get(i) - m) * kLog2e);
          }
          s += sum;
        }
        // (NaN: fmaxf passes it over, the sum does not)
        const bool hot = !(vm < need_value) || sum != sum;
        const uint64_t who = __ballot(hot);
        if (who) {
          if (hot)
            lists[wave][listed + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32),
                                                           __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0))] =
                (uint32_t)((t0 + u * kTopkStep) / 8 + tid);
          listed += __popcll(who);
        }
      }
      if (lane == 0) sh.pending[side][wave] = (uint32_t)listed;
      __syncthreads();  // (the other side is written only after everyone has passed the next barrier)
      uint32_t most = 0;
#pragma unroll
      for (int w = 0; w < kTopkThreads / 64; ++w) most = sh.pending[side][w] > most ? sh.pending[side][w] : most;
      side ^= 1;
      if (most > kTopkList - 64 * kTopkVecs || last) {
        uint32_t key;
#pragma unroll 1
        for (int i0 = 0; i0 < (int)most; i0 += 64) {
          int hits = 0, j = 0;
          Raw8<T> r;
          r.clear();
          if (i0 + lane < listed) {
            j = (int)lists[wave][i0 + lane] * 8;
            r = fetch(j);
            hits = wanted(r, j);
          }
          int inc = wave_scan(__popc(hits));
          if (lane == 63) sh.pending[side][wave] = (uint32_t)inc;
          __syncthreads();
          int at = n + inc - __popc(hits), all = 0;
#pragma unroll
          for (int w = 0; w < kTopkThreads / 64; ++w) {
            const int c = (int)sh.pending[side][w];
            all += c;
            at += w < wave ? c : 0;
          }
          side ^= 1;
          if (n + all > CAP) {
            // (elements with this very key may still be on the lists with lower indices)
            const int before = n;
            n = topk_cut<CAP>(buf, n, K, mid_limit, sh, &key);
            at -= before - n;
            need = key > need ? key : need;
            after = key + 1 > after ? key + 1 : after;
            need_value = key_value(need);
          }
          n += all;
          while (hits) {
            const int i = __ffs(hits) - 1;
            hits &= hits - 1;
            buf[at++] = ((uint64_t)order_key(r.pick(i)) << 32) | ~(uint32_t)(j - shift + i);
          }
        }
        listed = 0;
        // words above the key come at a rate that the key's age sets: the
        // buffer is cut when it holds twice what a cut leaves
        if (n > cut_at && !last) {
          n = topk_cut<CAP>(buf, n, K, mid_limit, sh, &key);
          after = key + 1 > after ? key + 1 : after;
        }
        need = after > need ? after : need;
        need_value = key_value(need);
      }
    }
#pragma unroll
    for (int u = 0; u < kTopkVecs; ++u) raw[u] = next[u];
    if (t0 < lo) {
      // the first tile's key: what is wanted of that tile, and `after` of the rest
      const int to = hi < lo + kTopkTile ? hi : lo + kTopkTile, total = to - first;
      if (total > mid_limit) {
        uint32_t key[kTopkVecs * 8];  // 0 outside the row
        uint32_t most = 0, least_vec = ~0u, least = ~0u;
#pragma unroll
        for (int u = 0; u < kTopkVecs; ++u) {
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int j = lo + u * kTopkStep + tid * 8 + i;
            const uint32_t k = j >= first && j < hi ? order_key(raw[u].get(i)) : 0;
            key[u * 8 + i] = k;
            top = k > top ? k : top;
            least = k != 0 && k < least ? k : least;
          }
          most = top > most ? top : most;
          least_vec = top != 0 && top < least_vec ? top : least_vec;
        }
        // the least of K or more maxima (of the threads, of the vectors that
        // hold any of the row) is reached by K elements; so is the least element
        const int vecs = (to - lo + 7) / 8, busy = vecs < kTopkThreads ? vecs : kTopkThreads;
        uint32_t from = K <= busy ? (most != 0 ? most : ~0u) : K <= vecs ? least_vec : least;
        topk_range(from, most, sh);
        int got;
        need = topk_select(
            [&](auto f) {
#pragma unroll
              for (int e = 0; e < kTopkVecs * 8; ++e) f(key[e]);
            },
            from, most + 1, total, K, mid_limit, sh, &got);
        after = need + 1;
        need_value = key_value(need);
      }
      __syncthreads();
    }
  }
  float e = 0.f;
  if constexpr (ENT) {
    acc.settle();
    m = acc.m;
    s = acc.s;
    e = acc.e;
    ent_reduce(m, s, e, sh.wave_m, sh.wave_s, sh.wave_e);
  } else {
    if (fabsf(neg) < kTopkNegLimit && m > -INFINITY) s *= fast_exp2(-fmaf(m, kLog2e, neg));  // the rounding of neg
    topk_reduce_state(m, s, sh);
  }
  if (segments == 1) {
    const float l = topk_finish<CAP, ENT>(buf, n, K, m, s, logprob, idx + row * K, val + row * K, lse + row, sh);
    if (ENT && tid == 0) row_outputs(out, logits, row, V, l, m, s, e);
  } else {
    const int slots = topk_slots(K);
    if (n > slots) {
      uint32_t key;
      n = topk_cut<CAP>(buf, n, K, slots, sh, &key);
    }
    __syncthreads();
    uint64_t* c = cand + (int64_t)blockIdx.x * slots;
    for (int k = tid; k < slots; k += kTopkThreads) c[k] = k < n ? buf[k] : 0;
    if (tid == 0) state[blockIdx.x] = make_float2(m, s);
    if (ENT && tid == 0) out.state_e[blockIdx.x] = e;
  }
}

// The segments' words of a row, cut and sorted in the same way.
template <typename T, int CAP, bool ENT = false>
__global__ __launch_bounds__(kTopkThreads, CAP <= 4096 ? 4 : 2) void topk_merge_kernel(
    const uint64_t* __restrict__ cand, const float2* __restrict__ state, int K, int segments, int logprob,
    const uint8_t* __restrict__ mask, int* __restrict__ idx, float* __restrict__ val, float* __restrict__ lse,
    const T* __restrict__ logits, int V, RowOut out) {
  __shared__ __attribute__((aligned(16))) uint64_t buf[CAP];
  __shared__ TopkShared<CAP <= 4096 ? 256 : 1024> sh;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  if (mask != nullptr && mask[row] == 0) {
    topk_masked_row(K, idx + row * K, val + row * K, lse + row);
    if (ENT && tid == 0) out.logprob[row] = out.entropy[row] = 0.f;
    return;
  }
  const int total = segments * topk_slots(K);
  const uint64_t* c = cand + row * total;
  if (tid == 0) sh.count = 0;
  __syncthreads();
  uint32_t need = 1;  // (empty slots are zero)
  int n = 0;
  for (int t0 = 0; t0 < total; t0 += kTopkStep) {
    if (n > CAP - kTopkStep) {
      // (the words of a segment are in no order, so one with this very key may
      // still come with a lower index)
      n = topk_cut<CAP>(buf, n, K, K + K / 4 + 64, sh, &need);
    }
    uint64_t w[8];
    int hits = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = t0 + i * kTopkThreads + tid;
      w[i] = at < total ? c[at] : 0;
      hits += (uint32_t)(w[i] >> 32) >= need ? 1 : 0;
    }
    int at = topk_place(hits, sh);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((uint32_t)(w[i] >> 32) >= need) buf[at++] = w[i];
    __syncthreads();
    n = (int)sh.count;
    __syncthreads();
  }
  float m = -INFINITY, s = 0.f, e = 0.f;
  for (int i = tid; i < segments; i += kTopkThreads) {
    const float2 st = state[row * segments + i];
    if constexpr (ENT)
      ent_merge(m, s, e, st.x, st.y, out.state_e[row * segments + i]);
    else
      exp_merge(m, s, st.x, st.y);
  }
  if constexpr (ENT)
    ent_reduce(m, s, e, sh.wave_m, sh.wave_s, sh.wave_e);
  else
    topk_reduce_state(m, s, sh);
  const float l = topk_finish<CAP, ENT>(buf, n, K, m, s, logprob, idx + row * K, val + row * K, lse + row, sh);
  if (ENT && tid == 0) row_outputs(out, logits, row, V, l, m, s, e);
}

}  // namespace

}  // namespace ckl
