// gfx950 kernels of the operators around the distillation loss: the top-K
// teacher cache made from logits, the embedding table tied to the output head
// with its gradient, and activations held in 8 bits with the RMS norm whose
// backward pass reads them.
#include "ckl_ops.hpp"

#include <algorithm>
#include <type_traits>

#include "ckl_common.hpp"

namespace ckl {

namespace {

// ---------------------------------------------------------------- helpers --
// Eight consecutive elements (16-byte aligned) as floats, and back with one
// rounding.
__device__ __forceinline__ void load8(const bf16_t* p, float* f) {
  const u32x4 v = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* f) {
  const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = a[i];
    f[4 + i] = b[i];
  }
}
__device__ __forceinline__ void store8(bf16_t* p, const float* f) {
  *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                       pack_bf16x2(f[6], f[7])};
}
__device__ __forceinline__ void store8(float* p, const float* f) {
  reinterpret_cast<f32x4*>(p)[0] = f32x4{f[0], f[1], f[2], f[3]};
  reinterpret_cast<f32x4*>(p)[1] = f32x4{f[4], f[5], f[6], f[7]};
}
__device__ __forceinline__ void store4(bf16_t* p, f32x4 v) {
  *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}
__device__ __forceinline__ void store4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
// The same without a place in the caches for what is written: for outputs larger
// than they are (embedding of 32768 x 2880: 71 -> 56 us).
__device__ __forceinline__ void stream8(bf16_t* p, const float* f) {
  const u32x4 v = {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
}
__device__ __forceinline__ void stream8(float* p, const float* f) {
  __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4*>(p));
  __builtin_nontemporal_store(f32x4{f[4], f[5], f[6], f[7]}, reinterpret_cast<f32x4*>(p) + 1);
}
// Four elements.
__device__ __forceinline__ void load4(const bf16_t* p, float* f) {
  const u32x2 v = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load4(const float* p, float* f) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = a[i];
}
// Four elements that nothing else will read.
__device__ __forceinline__ void load4_once(const bf16_t* p, float* f) {
  const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load4_once(const float* p, float* f) {
  const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = a[i];
}
// A weight of either type, eight columns.
__device__ __forceinline__ void load8_any(const void* p, int is_bf16, int64_t at, float* f) {
  if (is_bf16)
    load8(reinterpret_cast<const bf16_t*>(p) + at, f);
  else
    load8(reinterpret_cast<const float*>(p) + at, f);
}

__device__ __forceinline__ float wave_sum_f(float x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

// Inclusive sums over the wave, lane by lane.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);  // from 1, 2, 4, 8 lanes below in the row of 16
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // row ends into rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // lane 31 into rows 2 and 3
  return x;
}

// Rows of n units each, cut into runs of consecutive units: the row and column
// of unit base + off, for off below a few thousand and base below 2^40.
struct Units {
  uint32_t n;
  uint64_t m64;  // 2^64 / n rounded up (n > 1): base / n is the high word of base m64
  uint32_t m32;  // the same for 32 bits
};
__device__ __forceinline__ void unit_at(const Units& q, int64_t base, uint32_t off, int64_t* row, uint32_t* col) {
  if (q.n == 1) {
    *row = base + off;
    *col = 0;
    return;
  }
  const uint64_t r0 = __umul64hi((uint64_t)base, q.m64);
  const uint32_t u = (uint32_t)((uint64_t)base - r0 * q.n) + off;
  const uint32_t r = __umulhi(u, q.m32);
  *row = (int64_t)(r0 + r);
  *col = u - r * q.n;
}
Units units(int64_t n) {
  Units q{(uint32_t)n, 0, 0};
  if (n > 1) {
    q.m64 = ~(uint64_t)0 / (uint64_t)n + 1;
    q.m32 = (uint32_t)((((uint64_t)1 << 32) / (uint64_t)n) + 1);
  }
  return q;
}

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
  uint32_t hist[BINS];
  uint32_t wave_n[4];
  uint32_t range[2][4];
  uint32_t pending[2][4];
  float wave_m[4], wave_s[4];
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

// The K largest of a row's n words in order, and its state, as the row's
// results.  The words are put into bins over the range of their keys, and in its
// bin a word's place is the number of larger words there.  Where a bin that
// matters holds more than 256 words (keys that are mostly equal, or a far
// outlier) a bitonic sort does it.  (2048 rows of 100000 bf16, K = 2048: 352 us
// a call with this, 580 with the bitonic sort.)
template <int CAP, typename S>
__device__ __forceinline__ void topk_finish(uint64_t* buf, int n, int K, float m, float s, int logprob, int* idx,
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
  auto put = [&](int place, uint64_t word) {
    float v = key_value((uint32_t)(word >> 32));
    if (logprob && v != -INFINITY) v -= l;  // a logit of -inf has log-probability -inf in every row
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
    return;
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
}

__device__ __forceinline__ void topk_masked_row(int K, int* idx, float* val, float* lse) {
  for (int k = threadIdx.x; k < K; k += kTopkThreads) {
    idx[k] = k;
    val[k] = 0.f;
  }
  if (threadIdx.x == 0) *lse = 0.f;
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
  __device__ __forceinline__ float pick(int i) const {
    const f32x4 w = (i & 4) ? a[1] : a[0];
    const float lo = (i & 1) ? w[1] : w[0], hi = (i & 1) ? w[3] : w[2];
    return (i & 2) ? hi : lo;
  }
};

// What a segment of a row leaves for the merge: up to `slots` words.
__host__ __device__ inline int topk_slots(int K) { return K + K / 8 + 32; }

template <typename T, int CAP>
__global__ __launch_bounds__(kTopkThreads, CAP <= 4096 ? 4 : 2) void topk_rows_kernel(
    const T* __restrict__ logits, int64_t rows, int V, int K, int segments, int seg_cols, int logprob,
    const uint8_t* __restrict__ mask, int* __restrict__ idx, float* __restrict__ val, float* __restrict__ lse,
    uint64_t* __restrict__ cand, float2* __restrict__ state) {
  __shared__ __attribute__((aligned(16))) uint64_t buf[CAP];
  __shared__ TopkShared<CAP <= 4096 ? 256 : 1024> sh;
  __shared__ uint32_t lists[kTopkThreads / 64][kTopkList];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x / segments;
  const int seg = (int)(blockIdx.x - row * segments);
  if (mask != nullptr && mask[row] == 0) {
    if (segments == 1) topk_masked_row(K, idx + row * K, val + row * K, lse + row);
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
  if (fabsf(neg) < kTopkNegLimit && m > -INFINITY) s *= fast_exp2(-fmaf(m, kLog2e, neg));  // the rounding of neg
  topk_reduce_state(m, s, sh);
  if (segments == 1) {
    topk_finish<CAP>(buf, n, K, m, s, logprob, idx + row * K, val + row * K, lse + row, sh);
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
  }
}

// The segments' words of a row, cut and sorted in the same way.
template <int CAP>
__global__ __launch_bounds__(kTopkThreads, CAP <= 4096 ? 4 : 2) void topk_merge_kernel(
    const uint64_t* __restrict__ cand, const float2* __restrict__ state, int K, int segments, int logprob,
    const uint8_t* __restrict__ mask, int* __restrict__ idx, float* __restrict__ val, float* __restrict__ lse) {
  __shared__ __attribute__((aligned(16))) uint64_t buf[CAP];
  __shared__ TopkShared<CAP <= 4096 ? 256 : 1024> sh;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  if (mask != nullptr && mask[row] == 0) {
    topk_masked_row(K, idx + row * K, val + row * K, lse + row);
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
  float m = -INFINITY, s = 0.f;
  for (int i = tid; i < segments; i += kTopkThreads) {
    const float2 st = state[row * segments + i];
    exp_merge(m, s, st.x, st.y);
  }
  topk_reduce_state(m, s, sh);
  topk_finish<CAP>(buf, n, K, m, s, logprob, idx + row * K, val + row * K, lse + row, sh);
}

// ---------------------------------------------------------------- embedding --
// The table's row of a token, V where it is outside [v_offset, v_offset + V).  The
// difference is taken modulo 2^64: v_offset + V fits 63 bits, so no token at
// either end of its type comes out below V.
__device__ __forceinline__ int64_t token_row(int64_t token, int64_t V, int64_t v_offset) {
  const uint64_t v = (uint64_t)token - (uint64_t)v_offset;
  return v < (uint64_t)V ? (int64_t)v : V;
}

// out[t] = scale W[token_t - v_offset]; a zero row for a token outside the table.
// A thread takes four vectors, their tokens and then their rows loaded together.
// Bound by memory: 32768 x 2880 bf16 56 us, 4.6 TB/s.
constexpr int kEmbedUnits = 4;
template <typename T, typename I>
__global__ __launch_bounds__(256) void embedding_forward_kernel(const T* __restrict__ W, int64_t V, int64_t v_offset,
                                                                const I* __restrict__ tokens, int64_t rows, Units q,
                                                                float scale, T* __restrict__ out) {
  const int64_t base = (int64_t)blockIdx.x * (256 * kEmbedUnits);
  int64_t row[kEmbedUnits], v[kEmbedUnits];
  uint32_t col[kEmbedUnits];
#pragma unroll
  for (int k = 0; k < kEmbedUnits; ++k) {
    unit_at(q, base, k * 256 + threadIdx.x, &row[k], &col[k]);
    v[k] = row[k] < rows ? token_row(tokens[row[k]], V, v_offset) : V;
  }
  float f[kEmbedUnits][8];
#pragma unroll
  for (int k = 0; k < kEmbedUnits; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[k][i] = 0.f;
    if (v[k] < V) load8(W + (v[k] * q.n + col[k]) * 8, f[k]);
  }
#pragma unroll
  for (int k = 0; k < kEmbedUnits; ++k) {
    const bool in = v[k] < V;  // (a zero row whatever the scale)
#pragma unroll
    for (int i = 0; i < 8; ++i) f[k][i] = in ? f[k][i] * scale : 0.f;
    if (row[k] < rows) stream8(out + (row[k] * q.n + col[k]) * 8, f[k]);
  }
}

// Gradient: dW[v] = scale sum of dY[t] over the positions t of token v, summed
// in the order of the positions.  The positions are first sorted by token
// (stable, so ascending within a token); tokens outside the table take the key
// V, which sorts last and is never summed.
template <typename I>
__device__ __forceinline__ uint32_t token_key(const I* tokens, int64_t t, int64_t V, int64_t v_offset) {
  return (uint32_t)token_row(tokens[t], V, v_offset);
}

// Zeros, by the workgroups of a launch past its own `first`: the rows of dW that
// no token has are cleared while the positions are being sorted.
struct Fill {
  u32x4* p;
  int64_t n;
  int first;
};
__device__ __forceinline__ bool fill_instead(const Fill& fill) {
  if ((int)blockIdx.x < fill.first) return false;
  const int64_t stride = (int64_t)(gridDim.x - fill.first) * blockDim.x;
  for (int64_t i = (int64_t)(blockIdx.x - fill.first) * blockDim.x + threadIdx.x; i < fill.n; i += stride)
    fill.p[i] = u32x4{0, 0, 0, 0};
  return true;
}

// Very few positions (a prompt): one launch.  Workgroup (t, y) looks for the
// other positions of its token; the first of them adds their rows.  (200 x 2048
// bf16 added to fp32: 4.5 us, ranking and summing in three launches 13.)
constexpr int kFewMax = 256;
template <typename T, typename G, typename I, bool ADD>
__global__ __launch_bounds__(256) void embedding_few_kernel(const T* __restrict__ dY, const I* __restrict__ tokens,
                                                            int n, int64_t V, int64_t v_offset, int nv, float scale,
                                                            G* __restrict__ dW) {
  __shared__ uint64_t masks[kFewMax / 64];
  const int tid = threadIdx.x, t = blockIdx.x;
  const uint32_t k = token_key(tokens, t, V, v_offset);
  const uint64_t same = __ballot(tid < n && token_key(tokens, tid < n ? tid : 0, V, v_offset) == k);
  if ((tid & 63) == 0) masks[tid >> 6] = same;
  const int col = blockIdx.y * 256 + tid;
  const bool in = col < nv && k < V;
  G* dst = dW + ((int64_t)k * nv + col) * 8;
  float sum[8] = {}, old[8] = {};
  if (ADD && in) load8(dst, old);
  __syncthreads();
  if (!in) return;
  for (int w = 0; w < kFewMax / 64; ++w) {
    uint64_t m = masks[w];
    if (w <= t >> 6 && (m & (w == t >> 6 ? ((uint64_t)1 << (t & 63)) - 1 : ~(uint64_t)0))) return;  // not the first
    while (m) {
      float f[4][8];
      int p[4], c = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] = m ? w * 64 + __builtin_ctzll(m) : -1;
        c += m ? 1 : 0;
        m &= m - 1;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < c) load8(dY + ((int64_t)p[j] * nv + col) * 8, f[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < c) {
#pragma unroll
          for (int x = 0; x < 8; ++x) sum[x] += f[j][x];
        }
      }
    }
  }
#pragma unroll
  for (int x = 0; x < 8; ++x) sum[x] = ADD ? old[x] + scale * sum[x] : scale * sum[x];
  store8(dst, sum);
}

// Few positions: each one's rank is counted directly, T^2 comparisons over the
// whole GPU.  A workgroup ranks 16 positions; 64 slices share the keys, 16 at a
// time.  (4099 positions, 64 to a workgroup: 15 us; so, and with the zeros of 64
// MB besides, 11.)
constexpr int kRankMax = 8192;
constexpr int kRankWaves = 16;
constexpr int kRankRows = 16;
template <typename I>
__global__ __launch_bounds__(64 * kRankWaves) void rank_sort_kernel(const I* __restrict__ tokens, int n, int64_t V,
                                                                     int64_t v_offset, uint32_t* __restrict__ key_out,
                                                                     uint32_t* __restrict__ pos_out,
                                                                     uint32_t* __restrict__ joins, Fill fill) {
  __shared__ __attribute__((aligned(16))) uint32_t keys[kRankMax];
  __shared__ int part[kRankWaves][kRankRows];
  if (fill_instead(fill)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int padded = (n + 63) & ~63;
  if (blockIdx.x == 0 && threadIdx.x == 0) *joins = 0;
  for (int i = threadIdx.x; i < padded; i += 64 * kRankWaves)
    keys[i] = i < n ? token_key(tokens, i, V, v_offset) : 0xffffffffu;
  __syncthreads();
  const int t0 = blockIdx.x * kRankRows, t = t0 + (lane & (kRankRows - 1));
  const uint32_t mine = t < n ? keys[t] : 0;
  int less = 0;
  for (int i0 = wave * 64; i0 < padded; i0 += kRankWaves * 64) {
    const int i = i0 + (lane / kRankRows) * 16;
    u32x4 k[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const u32x4*>(keys + i + 4 * j);
    // equal keys count where they come earlier
    if (i0 + 64 <= t0) {
#pragma unroll
      for (int j = 0; j < 16; ++j) less += k[j >> 2][j & 3] <= mine ? 1 : 0;
    } else if (i0 >= t0 + kRankRows) {
#pragma unroll
      for (int j = 0; j < 16; ++j) less += k[j >> 2][j & 3] < mine ? 1 : 0;
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t x = k[j >> 2][j & 3];
        less += (x < mine || (x == mine && i + j < t)) ? 1 : 0;
      }
    }
  }
  less += __shfl_xor(less, 16);
  less += __shfl_xor(less, 32);
  if (lane < kRankRows) part[wave][lane] = less;
  __syncthreads();
  if (threadIdx.x < kRankRows && t < n) {
    int r = 0;
#pragma unroll
    for (int w = 0; w < kRankWaves; ++w) r += part[w][lane];
    key_out[r] = mine;
    pos_out[r] = (uint32_t)t;
  }
}

// Many positions: a stable radix sort, digits of up to 9 bits, a workgroup per
// block of 1024 ROUNDS keys.  hist[block][digit] counts the keys of a block.
// (Counting the next pass's digits while a pass scatters, by atomics, took
// 40 us more than a launch of its own: frequent tokens meet on one counter.)
// 32768 positions, 18 bits of key: two passes of 5 + 5 us, all latency.
constexpr int kSortWaves = 16;
constexpr int kSortBins = 512;

template <typename I, int ROUNDS>
__global__ __launch_bounds__(64 * kSortWaves) void sort_hist_kernel(const I* __restrict__ tokens, int64_t n, int64_t V,
                                                                     int64_t v_offset, int bins, int shift,
                                                                     uint32_t* __restrict__ key,
                                                                     uint32_t* __restrict__ hist,
                                                                     uint32_t* __restrict__ joins, Fill fill) {
  // tokens NULL: the keys are there already
  __shared__ uint32_t h[kSortBins];
  if (fill_instead(fill)) return;
  if (blockIdx.x == 0 && threadIdx.x == 0) *joins = 0;
  if (threadIdx.x < kSortBins) h[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int64_t t = ((int64_t)blockIdx.x * ROUNDS + r) * 1024 + threadIdx.x;
    if (t < n) {
      uint32_t k;
      if (tokens != nullptr)
        key[t] = k = token_key(tokens, t, V, v_offset);
      else
        k = key[t];
      atomicAdd(&h[(k >> shift) & (bins - 1)], 1u);
    }
  }
  __syncthreads();
  if (threadIdx.x < kSortBins) hist[(int64_t)blockIdx.x * kSortBins + threadIdx.x] = h[threadIdx.x];
}

template <int ROUNDS>
__global__ __launch_bounds__(64 * kSortWaves) void sort_scatter_kernel(
    const uint32_t* __restrict__ key_in, const uint32_t* __restrict__ pos_in, int64_t n, int shift, int digit_bits,
    const uint32_t* __restrict__ hist, uint32_t* __restrict__ key_out, uint32_t* __restrict__ pos_out) {
  __shared__ uint32_t cnt[kSortWaves][kSortBins];  // per wave: keys of a digit, then the wave's next place
  __shared__ uint32_t wtot[kSortBins / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int bins = 1 << digit_bits;

  // a wave's keys are consecutive, so waves, rounds and lanes are in order
  uint32_t k[ROUNDS], pos[ROUNDS];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int64_t t = ((int64_t)blockIdx.x * 1024 + wave * 64) * ROUNDS + r * 64 + lane;
    k[r] = t < n ? key_in[t] : 0;
    pos[r] = (t < n && pos_in != nullptr) ? pos_in[t] : (uint32_t)t;
  }
  for (int i = tid; i < kSortWaves * kSortBins; i += 64 * kSortWaves) (&cnt[0][0])[i] = 0;
  uint32_t before = 0, total = 0;
  if (tid < bins) {
    const int blocks = gridDim.x, me = blockIdx.x;
#pragma unroll 16
    for (int b = 0; b < blocks; ++b) {
      const uint32_t c = hist[(int64_t)b * kSortBins + tid];
      total += c;
      before += b < me ? c : 0;
    }
  }
  // exclusive sums of the totals over the digits
  uint32_t inc = total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t v = __shfl_up(inc, o);
    if (lane >= o) inc += v;
  }
  if (wave < kSortBins / 64 && lane == 63) wtot[wave] = inc;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int64_t t = ((int64_t)blockIdx.x * 1024 + wave * 64) * ROUNDS + r * 64 + lane;
    if (t < n) atomicAdd(&cnt[wave][(k[r] >> shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  if (tid < kSortBins) {
    uint32_t at = inc - total + before;
    for (int w = 0; w < wave; ++w) at += wtot[w];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = cnt[w][tid];
      cnt[w][tid] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int64_t t = ((int64_t)blockIdx.x * 1024 + wave * 64) * ROUNDS + r * 64 + lane;
    const bool ok = t < n;
    const uint32_t dgt = (k[r] >> shift) & (bins - 1);
    uint64_t same = __ballot(ok);
#pragma unroll
    for (int b = 0; b < 9; ++b) {  // (bits past digit_bits are zero everywhere)
      const uint64_t one = __ballot((dgt >> b) & 1);
      same &= ((dgt >> b) & 1) ? one : ~one;
    }
    const uint64_t below = same & (((uint64_t)1 << lane) - 1);
    uint32_t at = 0;
    if (ok) at = cnt[wave][dgt] + (uint32_t)__popcll(below);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // all lanes have read before one of each digit adds
    if (ok && below == 0) cnt[wave][dgt] += (uint32_t)__popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (ok) {
      key_out[at] = k[r];
      pos_out[at] = pos[r];
    }
  }
}

// A thread sums four columns over one chunk of the sorted positions, four at a
// time: their rows, and the old gradients of the tokens that end among them,
// are loaded together, so that eight loads are under way instead of one (the
// rows of a token are anywhere in dY).  Runs of one token inside the chunk are
// final; a run that crosses a border leaves its sum in part[chunk][0] (it began
// before the chunk) or part[chunk][1] (it begins here and goes on; the chunk is
// then listed for the join).  Bound by memory: 32768 x 2880 bf16 (an eighth
// padding, word frequencies) added to fp32 95 us, 4.7 TB/s; eight columns a
// thread 106.
constexpr int kSumBatch = 4;
template <typename T, typename G, bool ADD>
__global__ __launch_bounds__(256) void embedding_sum_kernel(const T* __restrict__ dY, const uint32_t* __restrict__ key,
                                                            const uint32_t* __restrict__ pos, int64_t n, int chunk,
                                                            int64_t chunks, Units q, uint32_t V, float scale,
                                                            G* __restrict__ dW, float* __restrict__ part,
                                                            uint32_t* __restrict__ joins) {
  int64_t c;
  uint32_t col;
  unit_at(q, (int64_t)blockIdx.x * 256, threadIdx.x, &c, &col);
  if (c >= chunks) return;
  const int64_t b = c * chunk, e = b + chunk < n ? b + chunk : n;
  bool from_before = b > 0 && key[b - 1] == key[b];
  float sum[4] = {};
  for (int64_t i = b; i < e; i += kSumBatch) {
    uint32_t k[kSumBatch + 1], p[kSumBatch];
    const int m = e - i < kSumBatch ? (int)(e - i) : kSumBatch;
#pragma unroll
    for (int j = 0; j < kSumBatch; ++j) {
      k[j] = j < m ? key[i + j] : 0xffffffffu;
      p[j] = j < m ? pos[i + j] : 0;
    }
    k[kSumBatch] = i + kSumBatch < e ? key[i + kSumBatch] : 0xffffffffu;
    if (k[0] >= V) return;
    float f[kSumBatch][4], old[kSumBatch][4];
#pragma unroll
    for (int j = 0; j < kSumBatch; ++j) {
      if (k[j] < V) load4_once(dY + ((int64_t)p[j] * q.n + col) * 4, f[j]);
      if (ADD && k[j] < V && k[j] != k[j + 1]) load4(dW + ((int64_t)k[j] * q.n + col) * 4, old[j]);
    }
#pragma unroll
    for (int j = 0; j < kSumBatch; ++j) {
      if (k[j] >= V) return;
#pragma unroll
      for (int x = 0; x < 4; ++x) sum[x] += f[j][x];
      if (k[j] != k[j + 1]) {  // the run ends here, or the chunk does
        const bool goes_on = i + j + 1 == e && e < n && key[e] == k[j];
        if (!from_before && !goes_on) {
#pragma unroll
          for (int x = 0; x < 4; ++x) sum[x] = ADD ? old[j][x] + scale * sum[x] : scale * sum[x];
          store4(dW + ((int64_t)k[j] * q.n + col) * 4, f32x4{sum[0], sum[1], sum[2], sum[3]});
        } else {
          store4(part + ((2 * c + (from_before ? 0 : 1)) * (int64_t)q.n + col) * 4,
                 f32x4{sum[0], sum[1], sum[2], sum[3]});
          if (!from_before && col == 0) joins[1 + atomicAdd(joins, 1u)] = (uint32_t)c;
        }
        from_before = false;
#pragma unroll
        for (int x = 0; x < 4; ++x) sum[x] = 0.f;
      }
    }
  }
}

// The runs that cross borders: the listed chunk, where one begins, and the
// chunks that it goes on through.  A workgroup takes 64 vectors of columns of
// one run; four slices share its chunks and are added in order, so the order of
// the list does not matter.  (The same sums 5 us; with the run's end found by
// binary search over the chunks 25.)
template <typename G, bool ADD>
__global__ __launch_bounds__(256) void embedding_join_kernel(const uint32_t* __restrict__ key, int chunk,
                                                             int64_t chunks, int nv, float scale, G* __restrict__ dW,
                                                             const float* __restrict__ part,
                                                             const uint32_t* __restrict__ joins) {
  __shared__ float sums[3][64][9];
  const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
  const int slabs = (nv + 63) / 64;
  const int64_t items = (int64_t)joins[0] * slabs;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t c = joins[1 + it / slabs];
    const int col = (int)(it % slabs) * 64 + lane;
    const uint32_t k = key[(c + 1) * chunk];
    G* dst = dW + ((int64_t)k * nv + col) * 8;
    float sum[8] = {}, old[8] = {};
    if (slice == 0 && col < nv) {
      load8(part + ((2 * c + 1) * (int64_t)nv + col) * 8, sum);
      if (ADD) load8(dst, old);
    }
    // the chunks after c that begin with this token, 64 at a time
    for (int64_t j0 = c + 1; j0 < chunks; j0 += 64) {
      const uint64_t in = __ballot(j0 + lane < chunks && key[(j0 + lane) * chunk] == k);
      const int m = in == ~(uint64_t)0 ? 64 : __builtin_ctzll(~in);
      if (col < nv) {
#pragma unroll 4
        for (int j = slice; j < m; j += 4) {
          float f[8];
          load8(part + (2 * (j0 + j) * (int64_t)nv + col) * 8, f);
#pragma unroll
          for (int x = 0; x < 8; ++x) sum[x] += f[x];
        }
      }
      if (m < 64) break;
    }
    if (slice > 0) {
#pragma unroll
      for (int x = 0; x < 8; ++x) sums[slice - 1][lane][x] = sum[x];
    }
    __syncthreads();
    if (slice == 0 && col < nv) {
#pragma unroll
      for (int s = 0; s < 3; ++s)
#pragma unroll
        for (int x = 0; x < 8; ++x) sum[x] += sums[s][lane][x];
#pragma unroll
      for (int x = 0; x < 8; ++x) sum[x] = ADD ? old[x] + scale * sum[x] : scale * sum[x];
      store8(dst, sum);
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(1024) void zero_kernel(Fill fill) { fill_instead(fill); }

// -------------------------------------------------- 8-bit activations, norm --
// Blocks of 32 columns of a row share a power of two 2^(E - 127), the smallest
// that brings the block's largest magnitude below 127.5, kept within 2^-126 and
// 2^121 (127 steps of a larger one are no float); a code is the value divided
// by it, rounded to the nearest whole number, ties to even, at most 127.
// Multiplying by powers of two is exact, so a code depends on nothing but its
// block, and a restored value (7 bits and a sign) is exact in bf16.
// E = 255 marks a block that holds an infinity or a NaN: all of it restores to
// NaN.
//
// A thread holds eight columns, four neighbouring lanes a block.  Encoding and
// decoding are bound by memory: 131072 x 2880 bf16 192 and 208 us, 6.0 and 5.5 TB/s.
__device__ __forceinline__ uint32_t top_bits(const float* f) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(f[i]) & 0x7fffffffu;  // as integers, NaN > inf > finite
    a = b > a ? b : a;
  }
  return a;
}
__device__ __forceinline__ uint32_t block_exponent(uint32_t top) {
  uint32_t o = __shfl_xor(top, 1);
  top = o > top ? o : top;
  o = __shfl_xor(top, 2);
  top = o > top ? o : top;
  if (top >= 0x7f800000u) return 255;
  // adding 2^16 carries into the exponent exactly when top >= 127.5 / 64 of its power of two
  const int e = (int)((top + 0x10000u) >> 23) - 6;
  return e < 1 ? 1u : e > 248 ? 248u : (uint32_t)e;
}
__device__ __forceinline__ u32x2 encode8(const float* f, uint32_t e) {
  if (e == 255) return u32x2{0, 0};
  const float inv = __uint_as_float((254u - e) << 23);
  u32x2 c = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int v = (int)fminf(fmaxf(rintf(f[i] * inv), -127.f), 127.f);  // past 127 only at E = 248
    c[i >> 2] |= ((uint32_t)v & 255u) << (8 * (i & 3));
  }
  return c;
}
__device__ __forceinline__ float block_step(uint32_t e) {
  return e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(e << 23);
}
__device__ __forceinline__ void decode8(u32x2 c, float step, float* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = (float)(int)(int8_t)(c[i >> 2] >> (8 * (i & 3))) * step;
}

template <typename T>
__global__ __launch_bounds__(256) void act_encode_kernel(const T* __restrict__ x, int64_t rows, int nv, Units q,
                                                         int8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  // q.n = nv rounded up to whole blocks: lanes past nv hold zeros
  const int64_t base = (int64_t)blockIdx.x * 1024;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    int64_t row;
    uint32_t col;
    unit_at(q, base, k * 256 + threadIdx.x, &row, &col);
    float f[8] = {};
    const bool ok = row < rows && (int)col < nv;
    if (ok) load8(x + (row * nv + col) * 8, f);
    const uint32_t e = block_exponent(top_bits(f));
    if (ok) {
      *reinterpret_cast<u32x2*>(codes + (row * nv + col) * 8) = encode8(f, e);
      if ((col & 3) == 0) exps[row * (q.n / 4) + col / 4] = (uint8_t)e;
    }
  }
}

template <typename T, bool NORM>
__global__ __launch_bounds__(256) void act_decode_kernel(const int8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ exps, int64_t rows, Units q,
                                                         const float* __restrict__ rstd,
                                                         const void* __restrict__ weight, int weight_bf16,
                                                         T* __restrict__ out) {
  const int64_t base = (int64_t)blockIdx.x * 1024;
  const int64_t nb = (q.n + 3) / 4;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    int64_t row;
    uint32_t col;
    unit_at(q, base, k * 256 + threadIdx.x, &row, &col);
    if (row >= rows) return;
    const int64_t at = row * q.n + col;
    float f[8];
    decode8(*reinterpret_cast<const u32x2*>(codes + at * 8), block_step(exps[row * nb + col / 4]), f);
    if (NORM) {
      float w[8];
      load8_any(weight, weight_bf16, (int64_t)col * 8, w);
      const float r = rstd[row];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * r * w[i];
    }
    stream8(out + at * 8, f);
  }
}

// Sum over the workgroup, in every thread.  `slots` holds one float per wave.
__device__ __forceinline__ float group_sum(float x, float* slots) {
  x = wave_sum_f(x);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return x;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = x;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < waves; ++w) s += slots[w];
  __syncthreads();
  return s;
}

// y = x rstd weight with rstd = 1 / sqrt(mean x^2 + eps), and x in 8 bits for
// the backward pass.  A workgroup takes a row; a thread holds NV vectors of eight
// columns (vector v of the row in thread v mod blockDim), so that the row is read
// once.  Bound by memory: 32768 x 2880 bf16 85 to 92 us by board, 5.2 to 5.6 TB/s;
// not on rows below 512 columns, where most lanes of the row's wave have nothing
// (262144 x 64: 78 us, 1.1 TB/s).
template <typename T, int NV>
__global__ __launch_bounds__(1024) void norm_forward_kernel(const T* __restrict__ x, int64_t rows, int nv,
                                                            const void* __restrict__ weight, int weight_bf16,
                                                            float eps, T* __restrict__ y, int8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ exps, float* __restrict__ rstd) {
  __shared__ float slots[16];
  const int nb = (nv + 3) / 4;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    float f[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * blockDim.x + threadIdx.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[k][i] = 0.f;
      if (v < nv) load8(x + (row * nv + v) * 8, f[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += f[k][i] * f[k][i];
    }
    ss = group_sum(ss, slots);
    const float r = 1.f / sqrtf(ss / (float)(nv * 8) + eps);
    if (codes != nullptr && threadIdx.x == 0) rstd[row] = r;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * blockDim.x + threadIdx.x;
      const uint32_t e = block_exponent(top_bits(f[k]));
      if (v < nv) {
        const int64_t at = row * nv + v;
        if (codes != nullptr) {
          __builtin_nontemporal_store(encode8(f[k], e), reinterpret_cast<u32x2*>(codes + at * 8));
          if ((v & 3) == 0) exps[row * nb + v / 4] = (uint8_t)e;
        }
        float w[8];
        load8_any(weight, weight_bf16, (int64_t)v * 8, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = f[k][i] * r * w[i];
        stream8(y + at * 8, w);
      }
    }
  }
}

// With x restored from 8 bits and n = x rstd:
//   dx = rstd (dy w - n mean(dy w n)),   dw = sum over rows of dy n.
// A workgroup walks rows blockIdx, blockIdx + gridDim, ... and keeps its
// columns' share of dw in registers; norm_dweight_kernel adds the workgroups.
// Bound by memory: 32768 x 2880 bf16 87 us, 5.5 TB/s.  Not on narrow rows, which
// follow one another without the next one's loads under way (262144 x 64: 86 us,
// 1.0 TB/s), nor on the widest, where four and eight vectors in each of 1024
// threads leave few registers or too few (4096 x 32768: 227 us, 3.0 TB/s; 2048 x
// 65536: 587 us, 1.2 TB/s).
template <typename T, int NV>
__global__ __launch_bounds__(1024) void norm_backward_kernel(const T* __restrict__ dy, int64_t rows, int nv,
                                                             const int8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ exps,
                                                             const float* __restrict__ rstd,
                                                             const void* __restrict__ weight, int weight_bf16,
                                                             T* __restrict__ dx, float* __restrict__ part) {
  __shared__ float slots[16];
  const int nb = (nv + 3) / 4;
  float dw[NV][8] = {};
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float r = rstd[row];
    float n[NV][8], g[NV][8];
    float c = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * blockDim.x + threadIdx.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) n[k][i] = g[k][i] = 0.f;
      if (v < nv) {
        const int64_t at = row * nv + v;
        decode8(*reinterpret_cast<const u32x2*>(codes + at * 8), block_step(exps[row * nb + v / 4]) * r, n[k]);
        load8(dy + at * 8, g[k]);
        float w[8];
        load8_any(weight, weight_bf16, (int64_t)v * 8, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[k][i] += g[k][i] * n[k][i];
          g[k][i] *= w[i];
          c += g[k][i] * n[k][i];
        }
      }
    }
    c = group_sum(c, slots) / (float)(nv * 8);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * blockDim.x + threadIdx.x;
      if (v < nv) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[k][i] = r * (g[k][i] - n[k][i] * c);
        store8(dx + (row * nv + v) * 8, g[k]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = k * blockDim.x + threadIdx.x;
    if (v < nv) store8(part + ((int64_t)blockIdx.x * nv + v) * 8, dw[k]);
  }
}

// The workgroups' shares added: 16 lanes of four columns each and 64 slices of
// the shares, the slices added in a fixed order.  (One thread per eight columns
// walking all 1024 shares took 282 us at d = 2880, on two workgroups; this
// takes 8 us.)
template <typename T>
__global__ __launch_bounds__(1024) void norm_dweight_kernel(const float* __restrict__ part, int groups, int d,
                                                            T* __restrict__ dweight) {
  __shared__ f32x4 sums[64][16];
  const int lane = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int col = (blockIdx.x * 16 + lane) * 4;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  if (col < d) {
#pragma unroll 8
    for (int g = slice; g < groups; g += 64) sum += *reinterpret_cast<const f32x4*>(part + (int64_t)g * d + col);
  }
  sums[slice][lane] = sum;
  __syncthreads();
  if (slice == 0 && col < d) {
#pragma unroll 8
    for (int i = 1; i < 64; ++i) sum += sums[i][lane];
    store4(dweight + col, sum);
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// -------------------------------------------------------------- launchers --
// Segments of whole tiles to a row: as many as make the call shortest when a
// workgroup takes 2 us a tile by itself, all of them together read 2500 columns a
// nanosecond, and joining segments costs 8 us.  (us at bf16, K = 100, in 1 / 2 / 3
// segments: 300 rows of 201088 58 / 50 / 48; 600 rows of 32000 23 / 35 / 34; 600
// rows of 201088 69 / 80 / 80; one row of 201088 51 / 39 / 34, in 25 20.)
// The rule knows neither the type nor K, with which tiles and joining take
// longer.  fp32: 300 rows of 201088 66 in the 3 it takes, 68 whole.  K = 1000: one
// row 49 in 25, 46 in 13; 300 rows 87 in 3, 88 in 2, 96 whole.  It is off at
// K = 4096: one row 140 in 25, 118 in 9; 300 rows 235 in 3, 178 whole.
void topk_plan(int64_t rows, int64_t V, int* segments, int64_t* seg_cols) {
  const int64_t tiles = cdiv(V + 7, kTopkTile);
  const double read_us = (double)rows * V * 2 / 5e6;
  double best = 0;
  *seg_cols = 0;
  for (int64_t want = 1; want <= std::min<int64_t>(tiles, 64); ++want) {
    const int64_t per = cdiv(tiles, want);
    if (cdiv(tiles, per) != want) continue;  // the same as fewer
    const double us = std::max(read_us, 2.0 * per) + (want > 1 ? 8.0 : 0.0);
    if (*seg_cols == 0 || us < best) {
      best = us;
      *seg_cols = per * kTopkTile;
      *segments = (int)want;
    }
  }
}
int64_t topk_segment_words(int64_t K) { return topk_slots((int)K); }

hipError_t launch_teacher_topk(const void* logits, int bf16, int64_t rows, int64_t V, int K, int logprob,
                               const uint8_t* mask, int* idx, float* val, float* lse, uint64_t* cand, float2* state,
                               hipStream_t st) {
  int segments;
  int64_t seg_cols;
  topk_plan(rows, V, &segments, &seg_cols);
  const unsigned blocks = (unsigned)(rows * segments);
  auto go = [&](auto* p, auto cap) {
    using E = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    constexpr int CAP = decltype(cap)::value;
    topk_rows_kernel<E, CAP><<<blocks, kTopkThreads, 0, st>>>(p, rows, (int)V, K, segments, (int)seg_cols, logprob,
                                                              mask, idx, val, lse, cand, state);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || segments == 1) return e;
    topk_merge_kernel<CAP><<<(unsigned)rows, kTopkThreads, 0, st>>>(cand, state, K, segments, logprob, mask, idx, val,
                                                                   lse);
    return hipGetLastError();
  };
  // room for what a cut may leave and 2048 more words, and for the final sort
  using Small = std::integral_constant<int, 4096>;
  using Large = std::integral_constant<int, 8192>;
  if (bf16) return K <= 1024 ? go((const bf16_t*)logits, Small{}) : go((const bf16_t*)logits, Large{});
  return K <= 1024 ? go((const float*)logits, Small{}) : go((const float*)logits, Large{});
}

hipError_t launch_embedding_forward(const void* W, int bf16, int64_t V, int d, int64_t v_offset, const void* tokens,
                                    int tokens64, int64_t T, float scale, void* out, hipStream_t st) {
  const Units q = units(d / 8);
  const unsigned blocks = (unsigned)cdiv(T * q.n, 256 * kEmbedUnits);
  auto go = [&](auto* w, auto* tok) {
    using E = std::remove_const_t<std::remove_pointer_t<decltype(w)>>;
    embedding_forward_kernel<<<blocks, 256, 0, st>>>(w, V, v_offset, tok, T, q, scale, (E*)out);
  };
  if (bf16 && tokens64) go((const bf16_t*)W, (const int64_t*)tokens);
  if (bf16 && !tokens64) go((const bf16_t*)W, (const int32_t*)tokens);
  if (!bf16 && tokens64) go((const float*)W, (const int64_t*)tokens);
  if (!bf16 && !tokens64) go((const float*)W, (const int32_t*)tokens);
  return hipGetLastError();
}

EmbedWs embed_ws(int64_t T, int64_t V, int64_t d) {
  EmbedWs w{};
  if (T <= kFewMax) return w;  // (no workspace)
  size_t o = 0;
  auto take = [&](size_t bytes) {
    size_t at = o;
    o += (bytes + 255) & ~(size_t)255;
    return at;
  };
  // Long chunks leave few borders to join, short ones enough waves: the longest
  // with 4096 of them, four to a SIMD.  (32768 x 2880 added to fp32, chunks of 16
  // / 32 / 64: 125 / 129 / 117 us; 16384 x 2880 81 / 71 / 71; 12000 x 768 42 / 51.)
  for (w.chunk = 64; w.chunk > 8 && cdiv(T, w.chunk) * (d / 4) < 4096 * 64; w.chunk /= 2) {}
  w.chunks = cdiv(T, w.chunk);
  if (T > kRankMax) {
    int bits = 1;
    while (((int64_t)1 << bits) <= V) ++bits;  // keys 0 .. V
    w.passes = (int)cdiv(bits, 9);
    w.digit_bits = (int)cdiv(bits, w.passes);
    // a scattering workgroup adds up the counts of all blocks: few of them
    w.sort_rounds = T <= 65536 ? 1 : 4;
    w.sort_blocks = cdiv(T, 1024 * w.sort_rounds);
  }
  w.key0 = take(T * 4);
  w.pos0 = take(T * 4);
  if (w.passes) {
    w.key1 = take(T * 4);
    w.pos1 = take(T * 4);
    w.hist = take((size_t)w.sort_blocks * kSortBins * 4);
  }
  w.joins = take((size_t)(1 + w.chunks) * 4);
  w.part = take((size_t)2 * w.chunks * d * 4);
  w.total = o;
  return w;
}

template <bool ADD, typename T, typename G>
static hipError_t embedding_reduce(const T* dY, int64_t n, int d, int64_t V, float scale, G* dW, const EmbedWs& w,
                                   char* ws, const uint32_t* key, const uint32_t* pos, hipStream_t st) {
  const Units q = units(d / 4);
  float* part = (float*)(ws + w.part);
  uint32_t* joins = (uint32_t*)(ws + w.joins);
  embedding_sum_kernel<T, G, ADD><<<(unsigned)cdiv(w.chunks * q.n, 256), 256, 0, st>>>(
      dY, key, pos, n, (int)w.chunk, w.chunks, q, (uint32_t)V, scale, dW, part, joins);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || w.chunks < 2) return e;
  const int nv = d / 8;
  const int64_t most = (w.chunks - 1) * cdiv(nv, 64);
  embedding_join_kernel<G, ADD><<<(unsigned)std::min<int64_t>(most, 2048), 256, 0, st>>>(
      key, (int)w.chunk, w.chunks, nv, scale, dW, part, joins);
  return hipGetLastError();
}

// Workgroups of 1024 threads for n 16-byte words of zeros.
static unsigned fill_blocks(int64_t n) { return (unsigned)std::min<int64_t>(cdiv(n, 4096), 2048); }

template <int ROUNDS, typename I>
static hipError_t embedding_radix(const I* tokens, int64_t T, int64_t V, int64_t v_offset, const EmbedWs& w, char* ws,
                                  Fill fill, const uint32_t** key, const uint32_t** pos, hipStream_t st) {
  uint32_t* k[2] = {(uint32_t*)(ws + w.key0), (uint32_t*)(ws + w.key1)};
  uint32_t* p[2] = {(uint32_t*)(ws + w.pos0), (uint32_t*)(ws + w.pos1)};
  uint32_t* hist = (uint32_t*)(ws + w.hist);
  const unsigned blocks = (unsigned)w.sort_blocks, threads = 64 * kSortWaves;
  for (int i = 0; i < w.passes; ++i) {
    const int from = i & 1, shift = i * w.digit_bits;
    fill.first = (int)blocks;
    sort_hist_kernel<I, ROUNDS><<<blocks + (i ? 0 : fill_blocks(fill.n)), threads, 0, st>>>(
        i ? nullptr : tokens, T, V, v_offset, 1 << w.digit_bits, shift, k[from], hist, (uint32_t*)(ws + w.joins),
        fill);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    sort_scatter_kernel<ROUNDS><<<blocks, threads, 0, st>>>(k[from], i ? p[from] : nullptr, T, shift, w.digit_bits,
                                                            hist, k[from ^ 1], p[from ^ 1]);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  *key = k[w.passes & 1];
  *pos = p[w.passes & 1];
  return hipSuccess;
}

template <typename I>
static hipError_t embedding_sort(const I* tokens, int64_t T, int64_t V, int64_t v_offset, const EmbedWs& w, char* ws,
                                 Fill fill, const uint32_t** key, const uint32_t** pos, hipStream_t st) {
  if (w.passes)
    return w.sort_rounds == 1 ? embedding_radix<1>(tokens, T, V, v_offset, w, ws, fill, key, pos, st)
                              : embedding_radix<4>(tokens, T, V, v_offset, w, ws, fill, key, pos, st);
  *key = (uint32_t*)(ws + w.key0);
  *pos = (uint32_t*)(ws + w.pos0);
  fill.first = (int)cdiv(T, kRankRows);
  rank_sort_kernel<<<(unsigned)fill.first + fill_blocks(fill.n), 64 * kRankWaves, 0, st>>>(
      tokens, (int)T, V, v_offset, (uint32_t*)(ws + w.key0), (uint32_t*)(ws + w.pos0), (uint32_t*)(ws + w.joins),
      fill);
  return hipGetLastError();
}

hipError_t launch_embedding_backward(const void* dY, int bf16, int64_t T, int d, const void* tokens, int tokens64,
                                     int64_t V, int64_t v_offset, float scale, void* dW, int dw_bf16, int accumulate,
                                     char* ws, hipStream_t st) {
  const Fill fill{(u32x4*)dW, accumulate ? 0 : V * d * (dw_bf16 ? 2 : 4) / 16, 0};
  hipError_t e;
  if (T <= kFewMax && fill.n > 0) {
    zero_kernel<<<fill_blocks(fill.n), 1024, 0, st>>>(fill);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (T == 0) return hipSuccess;
  if (T <= kFewMax) {
    const dim3 grid((unsigned)T, (unsigned)cdiv(d / 8, 256));
    auto go = [&](auto* dy, auto* tok, auto* dw) {
      using A = std::remove_const_t<std::remove_pointer_t<decltype(dy)>>;
      using I = std::remove_const_t<std::remove_pointer_t<decltype(tok)>>;
      using G = std::remove_pointer_t<decltype(dw)>;
      if (accumulate)
        embedding_few_kernel<A, G, I, true><<<grid, 256, 0, st>>>(dy, tok, (int)T, V, v_offset, d / 8, scale, dw);
      else
        embedding_few_kernel<A, G, I, false><<<grid, 256, 0, st>>>(dy, tok, (int)T, V, v_offset, d / 8, scale, dw);
    };
    auto with_dw = [&](auto* dy, auto* tok) { dw_bf16 ? go(dy, tok, (bf16_t*)dW) : go(dy, tok, (float*)dW); };
    auto with_tok = [&](auto* dy) {
      tokens64 ? with_dw(dy, (const int64_t*)tokens) : with_dw(dy, (const int32_t*)tokens);
    };
    bf16 ? with_tok((const bf16_t*)dY) : with_tok((const float*)dY);
    return hipGetLastError();
  }
  const EmbedWs w = embed_ws(T, V, d);
  const uint32_t *key, *pos;
  if (tokens64)
    e = embedding_sort((const int64_t*)tokens, T, V, v_offset, w, ws, fill, &key, &pos, st);
  else
    e = embedding_sort((const int32_t*)tokens, T, V, v_offset, w, ws, fill, &key, &pos, st);
  if (e != hipSuccess) return e;
  auto go = [&](auto* dy, auto* dw) {
    return accumulate ? embedding_reduce<true>(dy, T, d, V, scale, dw, w, ws, key, pos, st)
                      : embedding_reduce<false>(dy, T, d, V, scale, dw, w, ws, key, pos, st);
  };
  if (bf16) return dw_bf16 ? go((const bf16_t*)dY, (bf16_t*)dW) : go((const bf16_t*)dY, (float*)dW);
  return dw_bf16 ? go((const float*)dY, (bf16_t*)dW) : go((const float*)dY, (float*)dW);
}

hipError_t launch_act_encode(const void* x, int bf16, int64_t T, int d, int8_t* codes, uint8_t* exps, hipStream_t st) {
  const int nv = d / 8;
  const Units q = units(cdiv(nv, 4) * 4);
  const unsigned blocks = (unsigned)cdiv(T * q.n, 1024);
  if (bf16)
    act_encode_kernel<<<blocks, 256, 0, st>>>((const bf16_t*)x, T, nv, q, codes, exps);
  else
    act_encode_kernel<<<blocks, 256, 0, st>>>((const float*)x, T, nv, q, codes, exps);
  return hipGetLastError();
}

hipError_t launch_act_decode(const int8_t* codes, const uint8_t* exps, int64_t T, int d, const float* rstd,
                             const void* weight, int weight_bf16, void* out, int out_bf16, hipStream_t st) {
  const Units q = units(d / 8);
  const unsigned blocks = (unsigned)cdiv(T * q.n, 1024);
  auto go = [&](auto* o) {
    using E = std::remove_pointer_t<decltype(o)>;
    if (rstd)
      act_decode_kernel<E, true><<<blocks, 256, 0, st>>>(codes, exps, T, q, rstd, weight, weight_bf16, o);
    else
      act_decode_kernel<E, false><<<blocks, 256, 0, st>>>(codes, exps, T, q, rstd, weight, weight_bf16, o);
  };
  if (out_bf16)
    go((bf16_t*)out);
  else
    go((float*)out);
  return hipGetLastError();
}

template <int N>
using Count = std::integral_constant<int, N>;

// Threads and vectors per thread for rows of nv vectors.  Two vectors a thread
// have the loads in flight that one has in twice the threads, and half the waves
// to wait for at the row's sum.  (32768 x 2880 bf16, forward: one vector in 384
// threads 110 us, two in 192 85, three in 128 91, six in 64 110; backward 134,
// 98, 101, 308.)  More than two where a workgroup's 1024 threads need it.
static void norm_shape(int nv, int* threads, int* per) {
  *per = nv <= 64 ? 1 : nv <= 2048 ? 2 : nv <= 4096 ? 4 : 8;
  *threads = (int)cdiv(cdiv(nv, *per), 64) * 64;
}

hipError_t launch_norm_forward(const void* x, int bf16, int64_t T, int d, const void* weight, int weight_bf16,
                               float eps, void* y, int8_t* codes, uint8_t* exps, float* rstd, hipStream_t st) {
  const int nv = d / 8;
  int threads, per;
  norm_shape(nv, &threads, &per);
  const unsigned blocks = (unsigned)T;
  auto go = [&](auto* p) {
    using E = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    auto run = [&](auto n) {
      norm_forward_kernel<E, decltype(n)::value>
          <<<blocks, threads, 0, st>>>(p, T, nv, weight, weight_bf16, eps, (E*)y, codes, exps, rstd);
    };
    per == 1 ? run(Count<1>{}) : per == 2 ? run(Count<2>{}) : per == 4 ? run(Count<4>{}) : run(Count<8>{});
  };
  if (bf16)
    go((const bf16_t*)x);
  else
    go((const float*)x);
  return hipGetLastError();
}

// Sixteen waves on each of the 256 compute units.  (32768 x 2880: 3 / 4 / 5 / 6 /
// 8 workgroups of three waves a unit 121 / 103 / 98 / 99 / 115 us.)
int64_t norm_backward_groups(int64_t T, int64_t d) {
  int threads, per;
  norm_shape((int)(d / 8), &threads, &per);
  return std::min<int64_t>(T, 256 * std::max(1, 1024 / threads));
}

hipError_t launch_norm_backward(const void* dy, int bf16, int64_t T, int d, const int8_t* codes, const uint8_t* exps,
                                const float* rstd, const void* weight, int weight_bf16, void* dx, void* dweight,
                                float* part, hipStream_t st) {
  const int nv = d / 8;
  int threads, per;
  norm_shape(nv, &threads, &per);
  const unsigned groups = (unsigned)norm_backward_groups(T, d);
  auto go = [&](auto* p) {
    using E = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    auto run = [&](auto n) {
      norm_backward_kernel<E, decltype(n)::value>
          <<<groups, threads, 0, st>>>(p, T, nv, codes, exps, rstd, weight, weight_bf16, (E*)dx, part);
    };
    per == 1 ? run(Count<1>{}) : per == 2 ? run(Count<2>{}) : per == 4 ? run(Count<4>{}) : run(Count<8>{});
  };
  if (groups > 0) {
    if (bf16)
      go((const bf16_t*)dy);
    else
      go((const float*)dy);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const unsigned blocks = (unsigned)cdiv(d, 64);
  if (weight_bf16)
    norm_dweight_kernel<<<blocks, 1024, 0, st>>>(part, (int)groups, d, (bf16_t*)dweight);
  else
    norm_dweight_kernel<<<blocks, 1024, 0, st>>>(part, (int)groups, d, (float*)dweight);
  return hipGetLastError();
}

}  // namespace ckl
