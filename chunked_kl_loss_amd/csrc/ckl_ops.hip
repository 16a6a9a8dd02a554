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
// segment in tiles; elements above the threshold go into a buffer in shared
// memory, and when a further tile might not fit, the buffer is cut to its K
// best and the threshold becomes the K-th key.  Later elements with that very
// key have higher indices than all kept, so they lose and a strict comparison
// is enough.  The log-sum-exp runs along (maximum and sum per thread).
constexpr int kTopkThreads = 256;
constexpr int kTopkTile = kTopkThreads * 8;

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 + 0 = +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k == 0xffffffffu) return __uint_as_float(0x7fc00000u);
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

struct TopkShared {
  uint32_t hist[256];
  uint32_t wave_n[4];
  float wave_m[4], wave_s[4];
  uint32_t count, sel, need, bin, min_key;
};

// Cuts the n > K words of buf to the K largest, in any order, and returns the
// smallest of their keys.  All threads of the workgroup call it; it begins and
// ends with a barrier.
__device__ uint32_t topk_cut(uint64_t* buf, int n, int K, TopkShared& sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint64_t prefix = 0, pmask = 0;
  uint32_t need = (uint32_t)K;
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
  if (tid == 0) {
    sh.count = 0;
    sh.min_key = 0xffffffffu;
  }
  // in place: the words kept so far never reach past the words read so far
  for (int i0 = 0; i0 < n; i0 += kTopkThreads) {
    const int i = i0 + tid;
    const uint64_t c = i < n ? buf[i] : 0;
    __syncthreads();
    if (i < n && (c & pmask) >= prefix) {
      buf[atomicAdd(&sh.count, 1u)] = c;
      atomicMin(&sh.min_key, (uint32_t)(c >> 32));
    }
  }
  __syncthreads();
  return sh.min_key;
}

// Descending bitonic sort of the first n <= cap words (padded with zeros up to
// a power of two, which must fit the buffer).
__device__ void topk_sort(uint64_t* buf, int n) {
  int p = 1;
  while (p < n) p <<= 1;
  for (int i = n + (int)threadIdx.x; i < p; i += kTopkThreads) buf[i] = 0;
  __syncthreads();
  for (int size = 2; size <= p; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      for (int i = threadIdx.x; i < p / 2; i += kTopkThreads) {
        const int a = 2 * i - (i & (stride - 1)), b = a + stride;
        const uint64_t x = buf[a], y = buf[b];
        const bool down = (a & size) == 0;
        if ((x < y) == down) {
          buf[a] = y;
          buf[b] = x;
        }
      }
      __syncthreads();
    }
  }
}

// Merge of two (maximum, sum of exp(x - maximum)) states.
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
__device__ __forceinline__ void topk_reduce_state(float& m, float& s, TopkShared& sh) {
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
  __syncthreads();
}

// The sorted words of a row and its state, as the row's results.
__device__ void topk_write(const uint64_t* buf, int K, float m, float s, int logprob, int* idx, float* val,
                           float* lse) {
  const float top = key_value((uint32_t)(buf[0] >> 32));
  float l;
  if (top != top)
    l = top;  // a NaN anywhere in the row comes first
  else if (top == INFINITY || top == -INFINITY)
    l = top;
  else
    l = m + logf(s);
  for (int k = threadIdx.x; k < K; k += kTopkThreads) {
    const uint64_t c = buf[k];
    float v = key_value((uint32_t)(c >> 32));
    if (logprob && v != -INFINITY) v -= l;  // a logit of -inf has log-probability -inf in every row
    idx[k] = (int)~(uint32_t)c;
    val[k] = v;
  }
  if (threadIdx.x == 0) *lse = l;
}

__device__ __forceinline__ void topk_masked_row(int K, int* idx, float* val, float* lse) {
  for (int k = threadIdx.x; k < K; k += kTopkThreads) {
    idx[k] = k;
    val[k] = 0.f;
  }
  if (threadIdx.x == 0) *lse = 0.f;
}

template <typename T, int CAP>
__global__ __launch_bounds__(kTopkThreads) void topk_rows_kernel(const T* __restrict__ logits, int64_t V, int K,
                                                                 int segments, int64_t seg_cols, int logprob,
                                                                 const uint8_t* __restrict__ mask,
                                                                 int* __restrict__ idx, float* __restrict__ val,
                                                                 float* __restrict__ lse, uint64_t* __restrict__ cand,
                                                                 float2* __restrict__ state) {
  __shared__ __attribute__((aligned(16))) uint64_t buf[CAP];
  __shared__ TopkShared sh;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / segments;
  const int seg = (int)(blockIdx.x - row * segments);
  if (mask != nullptr && mask[row] == 0) {
    if (segments == 1) topk_masked_row(K, idx + row * K, val + row * K, lse + row);
    return;
  }
  // Columns shifted so that shifted column 0 lies on a 16-byte boundary (rows
  // of an odd V begin anywhere).
  const T* p = logits + row * V;
  const int shift = (int)(((uintptr_t)p & 15u) / sizeof(T));
  const T* base = p - shift;
  const int64_t lo = (int64_t)seg * seg_cols;
  const int64_t hi = (lo + seg_cols < V + shift) ? lo + seg_cols : V + shift;

  if (tid == 0) sh.count = 0;
  __syncthreads();
  uint32_t thr = 0;
  float m = -INFINITY, s = 0.f;
  for (int64_t t0 = lo; t0 < hi; t0 += kTopkTile) {
    const int64_t j = t0 + tid * 8;
    float x[8];
    int in = 0;
    if (j >= shift && j + 8 <= hi) {
      load8(base + j, x);
      in = 255;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool ok = j + i >= shift && j + i < hi;
        x[i] = ok ? (float)base[j + i] : -INFINITY;
        in |= ok ? 1 << i : 0;
      }
    }
    float vm = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) vm = fmaxf(vm, x[i]);
    if (vm > m) {
      s *= fast_exp2((m - vm) * kLog2e);
      m = vm;
    }
    if (m > -INFINITY) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s += fast_exp2((x[i] - m) * kLog2e);
    }
    int hits = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) hits |= order_key(x[i]) > thr ? 1 << i : 0;
    hits &= in;
    if (hits) {
      uint32_t at = atomicAdd(&sh.count, (uint32_t)__popc(hits));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (hits & (1 << i)) buf[at++] = ((uint64_t)order_key(x[i]) << 32) | ~(uint32_t)(j + i - shift);
    }
    __syncthreads();
    const int n = (int)sh.count;
    __syncthreads();
    if (n > CAP - kTopkTile) thr = topk_cut(buf, n, K, sh);
  }
  const int n = (int)sh.count;
  __syncthreads();
  if (n > K) topk_cut(buf, n, K, sh);
  topk_reduce_state(m, s, sh);
  if (segments == 1) {
    topk_sort(buf, K);
    topk_write(buf, K, m, s, logprob, idx + row * K, val + row * K, lse + row);
  } else {
    uint64_t* c = cand + (int64_t)blockIdx.x * K;
    for (int k = tid; k < K; k += kTopkThreads) c[k] = k < n ? buf[k] : 0;
    if (tid == 0) state[blockIdx.x] = make_float2(m, s);
  }
}

// The segments' words of a row, cut to the K best in the same way.
template <int CAP>
__global__ __launch_bounds__(kTopkThreads) void topk_merge_kernel(const uint64_t* __restrict__ cand,
                                                                  const float2* __restrict__ state, int K,
                                                                  int segments, int logprob,
                                                                  const uint8_t* __restrict__ mask,
                                                                  int* __restrict__ idx, float* __restrict__ val,
                                                                  float* __restrict__ lse) {
  __shared__ __attribute__((aligned(16))) uint64_t buf[CAP];
  __shared__ TopkShared sh;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  if (mask != nullptr && mask[row] == 0) {
    topk_masked_row(K, idx + row * K, val + row * K, lse + row);
    return;
  }
  const uint64_t* c = cand + row * segments * K;
  const int total = segments * K;
  if (tid == 0) sh.count = 0;
  __syncthreads();
  uint64_t floor_word = 0;
  for (int t0 = 0; t0 < total; t0 += kTopkTile) {
    for (int i = t0 + tid; i < total && i < t0 + kTopkTile; i += kTopkThreads) {
      const uint64_t w = c[i];
      if (w > floor_word) buf[atomicAdd(&sh.count, 1u)] = w;
    }
    __syncthreads();
    const int n = (int)sh.count;
    __syncthreads();
    // words of the K-th key itself may still be needed: segments come in index
    // order, but the words of one segment do not
    if (n > CAP - kTopkTile) floor_word = (uint64_t)topk_cut(buf, n, K, sh) << 32;
  }
  const int n = (int)sh.count;
  __syncthreads();
  if (n > K) topk_cut(buf, n, K, sh);
  float m = -INFINITY, s = 0.f;
  for (int i = tid; i < segments; i += kTopkThreads) exp_merge(m, s, state[row * segments + i].x, state[row * segments + i].y);
  topk_reduce_state(m, s, sh);
  topk_sort(buf, K);
  topk_write(buf, K, m, s, logprob, idx + row * K, val + row * K, lse + row);
}

// ---------------------------------------------------------------- embedding --
// out[t] = scale W[token_t - v_offset]; a zero row for a token outside the table.
template <typename T, typename I>
__global__ __launch_bounds__(256) void embedding_forward_kernel(const T* __restrict__ W, int64_t V, int64_t v_offset,
                                                                const I* __restrict__ tokens, int64_t rows, Units q,
                                                                float scale, T* __restrict__ out) {
  const int64_t base = (int64_t)blockIdx.x * 1024;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    int64_t row;
    uint32_t col;
    unit_at(q, base, k * 256 + threadIdx.x, &row, &col);
    if (row >= rows) return;
    const int64_t v = (int64_t)tokens[row] - v_offset;
    float f[8] = {};
    if (v >= 0 && v < V) {
      load8(W + (v * q.n + col) * 8, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= scale;
    }
    store8(out + (row * q.n + col) * 8, f);
  }
}

// Gradient: dW[v] = scale sum of dY[t] over the positions t of token v, summed
// in the order of the positions.  The positions are first sorted by token
// (stable, so ascending within a token); tokens outside the table take the key
// V, which sorts last and is never summed.
template <typename I>
__device__ __forceinline__ uint32_t token_key(const I* tokens, int64_t t, int64_t V, int64_t v_offset) {
  const int64_t v = (int64_t)tokens[t] - v_offset;
  return (v >= 0 && v < V) ? (uint32_t)v : (uint32_t)V;
}

// Few positions: each one's rank is counted directly.  A workgroup ranks 64
// positions; its waves share the comparisons.
constexpr int kRankMax = 8192;
constexpr int kRankWaves = 16;
template <typename I>
__global__ __launch_bounds__(64 * kRankWaves) void rank_sort_kernel(const I* __restrict__ tokens, int n, int64_t V,
                                                                     int64_t v_offset, uint32_t* __restrict__ key_out,
                                                                     uint32_t* __restrict__ pos_out) {
  __shared__ uint32_t keys[kRankMax];
  __shared__ int part[kRankWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < n; i += 64 * kRankWaves) keys[i] = token_key(tokens, i, V, v_offset);
  __syncthreads();
  const int t = blockIdx.x * 64 + lane;
  const uint32_t mine = t < n ? keys[t] : 0;
  int less = 0;
  for (int i = wave; i < n; i += kRankWaves) {
    const uint32_t k = keys[i];
    less += (k < mine || (k == mine && i < t)) ? 1 : 0;
  }
  part[wave][lane] = less;
  __syncthreads();
  if (wave == 0 && t < n) {
    int r = 0;
    for (int w = 0; w < kRankWaves; ++w) r += part[w][lane];
    key_out[r] = mine;
    pos_out[r] = (uint32_t)t;
  }
}

// Many positions: a stable radix sort, digits of up to 9 bits, blocks of 4096
// keys.  hist[pass][block][digit] counts the keys of a block: the first pass's
// table from the tokens, each later one while the pass before scatters.
constexpr int kSortKeys = 4096;
constexpr int kSortWaves = 16;
constexpr int kSortBins = 512;

template <typename I>
__global__ __launch_bounds__(64 * kSortWaves) void sort_hist_kernel(const I* __restrict__ tokens, int64_t n, int64_t V,
                                                                     int64_t v_offset, int bins, int passes,
                                                                     uint32_t* __restrict__ key,
                                                                     uint32_t* __restrict__ hist) {
  __shared__ uint32_t h[kSortBins];
  const int64_t row = (int64_t)gridDim.x * kSortBins;
  for (int i = threadIdx.x; i < kSortBins; i += 64 * kSortWaves) h[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < kSortKeys; i += 64 * kSortWaves) {
    const int64_t t = (int64_t)blockIdx.x * kSortKeys + i;
    if (t < n) {
      const uint32_t k = token_key(tokens, t, V, v_offset);
      key[t] = k;
      atomicAdd(&h[k & (bins - 1)], 1u);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kSortBins; i += 64 * kSortWaves) {
    uint32_t* at = hist + (int64_t)blockIdx.x * kSortBins + i;
    at[0] = h[i];
    for (int p = 1; p < passes; ++p) at[p * row] = 0;
  }
}

__global__ __launch_bounds__(64 * kSortWaves) void sort_scatter_kernel(
    const uint32_t* __restrict__ key_in, const uint32_t* __restrict__ pos_in, int64_t n, int pass, int passes,
    int digit_bits, uint32_t* hist, uint32_t* __restrict__ key_out, uint32_t* __restrict__ pos_out) {
  __shared__ uint32_t off[kSortBins];                 // where the block's first key of a digit goes
  __shared__ uint32_t cnt[kSortWaves][kSortBins];     // per wave: keys of a digit, then the wave's next place
  __shared__ uint32_t wtot[8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int bins = 1 << digit_bits, shift = pass * digit_bits;
  const int64_t row = (int64_t)gridDim.x * kSortBins;
  const uint32_t* mine = hist + (int64_t)pass * row;
  const int64_t begin = (int64_t)blockIdx.x * kSortKeys;

  for (int i = tid; i < kSortWaves * kSortBins; i += 64 * kSortWaves) (&cnt[0][0])[i] = 0;
  uint32_t before = 0, total = 0;
  if (tid < kSortBins && tid < bins) {
    for (int64_t b = 0; b < gridDim.x; ++b) {
      const uint32_t c = mine[b * kSortBins + tid];
      total += c;
      before += b < blockIdx.x ? c : 0;
    }
  }
  __syncthreads();
  // exclusive sums of the totals over the digits
  uint32_t inc = total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t v = __shfl_up(inc, o);
    if (lane >= o) inc += v;
  }
  if (wave < 8 && lane == 63) wtot[wave] = inc;
  __syncthreads();
  if (tid < kSortBins) {
    uint32_t o = inc - total + before;
    for (int w = 0; w < wave; ++w) o += wtot[w];
    off[tid] = o;
  }
  // a wave's keys are consecutive, so waves, rounds and lanes are in order
  constexpr int kRounds = kSortKeys / (64 * kSortWaves);
  uint32_t k[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t t = begin + (wave * kRounds + r) * 64 + lane;
    k[r] = t < n ? key_in[t] : 0;
    if (t < n) atomicAdd(&cnt[wave][(k[r] >> shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  if (tid < kSortBins) {
    uint32_t at = off[tid];
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = cnt[w][tid];
      cnt[w][tid] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t t = begin + (wave * kRounds + r) * 64 + lane;
    const bool ok = t < n;
    const uint32_t dgt = (k[r] >> shift) & (bins - 1);
    uint64_t same = __ballot(ok);
    for (int b = 0; b < digit_bits; ++b) {
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
      pos_out[at] = pos_in ? pos_in[t] : (uint32_t)t;
      if (pass + 1 < passes)
        atomicAdd(hist + (int64_t)(pass + 1) * row + (int64_t)(at / kSortKeys) * kSortBins +
                      ((k[r] >> (shift + digit_bits)) & (bins - 1)),
                  1u);
    }
  }
}

template <typename G>
__device__ __forceinline__ void write_grad(G* dst, const float* sum, float scale, int accumulate) {
  float f[8];
  if (accumulate) {
    load8(dst, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += scale * sum[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = scale * sum[i];
  }
  store8(dst, f);
}

// A thread sums eight columns over one chunk of the sorted positions.  Runs of
// one token inside the chunk are final; a run that crosses a border leaves its
// sum in part[chunk][0] (it began before the chunk) or part[chunk][1] (it
// begins here and goes on).
template <typename T, typename G>
__global__ __launch_bounds__(256) void embedding_sum_kernel(const T* __restrict__ dY, const uint32_t* __restrict__ key,
                                                            const uint32_t* __restrict__ pos, int64_t n, int chunk,
                                                            int64_t chunks, Units q, uint32_t V, float scale,
                                                            int accumulate, G* __restrict__ dW,
                                                            float* __restrict__ part) {
  int64_t c;
  uint32_t col;
  unit_at(q, (int64_t)blockIdx.x * 256, threadIdx.x, &c, &col);
  if (c >= chunks) return;
  const int64_t b = c * chunk, e = b + chunk < n ? b + chunk : n;
  int64_t i = b;
  while (i < e) {
    const uint32_t k = key[i];
    if (k >= V) return;
    float sum[8] = {};
    const bool from_before = i == b && b > 0 && key[b - 1] == k;
    for (; i < e && key[i] == k; ++i) {
      float f[8];
      load8(dY + ((int64_t)pos[i] * q.n + col) * 8, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += f[j];
    }
    const bool goes_on = i == e && e < n && key[e] == k;
    if (!from_before && !goes_on)
      write_grad(dW + ((int64_t)k * q.n + col) * 8, sum, scale, accumulate);
    else
      store8(part + ((2 * c + (from_before ? 0 : 1)) * (int64_t)q.n + col) * 8, sum);
  }
}

// The runs that cross borders: the chunk where one begins adds its parts.
template <typename G>
__global__ __launch_bounds__(256) void embedding_join_kernel(const uint32_t* __restrict__ key, int64_t n, int chunk,
                                                             int64_t chunks, Units q, uint32_t V, float scale,
                                                             int accumulate, G* __restrict__ dW,
                                                             const float* __restrict__ part) {
  int64_t c;
  uint32_t col;
  unit_at(q, (int64_t)blockIdx.x * 256, threadIdx.x, &c, &col);
  if (c + 1 >= chunks) return;
  const int64_t b = c * chunk, e = b + chunk;
  const uint32_t k = key[e - 1];
  if (k >= V || key[e] != k) return;                       // no run goes on from here
  if (key[b] == k && b > 0 && key[b - 1] == k) return;     // it began earlier
  float sum[8];
  load8(part + ((2 * c + 1) * (int64_t)q.n + col) * 8, sum);
  for (int64_t j = c + 1; j < chunks && key[j * chunk] == k; ++j) {
    float f[8];
    load8(part + (2 * j * (int64_t)q.n + col) * 8, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += f[i];
  }
  write_grad(dW + ((int64_t)k * q.n + col) * 8, sum, scale, accumulate);
}

__global__ __launch_bounds__(256) void zero_kernel(u32x4* __restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = u32x4{0, 0, 0, 0};
}

// -------------------------------------------------- 8-bit activations, norm --
// Blocks of 32 columns of a row share a power of two 2^(E - 127), the smallest
// that brings the block's largest magnitude below 127.5, kept within 2^-126 and
// 2^121 (127 steps of a larger one are no float); a code is the value divided
// by it, rounded to the nearest whole number, ties to even, at most 127.  Multiplying by powers of two is exact, so a code depends on nothing
// but its block, and a restored value (7 bits and a sign) is exact in bf16.
// E = 255 marks a block that holds an infinity or a NaN: all of it restores to
// NaN.
//
// A thread holds eight columns, four neighbouring lanes a block.
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
    store8(out + at * 8, f);
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
// the backward pass.  A workgroup takes a row at a time; a thread holds NV
// vectors of eight columns (vector v of the row in thread v mod blockDim).
template <typename T, int NV>
__global__ __launch_bounds__(1024) void norm_forward_kernel(const T* __restrict__ x, int64_t rows, int nv,
                                                            const void* __restrict__ weight, int weight_bf16, float eps,
                                                            T* __restrict__ y, int8_t* __restrict__ codes,
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
          *reinterpret_cast<u32x2*>(codes + at * 8) = encode8(f[k], e);
          if ((v & 3) == 0) exps[row * nb + v / 4] = (uint8_t)e;
        }
        float w[8];
        load8_any(weight, weight_bf16, (int64_t)v * 8, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = f[k][i] * r * w[i];
        store8(y + at * 8, w);
      }
    }
  }
}

// With x restored from 8 bits and n = x rstd:
//   dx = rstd (dy w - n mean(dy w n)),   dw = sum over rows of dy n.
// A workgroup walks rows blockIdx, blockIdx + gridDim, ... and keeps its
// columns' share of dw in registers; norm_dweight_kernel adds the workgroups.
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

template <typename T>
__global__ __launch_bounds__(256) void norm_dweight_kernel(const float* __restrict__ part, int groups, int nv,
                                                           T* __restrict__ dweight) {
  const int v = blockIdx.x * 256 + threadIdx.x;
  if (v >= nv) return;
  float sum[8] = {};
  for (int g = 0; g < groups; ++g) {
    float f[8];
    load8(part + ((int64_t)g * nv + v) * 8, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += f[i];
  }
  store8(dweight + (int64_t)v * 8, sum);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// -------------------------------------------------------------- launchers --
void topk_plan(int64_t rows, int64_t V, int64_t K, int* segments, int64_t* seg_cols) {
  const int64_t tiles = cdiv(V + 7, kTopkTile);
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>({cdiv(1024, std::max<int64_t>(rows, 1)), tiles, 64}));
  const int64_t per = cdiv(tiles, want);
  *seg_cols = per * kTopkTile;
  *segments = (int)cdiv(tiles, per);
}

hipError_t launch_teacher_topk(const void* logits, int bf16, int64_t rows, int64_t V, int K, int logprob,
                               const uint8_t* mask, int* idx, float* val, float* lse, uint64_t* cand, float2* state,
                               hipStream_t st) {
  int segments;
  int64_t seg_cols;
  topk_plan(rows, V, K, &segments, &seg_cols);
  const unsigned blocks = (unsigned)(rows * segments);
  auto go = [&](auto* p, auto cap) {
    using E = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    constexpr int CAP = decltype(cap)::value;
    topk_rows_kernel<E, CAP><<<blocks, kTopkThreads, 0, st>>>(p, V, K, segments, seg_cols, logprob, mask, idx, val, lse,
                                                             cand, state);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || segments == 1) return e;
    topk_merge_kernel<CAP><<<(unsigned)rows, kTopkThreads, 0, st>>>(cand, state, K, segments, logprob, mask, idx, val,
                                                                   lse);
    return hipGetLastError();
  };
  // the buffer holds K words and a tile, and a power of two for the sort
  using Small = std::integral_constant<int, 4096>;
  using Large = std::integral_constant<int, 8192>;
  if (bf16) return K <= 1024 ? go((const bf16_t*)logits, Small{}) : go((const bf16_t*)logits, Large{});
  return K <= 1024 ? go((const float*)logits, Small{}) : go((const float*)logits, Large{});
}

hipError_t launch_embedding_forward(const void* W, int bf16, int64_t V, int d, int64_t v_offset, const void* tokens,
                                    int tokens64, int64_t T, float scale, void* out, hipStream_t st) {
  const Units q = units(d / 8);
  const unsigned blocks = (unsigned)cdiv(T * q.n, 1024);
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
  size_t o = 0;
  auto take = [&](size_t bytes) {
    size_t at = o;
    o += (bytes + 255) & ~(size_t)255;
    return at;
  };
  w.chunk = T <= 4096 ? 8 : 32;
  w.chunks = cdiv(T, w.chunk);
  if (T > kRankMax) {
    int bits = 1;
    while (((int64_t)1 << bits) <= V) ++bits;  // keys 0 .. V
    w.passes = (int)cdiv(bits, 9);
    w.digit_bits = (int)cdiv(bits, w.passes);
    w.sort_blocks = cdiv(T, kSortKeys);
  }
  w.key0 = take(T * 4);
  w.pos0 = take(T * 4);
  if (w.passes) {
    w.key1 = take(T * 4);
    w.pos1 = take(T * 4);
    w.hist = take((size_t)w.passes * w.sort_blocks * kSortBins * 4);
  }
  w.part = take((size_t)2 * w.chunks * d * 4);
  w.total = o;
  return w;
}

template <typename T, typename G>
static hipError_t embedding_reduce(const T* dY, int64_t n, int d, int64_t V, float scale, G* dW, int accumulate,
                                   const EmbedWs& w, const uint32_t* key, const uint32_t* pos, float* part,
                                   hipStream_t st) {
  const Units q = units(d / 8);
  const unsigned blocks = (unsigned)cdiv(w.chunks * q.n, 256);
  embedding_sum_kernel<<<blocks, 256, 0, st>>>(dY, key, pos, n, (int)w.chunk, w.chunks, q, (uint32_t)V, scale,
                                               accumulate, dW, part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || w.chunks < 2) return e;
  embedding_join_kernel<<<blocks, 256, 0, st>>>(key, n, (int)w.chunk, w.chunks, q, (uint32_t)V, scale, accumulate, dW,
                                                (const float*)part);
  return hipGetLastError();
}

template <typename I>
static hipError_t embedding_sort(const I* tokens, int64_t T, int64_t V, int64_t v_offset, const EmbedWs& w, char* ws,
                                 const uint32_t** key, const uint32_t** pos, hipStream_t st) {
  uint32_t* k[2] = {(uint32_t*)(ws + w.key0), (uint32_t*)(ws + w.key1)};
  uint32_t* p[2] = {(uint32_t*)(ws + w.pos0), (uint32_t*)(ws + w.pos1)};
  hipError_t e;
  if (!w.passes) {
    rank_sort_kernel<<<(unsigned)cdiv(T, 64), 64 * kRankWaves, 0, st>>>(tokens, (int)T, V, v_offset, k[0], p[0]);
    *key = k[0];
    *pos = p[0];
    return hipGetLastError();
  }
  uint32_t* hist = (uint32_t*)(ws + w.hist);
  const unsigned blocks = (unsigned)w.sort_blocks;
  sort_hist_kernel<<<blocks, 64 * kSortWaves, 0, st>>>(tokens, T, V, v_offset, 1 << w.digit_bits, w.passes, k[0], hist);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  for (int i = 0; i < w.passes; ++i) {
    sort_scatter_kernel<<<blocks, 64 * kSortWaves, 0, st>>>(k[i & 1], i ? p[i & 1] : nullptr, T, i, w.passes,
                                                            w.digit_bits, hist, k[~i & 1], p[~i & 1]);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  *key = k[w.passes & 1];
  *pos = p[w.passes & 1];
  return hipSuccess;
}

hipError_t launch_embedding_backward(const void* dY, int bf16, int64_t T, int d, const void* tokens, int tokens64,
                                     int64_t V, int64_t v_offset, float scale, void* dW, int dw_bf16, int accumulate,
                                     char* ws, hipStream_t st) {
  hipError_t e;
  if (!accumulate) {
    const int64_t n = V * d * (dw_bf16 ? 2 : 4) / 16;
    zero_kernel<<<(unsigned)std::min<int64_t>(cdiv(n, 256), 8192), 256, 0, st>>>((u32x4*)dW, n);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (T == 0) return hipSuccess;
  const EmbedWs w = embed_ws(T, V, d);
  const uint32_t *key, *pos;
  if (tokens64)
    e = embedding_sort((const int64_t*)tokens, T, V, v_offset, w, ws, &key, &pos, st);
  else
    e = embedding_sort((const int32_t*)tokens, T, V, v_offset, w, ws, &key, &pos, st);
  if (e != hipSuccess) return e;
  float* part = (float*)(ws + w.part);
  if (bf16 && dw_bf16) return embedding_reduce((const bf16_t*)dY, T, d, V, scale, (bf16_t*)dW, accumulate, w, key, pos, part, st);
  if (bf16) return embedding_reduce((const bf16_t*)dY, T, d, V, scale, (float*)dW, accumulate, w, key, pos, part, st);
  if (dw_bf16) return embedding_reduce((const float*)dY, T, d, V, scale, (bf16_t*)dW, accumulate, w, key, pos, part, st);
  return embedding_reduce((const float*)dY, T, d, V, scale, (float*)dW, accumulate, w, key, pos, part, st);
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

// Threads and vectors per thread for rows of nv vectors.
static void norm_shape(int nv, int* threads, int* per) {
  *threads = (int)std::min<int64_t>(1024, cdiv(nv, 64) * 64);
  const int64_t k = cdiv(nv, *threads);
  *per = k <= 1 ? 1 : k <= 2 ? 2 : k <= 4 ? 4 : 8;
}

hipError_t launch_norm_forward(const void* x, int bf16, int64_t T, int d, const void* weight, int weight_bf16,
                               float eps, void* y, int8_t* codes, uint8_t* exps, float* rstd, hipStream_t st) {
  const int nv = d / 8;
  int threads, per;
  norm_shape(nv, &threads, &per);
  const unsigned blocks = (unsigned)T;
  auto go = [&](auto* p) {
    using E = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    switch (per) {
      case 1: norm_forward_kernel<E, 1><<<blocks, threads, 0, st>>>(p, T, nv, weight, weight_bf16, eps, (E*)y, codes, exps, rstd); break;
      case 2: norm_forward_kernel<E, 2><<<blocks, threads, 0, st>>>(p, T, nv, weight, weight_bf16, eps, (E*)y, codes, exps, rstd); break;
      case 4: norm_forward_kernel<E, 4><<<blocks, threads, 0, st>>>(p, T, nv, weight, weight_bf16, eps, (E*)y, codes, exps, rstd); break;
      default: norm_forward_kernel<E, 8><<<blocks, threads, 0, st>>>(p, T, nv, weight, weight_bf16, eps, (E*)y, codes, exps, rstd);
    }
  };
  if (bf16)
    go((const bf16_t*)x);
  else
    go((const float*)x);
  return hipGetLastError();
}

int64_t norm_backward_groups(int64_t T, int64_t) { return std::min<int64_t>(T, 1024); }

hipError_t launch_norm_backward(const void* dy, int bf16, int64_t T, int d, const int8_t* codes, const uint8_t* exps,
                                const float* rstd, const void* weight, int weight_bf16, void* dx, void* dweight,
                                float* part, hipStream_t st) {
  const int nv = d / 8;
  int threads, per;
  norm_shape(nv, &threads, &per);
  const unsigned groups = (unsigned)norm_backward_groups(T, d);
  auto go = [&](auto* p) {
    using E = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    switch (per) {
      case 1: norm_backward_kernel<E, 1><<<groups, threads, 0, st>>>(p, T, nv, codes, exps, rstd, weight, weight_bf16, (E*)dx, part); break;
      case 2: norm_backward_kernel<E, 2><<<groups, threads, 0, st>>>(p, T, nv, codes, exps, rstd, weight, weight_bf16, (E*)dx, part); break;
      case 4: norm_backward_kernel<E, 4><<<groups, threads, 0, st>>>(p, T, nv, codes, exps, rstd, weight, weight_bf16, (E*)dx, part); break;
      default: norm_backward_kernel<E, 8><<<groups, threads, 0, st>>>(p, T, nv, codes, exps, rstd, weight, weight_bf16, (E*)dx, part);
    }
  };
  if (groups > 0) {
    if (bf16)
      go((const bf16_t*)dy);
    else
      go((const float*)dy);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const unsigned blocks = (unsigned)cdiv(nv, 256);
  if (weight_bf16)
    norm_dweight_kernel<<<blocks, 256, 0, st>>>(part, (int)groups, nv, (bf16_t*)dweight);
  else
    norm_dweight_kernel<<<blocks, 256, 0, st>>>(part, (int)groups, nv, (float*)dweight);
  return hipGetLastError();
}

}  // namespace ckl
