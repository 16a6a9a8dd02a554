// gfx950 kernels of the operators around the distillation loss: the top-K
// teacher cache made from logits, the embedding table tied to the output head
// with its gradient, and activations held in 8 bits with the RMS norm whose
// backward pass reads them.
#include "ckl_ops.hpp"

#include <algorithm>
#include <type_traits>

#include "ckl_topk.hpp"
#include "ckl_vec.hpp"

namespace ckl {

namespace {

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
// A thread holds eight columns, four neighbouring lanes a block of 32.  Encoding and
// decoding are bound by memory: 131072 x 2880 bf16 192 and 208 us, 6.0 and 5.5 TB/s.
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
                                                              mask, idx, val, lse, cand, state, RowOut{});
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || segments == 1) return e;
    topk_merge_kernel<E, CAP><<<(unsigned)rows, kTopkThreads, 0, st>>>(cand, state, K, segments, logprob, mask, idx,
                                                                      val, lse, p, (int)V, RowOut{});
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

hipError_t launch_norm_dweight(const float* part, int groups, int d, int weight_bf16, void* dweight, hipStream_t st) {
  const unsigned blocks = (unsigned)cdiv(d, 64);
  if (weight_bf16)
    norm_dweight_kernel<<<blocks, 1024, 0, st>>>(part, groups, d, (bf16_t*)dweight);
  else
    norm_dweight_kernel<<<blocks, 1024, 0, st>>>(part, groups, d, (float*)dweight);
  return hipGetLastError();
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
  return launch_norm_dweight(part, (int)groups, d, weight_bf16, dweight, st);
}

}  // namespace ckl
