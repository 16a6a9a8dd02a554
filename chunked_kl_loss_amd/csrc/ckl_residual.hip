// gfx950 kernels between a branch's output and the next product: dropout from a
// counter-based generator, and the RMS norm with the residual's addition (and
// that dropout), its output in 16 or 32 bits or in 8 with scales, and its
// backward pass.
#include <algorithm>
#include <type_traits>

#include "ckl_ops.hpp"
#include "ckl_vec.hpp"

namespace ckl {

namespace {

// ---------------------------------------------------------------- dropout --
// An element is kept where its sixteen random bits reach the threshold, and then
// multiplied by 1 / (share kept).  The bits are those of Philox4x32 with ten
// rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1,
// 2, 3", SC 2011): the key is the seed, the counter is (index of the vector of
// eight elements, offset), and its 128 bits are the vector's, element 2 i + h in
// half h of word i.  So a mask is a function of (seed, offset, element) and is
// formed again where it is needed.  Sixteen bits an element, not 32: the share
// dropped is a multiple of 2^-16 (the scale is that share's own, so the mean is
// kept), and the ten rounds, whose 20 products of 32 x 32 bits take a quarter of
// the rate of additions, are paid once for eight elements.
struct Philox {
  uint32_t k0, k1, o0, o1;
};
// The seed and offset of a call: its own, or those in device memory with its
// offset added (a captured call then draws anew when the memory changes).
__device__ __forceinline__ Philox philox_key(uint64_t seed, uint64_t offset, const int64_t* state) {
  if (state != nullptr) {
    seed = (uint64_t)state[0];
    offset += (uint64_t)state[1];
  }
  return Philox{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
}
__device__ __forceinline__ u32x4 philox(const Philox& p, uint64_t vec) {
  uint32_t c0 = (uint32_t)vec, c1 = (uint32_t)(vec >> 32), c2 = p.o0, c3 = p.o1, k0 = p.k0, k1 = p.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}
// f scaled where kept, zero elsewhere (whatever f is there).
__device__ __forceinline__ void drop8(const Philox& p, uint64_t vec, uint32_t threshold, float scale, float* f) {
  const u32x4 r = philox(p, vec);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = (r[i] & 0xffffu) >= threshold ? f[2 * i] * scale : 0.f;
    f[2 * i + 1] = (r[i] >> 16) >= threshold ? f[2 * i + 1] * scale : 0.f;
  }
}

// Four vectors a thread, loaded before the first is looked at.  Bound by memory: 32768 x
// 2880 bf16 66 us, 5.7 TB/s (a copy 5.2).
constexpr int kDropVecs = 4;
template <typename T>
__global__ __launch_bounds__(256) void dropout_kernel(const T* __restrict__ x, int64_t n, uint32_t threshold,
                                                      float scale, uint64_t seed, uint64_t offset,
                                                      const int64_t* __restrict__ state, T* __restrict__ out) {
  const Philox p = philox_key(seed, offset, state);
  const int64_t whole = n / 8;
  const int64_t v0 = (int64_t)blockIdx.x * (256 * kDropVecs) + threadIdx.x;
  float f[kDropVecs][8];
#pragma unroll
  for (int k = 0; k < kDropVecs; ++k)
    if (v0 + k * 256 < whole) load8(x + (v0 + k * 256) * 8, f[k]);
#pragma unroll
  for (int k = 0; k < kDropVecs; ++k) {
    const int64_t v = v0 + k * 256;
    if (v < whole) {
      drop8(p, (uint64_t)v, threshold, scale, f[k]);
      stream8(out + v * 8, f[k]);
    } else if (v == whole && n % 8 != 0) {  // the last, short vector
      const int m = (int)(n % 8);
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = i < m ? (float)x[v * 8 + i] : 0.f;
      drop8(p, (uint64_t)v, threshold, scale, t);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < m) out[v * 8 + i] = (T)t[i];
    }
  }
}

// ------------------------------------------------- RMS norm behind a branch --
// h = residual + dropout(x), rounded to the residual's type; y = h r weight with
// r = 1 / sqrt(mean h^2 + eps) of the rounded h, which is what the backward pass
// and the next layer read.  A row's sum of squares is held in fp32.
//
// Threads of a row: rows of up to 512 columns take 8, 16, 32 or 64 lanes of a
// wave (several rows to a workgroup), wider ones a workgroup of whole waves.
// (WAVE: the first kind.)  A row is held in registers between the sum of squares and
// the output, so everything is read once.  Bound by memory: 32768 x 2880 bf16 125 us, 6.0
// TB/s; 262144 x 64 6.3, 65536 x 520 5.9, 32768 x 2048 7.0, 8192 x 8192 7.0, 2048 x 65536
// 5.3.  The output in 8 bits: 65536 x 2880 as int8 222 to 240 us, 5.5 to 5.9
// TB/s, as e4m3 221, 6.0.
struct RowShape {
  int threads, per;  // threads a row takes, vectors of eight a thread
};
RowShape row_shape(int nv) {
  RowShape s;
  if (nv <= 64) {
    s.per = 1;
    for (s.threads = 8; s.threads < nv; s.threads *= 2) {}
    return s;
  }
  s.per = nv <= 2048 ? 2 : nv <= 4096 ? 4 : 8;
  s.threads = (int)cdiv(cdiv(nv, s.per), 64) * 64;
  return s;
}

// The sum over a row's threads, in each of them.
template <bool WAVE>
__device__ __forceinline__ float row_sum(float x, int threads, float* slots) {
  if constexpr (WAVE) {
    for (int o = threads >> 1; o > 0; o >>= 1) x += __shfl_xor(x, o);
    return x;
  }
  return group_sum(x, slots);
}
// The same in 64 bits.
template <bool WAVE>
__device__ __forceinline__ double row_sum64(double x, int threads, double* slots) {
  const int lanes = WAVE ? threads : 64;
  for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor(x, o);
  if constexpr (!WAVE) {
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = x;
    __syncthreads();
    x = slots[0];
    for (int w = 1; w < (int)(blockDim.x >> 6); ++w) x += slots[w];
    __syncthreads();
  }
  return x;
}
// The largest of a row's threads, as unsigned integers.
template <bool WAVE>
__device__ __forceinline__ uint32_t row_top(uint32_t x, int threads, float* slots) {
  const int lanes = WAVE ? threads : 64;
  for (int o = lanes >> 1; o > 0; o >>= 1) {
    const uint32_t y = __shfl_xor(x, o);
    x = y > x ? y : x;
  }
  if constexpr (!WAVE) {
    uint32_t* s = reinterpret_cast<uint32_t*>(slots);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
    __syncthreads();
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) x = s[w] > x ? s[w] : x;
    __syncthreads();
  }
  return x;
}

struct Drop {
  uint32_t threshold;  // 0: no dropout
  float scale;
  uint64_t seed, offset;
  const int64_t* state;
};

__device__ __forceinline__ float round_to(float x, const bf16_t*) { return (float)(bf16_t)x; }
__device__ __forceinline__ float round_to(float x, const float*) { return x; }

// Eight values as e4m3 (four bits of exponent, three behind the first; RNE).
__device__ __forceinline__ u32x2 pack_e4m3(const float* f) {
  u32x2 c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], w, true);
    c[i] = (uint32_t)w;
  }
  return c;
}

enum { kOutRows = 0, kOutInt8 = 1, kOutE4M3 = 2 };
struct NormOut {
  void* y;        // rows of x's type, or codes
  void* scales;   // int8: exponents [T][ceil(d / 32)]; e4m3: float [T]
  float* rstd;    // may be NULL
};

template <typename TX, typename TR, int NV, bool WAVE, bool DROP, int OUT>
__global__ __launch_bounds__(1024) void add_norm_kernel(const TX* __restrict__ x, const TR* __restrict__ residual,
                                                        int64_t rows, int nv, int row_threads,
                                                        const void* __restrict__ weight, int weight_bf16, float eps,
                                                        Drop drop, TR* __restrict__ h, NormOut out) {
  constexpr bool CODES = OUT != kOutRows;
  __shared__ float slots[16];
  __shared__ double slots64[CODES ? 16 : 1];
  const int tid = WAVE ? (int)threadIdx.x & (row_threads - 1) : (int)threadIdx.x;
  const int64_t row = WAVE ? (int64_t)blockIdx.x * (blockDim.x / row_threads) + threadIdx.x / row_threads
                           : (int64_t)blockIdx.x;
  const bool live = row < rows;  // (WAVE: the last workgroup's rows; its lanes stay for the shuffles)
  Philox p{};
  if constexpr (DROP) p = philox_key(drop.seed, drop.offset, drop.state);
  float f[NV][8];
  // (8 bits: what y's own roundings move across the border of two codes is a whole step there, so there the sum is held
  // in 64 bits, r and its product with h in two floats, and y is rounded once; the bytes hide it)
  std::conditional_t<CODES, double, float> ss = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = k * row_threads + tid;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[k][i] = 0.f;
    if (live && v < nv) {
      const int64_t at = row * nv + v;
      float r[8];
      load8(x + at * 8, f[k]);
      load8(residual + at * 8, r);
      if constexpr (DROP) drop8(p, (uint64_t)at, drop.threshold, drop.scale, f[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[k][i] = round_to(f[k][i] + r[i], (const TR*)nullptr);
      stream8(h + at * 8, f[k]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += (decltype(ss))f[k][i] * f[k][i];
  }
  float r, r_low = 0.f;
  if constexpr (CODES) {
    const double r64 = 1.0 / sqrt(row_sum64<WAVE>(ss, row_threads, slots64) / (nv * 8) + (double)eps);
    r = (float)r64;
    r_low = (float)(r64 - (double)r);
  } else {
    ss = row_sum<WAVE>(ss, row_threads, slots);
    r = 1.f / sqrtf(ss / (float)(nv * 8) + eps);
    if (ss == INFINITY) {
      // the squares' sum is past fp32 (values near 1e19 and more), or the row holds an infinity: once more with h
      // 2^-96, beside which eps is nothing
      float s2 = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s2 += (f[k][i] * 0x1p-96f) * (f[k][i] * 0x1p-96f);
      r = 0x1p-96f / sqrtf(row_sum<WAVE>(s2, row_threads, slots) / (float)(nv * 8));
    }
  }
  if (out.rstd != nullptr && live && tid == 0) out.rstd[row] = r;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = k * row_threads + tid;
    if (live && v < nv) {
      float w[8];
      load8_any(weight, weight_bf16, (int64_t)v * 8, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = f[k][i] * r;
        if constexpr (CODES) {
          const float n_low = fmaf(f[k][i], r_low, fmaf(f[k][i], r, -n));
          f[k][i] = fmaf(n, w[i], n_low * w[i]);
        } else {
          f[k][i] = n * w[i];
        }
      }
      if constexpr (OUT == kOutRows) stream8((TX*)out.y + (row * nv + v) * 8, f[k]);
    }
  }
  if constexpr (OUT == kOutInt8) {
    const int nb = (nv + 3) / 4;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * row_threads + tid;
      const uint32_t e = block_exponent(top_bits(f[k]));  // (lanes past the row hold zeros)
      if (live && v < nv) {
        // a value that its rounding to fp32, at most 2^-18 steps, may have taken past the middle of two codes is formed
        // again in 64 bits (one vector in four thousand)
        const float inv = e == 255 ? 0.f : __uint_as_float((254u - e) << 23);
        bool close = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t = f[k][i] * inv;
          close |= fabsf(t - rintf(t)) > 0.5f - 0x1p-16f;
        }
        if (close) {
          float n[8], w[8];
          load8(h + (row * nv + v) * 8, n);
          load8_any(weight, weight_bf16, (int64_t)v * 8, w);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            f[k][i] = (float)rint((double)n[i] * ((double)r + r_low) * w[i] * inv) * block_step(e);
        }
        __builtin_nontemporal_store(encode8(f[k], e), reinterpret_cast<u32x2*>((int8_t*)out.y + (row * nv + v) * 8));
        if ((v & 3) == 0) ((uint8_t*)out.scales)[row * nb + v / 4] = (uint8_t)e;
      }
    }
  }
  if constexpr (OUT == kOutE4M3) {
    // the row's largest magnitude becomes 448, e4m3's largest; a row that holds an
    // infinity or a NaN gets a NaN for its scale and codes of zero
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const uint32_t t = top_bits(f[k]);
      top = t > top ? t : top;
    }
    top = row_top<WAVE>(top, row_threads, slots);
    const bool bad = top >= 0x7f800000u;
    const float scale = bad ? __uint_as_float(0x7fc00000u) : fmaxf(__uint_as_float(top) / 448.f, 0x1p-126f);
    const float inv = 1.f / scale;
    if (live && tid == 0) ((float*)out.scales)[row] = scale;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * row_threads + tid;
      if (live && v < nv) {
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          q[i] = f[k][i] * inv;
          q[i] = fmaf(fmaf(-q[i], scale, f[k][i]), inv, q[i]);  // the quotient, rounded once
          q[i] = bad ? 0.f : fminf(fmaxf(q[i], -448.f), 448.f);
        }
        __builtin_nontemporal_store(pack_e4m3(q), reinterpret_cast<u32x2*>((uint8_t*)out.y + (row * nv + v) * 8));
      }
    }
  }
}

// With n = h r, g = dy weight:  dres = dh + r (g - n mean(g n)),  dx = dropout of
// dres,  dw = sum over rows of dy n.  A workgroup walks its rows and keeps its
// columns' share of dw in registers; norm_dweight adds the workgroups.  Rows of
// more than two vectors a thread are read a second time (from the caches) instead
// of being held.  Bound by memory: 32768 x 2880 bf16 with dh 174 us, 5.4 TB/s; 262144 x
// 64 4.4, 65536 x 520 3.9, 8192 x 8192 5.1, 2048 x 65536 3.2 (read again past the L2; past
// 32768 columns the eight vectors of dw leave 48 to 57 registers spilled).
template <typename TX, typename TR, int NV, bool WAVE, bool DROP>
__global__ __launch_bounds__(1024) void add_norm_backward_kernel(
    const TX* __restrict__ dy, const TR* __restrict__ dh, const TR* __restrict__ h, const float* __restrict__ rstd,
    int64_t rows, int nv, int row_threads, const void* __restrict__ weight, int weight_bf16, Drop drop,
    TX* __restrict__ dx, TR* __restrict__ dres, float* __restrict__ part) {
  constexpr bool HOLD = NV <= 2;
  constexpr int H = HOLD ? NV : 1;
  __shared__ float slots[16];
  __shared__ __attribute__((aligned(16))) float sums[WAVE ? 256 * 8 : 8];
  const int tid = WAVE ? (int)threadIdx.x & (row_threads - 1) : (int)threadIdx.x;
  const int row_slots = WAVE ? (int)blockDim.x / row_threads : 1, slot = WAVE ? (int)threadIdx.x / row_threads : 0;
  Philox p{};
  if constexpr (DROP) p = philox_key(drop.seed, drop.offset, drop.state);
  float dw[NV][8] = {};
  // (rows past the end are walked too, so that a wave's lanes stay together)
  for (int64_t row0 = (int64_t)blockIdx.x * row_slots; row0 < rows; row0 += (int64_t)gridDim.x * row_slots) {
    const int64_t row = row0 + slot;
    const bool live = row < rows;
    const float r = live ? rstd[row] : 0.f;
    float n[H][8], g[H][8], a[H][8];
    float c = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * row_threads + tid, kh = HOLD ? k : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) n[kh][i] = g[kh][i] = a[kh][i] = 0.f;
      if (live && v < nv) {
        const int64_t at = row * nv + v;
        load8(h + at * 8, n[kh]);
        load8(dy + at * 8, g[kh]);
        if (HOLD && dh != nullptr) load8(dh + at * 8, a[kh]);
        float w[8];
        load8_any(weight, weight_bf16, (int64_t)v * 8, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          n[kh][i] *= r;
          dw[k][i] += g[kh][i] * n[kh][i];
          g[kh][i] *= w[i];
          c += g[kh][i] * n[kh][i];
        }
      }
    }
    c = row_sum<WAVE>(c, row_threads, slots) / (float)(nv * 8);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * row_threads + tid, kh = HOLD ? k : 0;
      if (live && v < nv) {
        const int64_t at = row * nv + v;
        if constexpr (!HOLD) {
          load8(h + at * 8, n[0]);
          load8(dy + at * 8, g[0]);
          float w[8];
          load8_any(weight, weight_bf16, (int64_t)v * 8, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            a[0][i] = 0.f;
            n[0][i] *= r;
            g[0][i] *= w[i];
          }
          if (dh != nullptr) load8(dh + at * 8, a[0]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) g[kh][i] = a[kh][i] + r * (g[kh][i] - n[kh][i] * c);
        stream8(dres + at * 8, g[kh]);
        if (dx != nullptr) {
          if constexpr (DROP) drop8(p, (uint64_t)at, drop.threshold, drop.scale, g[kh]);
          stream8(dx + at * 8, g[kh]);
        }
      }
    }
  }
  if constexpr (WAVE) {
    // the workgroup's rows' shares, added in their order
    float* mine = sums + threadIdx.x * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) mine[i] = dw[0][i];
    __syncthreads();
    if (slot == 0 && tid < nv) {
      for (int s = 1; s < row_slots; ++s) {
        const float* o = sums + (s * row_threads + tid) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[0][i] += o[i];
      }
      store8(part + ((int64_t)blockIdx.x * nv + tid) * 8, dw[0]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * row_threads + tid;
      if (v < nv) store8(part + ((int64_t)blockIdx.x * nv + v) * 8, dw[k]);
    }
  }
}

template <int N>
using Count = std::integral_constant<int, N>;
template <bool B>
using Flag = std::integral_constant<bool, B>;

Drop device_drop(const DropArgs& a) { return Drop{a.threshold, a.scale, a.seed, a.offset, a.state}; }

// f(x's type, residual's type) as null pointers, for (fp32, fp32), (bf16, bf16)
// and (bf16, fp32).
template <typename F>
void by_types(int x_bf16, int r_bf16, F&& f) {
  if (!x_bf16)
    f((float*)nullptr, (float*)nullptr);
  else if (r_bf16)
    f((bf16_t*)nullptr, (bf16_t*)nullptr);
  else
    f((bf16_t*)nullptr, (float*)nullptr);
}
// f(vectors a thread, whether rows share waves).
template <typename F>
void by_shape(const RowShape& s, int nv, F&& f) {
  if (nv <= 64)
    f(Count<1>{}, Flag<true>{});
  else if (s.per == 2)
    f(Count<2>{}, Flag<false>{});
  else if (s.per == 4)
    f(Count<4>{}, Flag<false>{});
  else
    f(Count<8>{}, Flag<false>{});
}

}  // namespace

// -------------------------------------------------------------- launchers --
hipError_t launch_dropout(const void* x, int bf16, int64_t n, const DropArgs& a, void* out, hipStream_t st) {
  const unsigned blocks = (unsigned)cdiv(cdiv(n, 8), 256 * kDropVecs);
  if (bf16)
    dropout_kernel<<<blocks, 256, 0, st>>>((const bf16_t*)x, n, a.threshold, a.scale, a.seed, a.offset, a.state,
                                           (bf16_t*)out);
  else
    dropout_kernel<<<blocks, 256, 0, st>>>((const float*)x, n, a.threshold, a.scale, a.seed, a.offset, a.state,
                                           (float*)out);
  return hipGetLastError();
}

hipError_t launch_add_norm(const void* x, int x_bf16, const void* residual, int r_bf16, int64_t T, int d,
                           const void* weight, int weight_bf16, float eps, const DropArgs& a, void* h, int form,
                           void* y, void* scales, float* rstd, hipStream_t st) {
  const int nv = d / 8;
  const RowShape s = row_shape(nv);
  const bool wave = nv <= 64;
  const int threads = wave ? 256 : s.threads;
  const unsigned blocks = (unsigned)(wave ? cdiv(T, 256 / s.threads) : T);
  const NormOut out{y, scales, rstd};
  by_types(x_bf16, r_bf16, [&](auto* px, auto* pr) {
    using TX = std::remove_pointer_t<decltype(px)>;
    using TR = std::remove_pointer_t<decltype(pr)>;
    by_shape(s, nv, [&](auto per, auto wv) {
      constexpr int NV = decltype(per)::value;
      constexpr bool WAVE = decltype(wv)::value;
      auto go = [&](auto drop, auto kind) {
        add_norm_kernel<TX, TR, NV, WAVE, decltype(drop)::value, decltype(kind)::value><<<blocks, threads, 0, st>>>(
            (const TX*)x, (const TR*)residual, T, nv, s.threads, weight, weight_bf16, eps, device_drop(a), (TR*)h,
            out);
      };
      if (form == kOutInt8)
        go(Flag<false>{}, Count<kOutInt8>{});
      else if (form == kOutE4M3)
        go(Flag<false>{}, Count<kOutE4M3>{});
      else if (a.threshold)
        go(Flag<true>{}, Count<kOutRows>{});
      else
        go(Flag<false>{}, Count<kOutRows>{});
    });
  });
  return hipGetLastError();
}

int64_t add_norm_backward_groups(int64_t T, int64_t d) {
  const int nv = (int)(d / 8);
  const RowShape s = row_shape(nv);
  if (nv <= 64) return std::min<int64_t>(cdiv(T, 256 / s.threads), 1024);
  return std::min<int64_t>(T, 256 * std::max(1, 1024 / s.threads));
}

hipError_t launch_add_norm_backward(const void* dy, int x_bf16, const void* dh, int r_bf16, int64_t T, int d,
                                    const void* h, const float* rstd, const void* weight, int weight_bf16,
                                    const DropArgs& a, void* dx, void* dres, void* dweight, float* part,
                                    hipStream_t st) {
  const int nv = d / 8;
  const RowShape s = row_shape(nv);
  const int threads = nv <= 64 ? 256 : s.threads;
  const int64_t groups = add_norm_backward_groups(T, d);
  if (groups > 0) {
    by_types(x_bf16, r_bf16, [&](auto* px, auto* pr) {
      using TX = std::remove_pointer_t<decltype(px)>;
      using TR = std::remove_pointer_t<decltype(pr)>;
      by_shape(s, nv, [&](auto per, auto wv) {
        constexpr int NV = decltype(per)::value;
        constexpr bool WAVE = decltype(wv)::value;
        auto go = [&](auto drop) {
          add_norm_backward_kernel<TX, TR, NV, WAVE, decltype(drop)::value><<<(unsigned)groups, threads, 0, st>>>(
              (const TX*)dy, (const TR*)dh, (const TR*)h, rstd, T, nv, s.threads, weight, weight_bf16, device_drop(a),
              (TX*)dx, (TR*)dres, part);
        };
        a.threshold ? go(Flag<true>{}) : go(Flag<false>{});
      });
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return launch_norm_dweight(part, (int)groups, d, weight_bf16, dweight, st);
}

}  // namespace ckl
