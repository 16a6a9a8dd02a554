// gfx950 kernels of the log probabilities of given tokens, and of the rows'
// entropies, straight from hidden states and the output head: the logits never
// leave the MFMA accumulators.
//   head_rows     z^T = W H^T by tiles; a row's log sum exp and sum of p log p
//                 behind a running maximum, the token's logit where it falls
//   head_finish   splits merged; log probability, entropy, log sum exp
// Backward (the logits are multiplied again, G = dloss / dz by blocks):
//   head_consts   what a row's gradient needs
//   head_grad     G = 1[v = token] a - q (a + b (log q + entropy))
// and the contractions dH = G W, dW = G^T H of the distillation loss.
#include "ckl_head.hpp"

#include <type_traits>

#include "ckl_tile.hpp"
#include "ckl_vec.hpp"

namespace ckl {

namespace {

// Tiles (vocabulary x token rows, and a wave's share of them).  Few rows: W is read
// once whatever the tile, and a narrow one leaves room for two workgroups or more on
// a compute unit, whose loads hide one another's latency.  (2880 x 201088 bf16, us,
// 256 x 32 / 128 x 32 / 64 x 32 for 8 rows: 199 / 243 / 209; 256 x 64 / 128 x 64 for 64:
// 210 / 271; 128 x 128 / 256 x 128 / 256 x 256 for 128: 263 / 279 / 295; 256 x 256 / 256 x
// 128 for 129: 300 / 395.  What a copy moves takes 221.)
using CfgWide = Dma64Cfg<256, 256, 128, 64>;
using CfgMiddle = Dma64Cfg<128, 128, 64, 32>;
using CfgNarrow = Dma64Cfg<256, 64, 64, 32>;
using CfgSlim = Dma64Cfg<256, 32, 64, 32>;
using CfgF32 = TileCfg<float, 128, 128, 64, 64>;
using CfgF32Small = TileCfg<float, 64, 64, 32, 32>;
using CfgF32Slim = TileCfg<float, 128, 32, 32, 32>;

constexpr float kExpZero = -1e4f;  // 2^x is zero from here on, and its product with x too

// A shift of (m, s, e) and its sum with another, in base 2: s = sum of 2^(x - m),
// e = sum of (x - m) 2^(x - m).
__device__ __forceinline__ void ent2_merge(float& m, float& s, float& e, float m2, float s2, float e2) {
  const float mn = fmaxf(m, m2);
  const float d1 = m == mn ? 0.f : fmaxf(m - mn, kExpZero), d2 = m2 == mn ? 0.f : fmaxf(m2 - mn, kExpZero);
  const float f1 = fast_exp2(d1), f2 = fast_exp2(d2);
  e = f1 * (e + d1 * s) + f2 * (e2 + d2 * s2);
  s = f1 * s + f2 * s2;
  m = mn;
}

// The column of packed row i's token, -1 where it is none.
__device__ __forceinline__ int token_column(const HeadRows& r, int i, int V) {
  const int t = r.perm != nullptr ? r.perm[i] : i;
  const int64_t v = r.tokens64 ? reinterpret_cast<const int64_t*>(r.tokens)[t]
                               : (int64_t)reinterpret_cast<const int32_t*>(r.tokens)[t];
  return v >= 0 && v < V ? (int)v : -1;
}

// ---------------------------------------------------------------- forward --
// A workgroup takes a block of BN rows and a run of vocabulary tiles, and walks
// the tiles with the rows' running (m, s, e).  With two column blocks a wave, lane
// group g owns block g's state; with one, both groups hold it.  Bound by the
// matrix units where there are many rows: beside the logits' product an element
// costs one exponential and three more operations (2048 x 2880 by 201088 words bf16
// 1.86 ms, 1.27 PFLOP/s; the logits by the library's product 1.76, without a
// softmax), and by W's bytes where there are few (8 rows 194 us, 6.0 TB/s).
constexpr int kGroupRows = 8;  // row blocks that walk the vocabulary together (they share W's tiles in an XCD's L2)

template <class C>
__global__ __launch_bounds__(C::NTHREADS) void head_rows_kernel(
    const typename C::TIn* __restrict__ H, const typename C::TIn* __restrict__ W, int T, int d, int V,
    HeadRows rows, int row0, float* __restrict__ ztok, float4* __restrict__ part, int n_vtiles, int tiles_per_split,
    int n_tblocks, int n_splits) {
  using TileT = typename C::TileT;
  using L = typename TileT::L;
  constexpr int MBK = TileT::MBK, NBK = TileT::NBK, BLK = L::BLK, RPB = L::RPB;
  static_assert(L::GROUPS == 2 && BLK == 32 && (NBK == 1 || NBK == 2), "columns of a wave");
  __shared__ __attribute__((aligned(16))) char smem[C::LDS_BYTES];
  const int lane = threadIdx.x & 63;
  const int wave = wave_id();
  const int wave_m = wave / C::WAVES_N, wave_n = wave % C::WAVES_N;
  int tblock, split;
  grouped_mn(xcd_remap(blockIdx.x, n_tblocks * n_splits), n_tblocks, n_splits, kGroupRows, tblock, split);
  const int t0 = tblock * C::BN;
  // packed rows: those past the last kept one are never read
  const int kept = rows.n != nullptr ? *rows.n - row0 : T;
  if (t0 >= kept) return;
  const int vt0 = split * tiles_per_split;
  const int vt1 = min(n_vtiles, vt0 + tiles_per_split);
  const int own_nb = NBK == 1 ? 0 : lane / 32;
  const int own_row = t0 + wave_n * C::WN + own_nb * BLK + (lane & 31);
  const int own_tok = own_row < min(T, kept) ? token_column(rows, row0 + own_row, V) : -1;
  float rm = -INFINITY, rs = 0.f, re = 0.f;

  TileT tile;
  constexpr bool kAhead = PrefetchOK<C>::value;  // the next tile's first slices go out behind a tile's epilogue
  const typename C::TIn* Ht0 = H + (int64_t)t0 * d;
  if constexpr (kAhead)
    if (vt0 < vt1) tile_k64_prologue<C>(W + (int64_t)vt0 * C::BM * d, d, V - vt0 * C::BM, Ht0, d, T - t0, d, smem);
  for (int vt = vt0; vt < vt1; ++vt) {
    const int v0 = vt * C::BM;
    if constexpr (kAhead)
      run_mma<C, true>(tile, W + (int64_t)v0 * d, d, V - v0, Ht0, d, T - t0, d, smem);
    else
      run_mma(tile, W + (int64_t)v0 * d, d, V - v0, Ht0, d, T - t0, d, smem);
    if constexpr (kAhead)
      if (vt + 1 < vt1)
        tile_k64_prologue<C>(W + (int64_t)(v0 + C::BM) * d, d, V - v0 - C::BM, Ht0, d, T - t0, d, smem);
    const int vbase = v0 + wave_m * C::WM;
    const bool full = vbase + C::WM <= V;  // every row of the wave's slice is a vocabulary row
#pragma unroll
    for (int nb = 0; nb < NBK; ++nb) {
      const int src = NBK == 1 ? lane : (lane & 31) + nb * 32;  // the owner of this lane's column
      const bool own = NBK == 1 || own_nb == nb;
      if (!full) {  // the last tile: columns past the vocabulary count for nothing
#pragma unroll
        for (int mb = 0; mb < MBK; ++mb)
#pragma unroll
          for (int r = 0; r < RPB; ++r)
            if (vbase + mb * BLK + L::row_in(r, lane) >= V) tile.acc[mb][nb][r] = -INFINITY;
      }
      // the token's logit, by the lane that holds it
      const int vl = __shfl(own_tok, src) - vbase;
      if (vl >= 0 && vl < C::WM && L::group_of(vl & 31) == lane / 32) {
        const int sel = (vl / BLK) * RPB + L::reg_of(vl & 31);
        float z = 0.f;
#pragma unroll
        for (int q = 0; q < MBK * RPB; ++q) z = (q == sel) ? tile.acc[q / RPB][nb][q % RPB] : z;
        ztok[opaque(t0 + wave_n * C::WN + nb * BLK + (lane & 31))] = z;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int mb = 0; mb < MBK; ++mb)
#pragma unroll
        for (int r = 0; r < RPB; ++r) mx = fmaxf(mx, tile.acc[mb][nb][r]);
      mx = fmaxf(mx, __shfl_xor(mx, 32)) * kLog2e;
      const float crm = __shfl(rm, src);
      const float mn = fmaxf(crm, mx);
      const float ref = mn == -INFINITY ? 0.f : mn;
      float ssum = 0.f, esum = 0.f;
      if (full) {
#pragma unroll
        for (int mb = 0; mb < MBK; ++mb)
#pragma unroll
          for (int r = 0; r < RPB; ++r) {
            const float x = tile.acc[mb][nb][r] * kLog2e - ref, u = fast_exp2(x);
            ssum += u;
            esum = fmaf(u, x, esum);
          }
      }
      if (!full || esum != esum) {  // (there are -infinities, which count for nothing, or a NaN, which stays)
        ssum = esum = 0.f;
#pragma unroll
        for (int mb = 0; mb < MBK; ++mb)
#pragma unroll
          for (int r = 0; r < RPB; ++r) {
            float x = tile.acc[mb][nb][r] * kLog2e - ref;
            x = x < kExpZero ? kExpZero : x;
            const float u = fast_exp2(x);
            ssum += u;
            esum = fmaf(u, x, esum);
          }
      }
      ssum += __shfl_xor(ssum, 32);
      esum += __shfl_xor(esum, 32);
      if (own && (mn > -INFINITY || ssum != ssum)) {
        const float dm = fmaxf(rm - mn, kExpZero), f = fast_exp2(dm);
        re = fmaf(f, fmaf(dm, rs, re), esum);
        rs = fmaf(f, rs, ssum);
        rm = mn;
      }
    }
  }

  // the waves that share the same rows
  wait_vmcnt<0>();
  __syncthreads();
  float4* red = reinterpret_cast<float4*>(smem);  // [WAVES_M][BN]
  static_assert(C::WAVES_M * C::BN * 16 <= C::LDS_BYTES, "states");
  if (NBK == 2 || lane < 32) red[wave_m * C::BN + wave_n * C::WN + lane] = make_float4(rm, rs, re, 0.f);
  __syncthreads();
  for (int i = threadIdx.x; i < C::BN; i += C::NTHREADS) {
    float4 a = red[i];
#pragma unroll
    for (int w = 1; w < C::WAVES_M; ++w) {
      const float4 b = red[w * C::BN + i];
      ent2_merge(a.x, a.y, a.z, b.x, b.y, b.z);
    }
    if (t0 + i < T) part[(int64_t)split * T + t0 + i] = a;
  }
}

// Packed row row0 + i: LANES lanes merge its splits ([S][count], with ztok from row0
// on) into its row of the call; and row row0 + i of the call, where it is masked,
// gets zeros.  (Few rows have many splits: 8 rows of 786 splits with 16 lanes 19 us.)
template <int LANES>
__global__ __launch_bounds__(256) void head_finish_kernel(const float4* __restrict__ part, int S, int count, int V,
                                                          HeadRows rows, int row0, const float* __restrict__ ztok,
                                                          float* __restrict__ logprob, float* __restrict__ entropy,
                                                          float* __restrict__ lse) {
  const int sub = threadIdx.x & (LANES - 1);
  const int i = blockIdx.x * (256 / LANES) + threadIdx.x / LANES, p = row0 + i;
  const bool live = i < count && (rows.n == nullptr || p < *rows.n);
  float m = -INFINITY, s = 0.f, e = 0.f;
  if (live)
    for (int k0 = sub; k0 < S; k0 += 4 * LANES) {
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = k0 + j * LANES < S ? part[(int64_t)(k0 + j * LANES) * count + i] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) ent2_merge(m, s, e, v[j].x, v[j].y, v[j].z);
    }
#pragma unroll
  for (int o = 1; o < LANES; o *= 2) {
    const float om = __shfl_xor(m, o), os = __shfl_xor(s, o), oe = __shfl_xor(e, o);
    ent2_merge(m, s, e, om, os, oe);
  }
  if (sub == 1 && i < count && rows.rank != nullptr && rows.rank[p] < 0) logprob[p] = entropy[p] = lse[p] = 0.f;
  if (sub != 0 || !live) return;
  const int t = rows.perm != nullptr ? rows.perm[p] : p;
  const float l2 = fast_log2(s), l = (m + l2) * kLn2;
  const float ent = s == 0.f ? 0.f : (l2 - e / s) * kLn2;
  lse[t] = l;
  entropy[t] = ent < 0.f ? 0.f : ent;
  float z = 0.f;
  if (token_column(rows, p, V) >= 0) {
    z = ztok[i];
    // from differences, as z - l would carry the rounding of l (-infinity has that log probability in a row of nothing
    // else, too)
    if (z != -INFINITY || l != l) z = (fmaf(z, kLog2e, -m) - l2) * kLn2;
  }
  logprob[t] = z;
}

// --------------------------------------------------------------- backward --
// With q = 2^x, x = z log2 e - lse log2 e, the gradient of a row's logits is
//   q (c0 + c1 x) + 1[v = token] a,   c0 = -(a + b entropy),   c1 = -b ln 2
// for its incoming gradients a (log probability) and b (entropy); q carries the
// rounding of lse, 2^-24 |lse|.  Row i:
// consts[i] = (c0, lse log2 e, c1, a), its token.  Rows past the last one and rows
// with no gradient get an lse that makes q zero.
__global__ __launch_bounds__(256) void head_consts_kernel(HeadRows rows, int T, int Tp, int V,
                                                          const float* __restrict__ lse,
                                                          const float* __restrict__ entropy,
                                                          const float* __restrict__ dlogprob,
                                                          const float* __restrict__ dentropy,
                                                          float4* __restrict__ consts, int* __restrict__ tok) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= Tp) return;
  int c = -1;
  float4 k = make_float4(0.f, 1e30f, 0.f, 0.f);
  if (i < (rows.n != nullptr ? *rows.n : T)) {
    const int t = rows.perm != nullptr ? rows.perm[i] : i;
    c = token_column(rows, i, V);
    const float a = c >= 0 && dlogprob != nullptr ? dlogprob[t] : 0.f;
    const float b = dentropy != nullptr ? dentropy[t] : 0.f;
    if (!(a == 0.f && b == 0.f))
      k = make_float4(b == 0.f ? -a : -(a + b * entropy[t]), lse[t] * kLog2e, -b * kLn2, a);
  }
  consts[i] = k;
  tok[i] = c;
}

// A block's rows by the 64 words that hold their token, in their order: a workgroup
// lists four such groups, behind the number of rows whose token lies below them (2048
// rows are 8 KB, read by every workgroup from the caches; 786 groups of 256 words 10 us).
__global__ __launch_bounds__(256) void head_buckets_kernel(const int* __restrict__ tok, int T, int Tc,
                                                           const int* __restrict__ n, int* __restrict__ order,
                                                           int* __restrict__ start) {
  __shared__ int counts[5][4], mine[2][4][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int v0 = blockIdx.x * 256;
  if (n != nullptr) T = min(T, *n);
  const int t0 = blockIdx.y * Tc;
  T = min(T, t0 + Tc);
  start += blockIdx.y * (gridDim.x * 4 + 1);
  int sum[5] = {};  // rows below the four groups, in the first, ..
  for (int i = t0 + threadIdx.x; i < T; i += 256) {
    const int c = tok[i], g = (c - v0) >> 6;
    sum[0] += c >= 0 && c < v0 ? 1 : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k + 1] += c >= v0 && g == k ? 1 : 0;
  }
#pragma unroll
  for (int k = 0; k < 5; ++k) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum[k] += __shfl_xor(sum[k], o);
    if (lane == 0) counts[k][wave] = sum[k];
  }
  __syncthreads();
  int at[4], all = t0;
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    all += counts[k][0] + counts[k][1] + counts[k][2] + counts[k][3];
    if (k < 4) at[k] = all;
  }
  if (threadIdx.x == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) start[blockIdx.x * 4 + k] = at[k];
    if (blockIdx.x == gridDim.x - 1) start[gridDim.x * 4] = all;
  }
  if (all == at[0]) return;  // no row's token is here
  int side = 0;
  for (int i0 = t0; i0 < T; i0 += 256) {
    const int i = i0 + threadIdx.x;
    const int c = i < T ? tok[i] : -1;
    const int g = c >= v0 && c < v0 + 256 ? (c - v0) >> 6 : -1;
    uint64_t who[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      who[k] = __ballot(g == k);
      if (lane == 0) mine[side][k][wave] = __popcll(who[k]);
    }
    __syncthreads();  // (the other side is written only after everyone has passed the next barrier)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      int p = at[k] + __popcll(who[k] & ((1ull << lane) - 1));
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        p += w < wave ? mine[side][k][w] : 0;
        at[k] += mine[side][k][w];
      }
      if (g == k) order[p] = i;
    }
    side ^= 1;
  }
}

// A block of rows of dH from its parts, what earlier blocks of words left (`sums`, may
// be NULL and may be `out`) and the tokens' entries, eight columns a thread; zeros in
// the block's rows of the call that are masked.  Bound by the parts' bytes.
template <typename TOut>
__global__ __launch_bounds__(256) void head_dh_kernel(const float* __restrict__ part, int64_t stride, int S,
                                                      const float* sums, int row0, int count, int nv,
                                                      const int* __restrict__ tok, const float* __restrict__ gtok,
                                                      const bf16_t* __restrict__ W, HeadRows rows, TOut* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(i / nv), c = (int)(i - (int64_t)t * nv), r = row0 + t;
  if (t >= count) return;
  float a[8] = {}, b[8];
  if (rows.rank != nullptr && rows.rank[r] < 0) store8(out + ((int64_t)r * nv + c) * 8, a);
  if (rows.n != nullptr && r >= *rows.n) return;
  const float* p = part + i * 8;
  int s = 0;
  if (sums != nullptr)
    load8(sums + ((int64_t)r * nv + c) * 8, a);
  else
    load8(p, a), s = 1;
#pragma unroll 4
  for (; s < S; ++s) {
    load8(p + s * stride, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] += b[j];
  }
  const int k = gtok != nullptr ? tok[r] : -1;
  if (k >= 0) {
    const float g = gtok[r];
    load8(W + ((int64_t)k * nv + c) * 8, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = fmaf(g, b[j], a[j]);
  }
  store8(out + ((int64_t)(rows.perm != nullptr ? rows.perm[r] : r) * nv + c) * 8, a);
}

// The same from parts of dH's transpose ([d][ldt]): 32 rows by 8 columns a workgroup,
// turned in the LDS; a thread sums one element, as there may be hundreds of parts (500
// x 256 of 196 20 us, by four elements a thread 210; 16 x 2048 of 63 9 and 66).
template <typename TOut>
__global__ __launch_bounds__(256) void head_dh_t_kernel(const float* __restrict__ part, int64_t stride, int64_t ldt,
                                                        int S, int T, int d, const int* __restrict__ tok,
                                                        const float* __restrict__ gtok, const bf16_t* __restrict__ W,
                                                        HeadRows rows, TOut* __restrict__ dH) {
  __shared__ float turn[8][33];
  const int c0 = blockIdx.y * 8, t0 = blockIdx.x * 32;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int t = t0 + tx;
  const int r = t >= T ? -1 : rows.rank != nullptr ? rows.rank[t] : t;
  float a = 0.f;
  if (r >= 0) {
    const float* p = part + (int64_t)(c0 + ty) * ldt + r;
#pragma unroll 16
    for (int s = 0; s < S; ++s) a += p[s * stride];
  }
  turn[ty][tx] = a;
  __syncthreads();
  if (threadIdx.x >= 32 || t >= T) return;
  float f[8], w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = turn[j][tx];
  const int k = r >= 0 ? tok[r] : -1;
  if (k >= 0) {
    const float g = gtok[r];
    load8(W + (int64_t)k * d + c0, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = fmaf(g, w[j], f[j]);
  }
  store8(dH + (int64_t)t * d + c0, f);
}

// The G block of rows [tb0, tb0 + BN n_tblocks) and columns [vb0, vb0 + BM
// n_vtiles): G[t - tb0][v - vb0], and for fp32 also its transpose Gt.  bf16 rounds
// G once, to what the contractions read, but for each row's largest entry as a rule,
// its token's: that one stays in fp32 (gtok[t], 0 in G) and is added to dH and dW as
// gtok W[token] and gtok H[t], so that its rounding, which a whole row of dH would
// share, does not come on top of theirs.  Rows past T and columns past V get 0.  Tiles leave through
// the LDS as 512-byte runs of G's rows, behind the issue of the next tile's first
// slices.  Bound by the matrix units: 2048 x 2880 by 201088 words bf16 2.1 ms, of which
// 0.25 over head_rows are the 0.8 GB of G.
template <class C>
__global__ __launch_bounds__(C::NTHREADS) void head_grad_kernel(
    const typename C::TIn* __restrict__ H, const typename C::TIn* __restrict__ W, int T, int d, int V,
    const float4* __restrict__ consts, const int* __restrict__ tok, float* __restrict__ gtok, int tb0, int vb0,
    int n_vtiles, int tiles_per_split, int n_tblocks, int n_splits, typename C::TIn* __restrict__ G, int64_t ldG,
    typename C::TIn* __restrict__ Gt, int64_t ldGt, const int* __restrict__ nrows) {
  using TIn = typename C::TIn;
  constexpr bool kStage = std::is_same<TIn, bf16_t>::value;
  static_assert(!kStage || (C::BM == 256 && C::BN == 256 && C::WM == 128 && C::LDS_BYTES >= 256 * 256 * 2 &&
                            PrefetchOK<C>::value), "staged tiles");
  __shared__ __attribute__((aligned(16))) char smem[C::LDS_BYTES + C::BN * 20];
  float4* s_row = reinterpret_cast<float4*>(smem + C::LDS_BYTES);
  int* s_tok = reinterpret_cast<int*>(smem + C::LDS_BYTES + C::BN * 16);
  uint16_t* stg = reinterpret_cast<uint16_t*>(smem);
  // 16-byte chunk c of row t sits at c ^ (t / 8): the column reads of eight rows spread over the banks
  auto stage_chunk = [](int t, int c) { return c ^ ((t >> 3) & 31); };
  (void)stg;
  (void)stage_chunk;
  const int lane = threadIdx.x & 63;
  const int wave = wave_id();
  const int wave_m = wave / C::WAVES_N, wave_n = wave % C::WAVES_N;
  int tblock, split;
  grouped_mn(xcd_remap(blockIdx.x, n_tblocks * n_splits), n_tblocks, n_splits, kGroupRows, tblock, split);
  const int t0 = tb0 + tblock * C::BN;
  if (nrows != nullptr && t0 >= *nrows) return;  // packed rows: the contractions read no G row of this block
  const int vt0 = split * tiles_per_split;
  const int vt1 = min(n_vtiles, vt0 + tiles_per_split);
  for (int i = threadIdx.x; i < C::BN; i += C::NTHREADS) {
    s_row[i] = consts[t0 + i];
    s_tok[i] = tok[t0 + i];
  }
  __syncthreads();
  typename C::TileT tile;
  const TIn* Ht0 = H + (int64_t)t0 * d;
  if constexpr (kStage)
    if (vt0 < vt1)
      tile_k64_prologue<C>(W + (int64_t)(vb0 + vt0 * C::BM) * d, d, V - vb0 - vt0 * C::BM, Ht0, d, T - t0, d, smem);
  for (int vt = vt0; vt < vt1; ++vt) {
    const int v0 = vb0 + vt * C::BM;
    if constexpr (kStage)
      run_mma<C, true>(tile, W + (int64_t)v0 * d, d, V - v0, Ht0, d, T - t0, d, smem);
    else
      run_mma(tile, W + (int64_t)v0 * d, d, V - v0, Ht0, d, T - t0, d, smem);
    const int vbase = v0 + wave_m * C::WM;
    const bool full = vbase + C::WM <= V;
#pragma unroll
    for (int nb = 0; nb < C::NB; ++nb) {
      const int tl = opaque(wave_n * C::WN + nb * 32 + (lane & 31));  // (formed here, not held across the loop)
      const float4 rc = s_row[tl];
#pragma unroll
      for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float x = tile.acc[mb][nb][r] * kLog2e - rc.y;
          tile.acc[mb][nb][r] = fast_exp2(x) * fmaf(rc.z, x, rc.x);
        }
      if (!full) {
#pragma unroll
        for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (vbase + mb * 32 + acc_row(r, lane) >= V) tile.acc[mb][nb][r] = 0.f;
      }
      const int tk = s_tok[tl], vl = tk - vbase;
      if (tk >= 0 && vl >= 0 && vl < C::WM && ((vl >> 2) & 1) == lane / 32) {
        const int sel = (vl >> 5) * 16 + ((vl & 31) >> 3) * 4 + (vl & 3);
#pragma unroll
        for (int q = 0; q < C::MB * 16; ++q)
          if (q == sel) {
            const float g = tile.acc[q / 16][nb][q % 16] + rc.w;
            tile.acc[q / 16][nb][q % 16] = kStage ? 0.f : g;
            if (kStage) gtok[t0 + tl] = g;
          }
      }
      if constexpr (kStage) {
        uint2* row = reinterpret_cast<uint2*>(stg + tl * 256);
#pragma unroll
        for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            row[stage_chunk(tl, wave_m * 16 + mb * 4 + i) * 2 + (lane >> 5)] =
                make_uint2(pack_bf16x2(tile.acc[mb][nb][4 * i], tile.acc[mb][nb][4 * i + 1]),
                           pack_bf16x2(tile.acc[mb][nb][4 * i + 2], tile.acc[mb][nb][4 * i + 3]));
      } else {
        const int64_t trow = t0 + tl - tb0;
#pragma unroll
        for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int vcol = vbase - vb0 + mb * 32 + acc_row(r, lane);
            Gt[(int64_t)vcol * ldGt + trow] = tile.acc[mb][nb][r];
          }
#pragma unroll
        for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f32x4*>(G + trow * ldG + (vbase - vb0 + mb * 32 + 8 * i + 4 * (lane >> 5))) =
                f32x4{tile.acc[mb][nb][4 * i], tile.acc[mb][nb][4 * i + 1], tile.acc[mb][nb][4 * i + 2],
                      tile.acc[mb][nb][4 * i + 3]};
      }
    }
    if constexpr (kStage) {
      __syncthreads();
      const int tid = opaque(threadIdx.x);
      constexpr int kPasses = 256 / (C::NTHREADS / 32);
      u32x4 out[kPasses];
#pragma unroll
      for (int pass = 0; pass < kPasses; ++pass) {
        const int tl = pass * (C::NTHREADS / 32) + (tid >> 5), q = tid & 31;
        out[pass] = reinterpret_cast<const u32x4*>(stg + tl * 256)[stage_chunk(tl, q)];
      }
      __syncthreads();
      if (vt + 1 < vt1)
        tile_k64_prologue<C>(W + (int64_t)(v0 + C::BM) * d, d, V - v0 - C::BM, Ht0, d, T - t0, d, smem);
      bf16_t* Gtile = reinterpret_cast<bf16_t*>(G) + (int64_t)(t0 - tb0) * ldG + (v0 - vb0);
#pragma unroll
      for (int pass = 0; pass < kPasses; ++pass) {
        const int tl = pass * (C::NTHREADS / 32) + (tid >> 5), q = tid & 31;
        __builtin_nontemporal_store(out[pass], reinterpret_cast<u32x4*>(Gtile + (int64_t)tl * ldG + q * 8));
      }
    }
  }
}

}  // namespace

// -------------------------------------------------------------- launchers --
#define CKL_LAUNCH_CHECK() \
  do { hipError_t e_ = hipGetLastError(); if (e_ != hipSuccess) return e_; } while (0)

enum { kF32, kF32Small, kF32Slim, kWide, kMiddle, kNarrow, kSlim };
template <typename F>
void by_tile(int kind, F&& f) {
  switch (kind) {
    case kF32: f(CfgF32{}); break;
    case kF32Small: f(CfgF32Small{}); break;
    case kF32Slim: f(CfgF32Slim{}); break;
    case kWide: f(CfgWide{}); break;
    case kMiddle: f(CfgMiddle{}); break;
    case kNarrow: f(CfgNarrow{}); break;
    default: f(CfgSlim{}); break;
  }
}

HeadTile head_tile(int in_bf16, int64_t rows, int64_t V) {
  int kind;
  if (in_bf16)
    kind = rows <= 32 ? kSlim : rows <= 64 ? kNarrow : rows <= 128 ? kMiddle : kWide;
  else
    // (fp32, us, 64 x 64 / 128 x 128: 64 rows of 520, 5003 words 18 / 44, 301 of them 28 / 46; 500 of 768, 32000 words
    // 245 / 230, 2048 of 1024 1237 / 1092)
    kind = rows <= 32 ? kF32Slim : (rows + 127) / 128 * ((V + 127) / 128) < 512 ? kF32Small : kF32;
  HeadTile t{kind, 0, 0, 0};
  by_tile(kind, [&](auto cfg) {
    using C = decltype(cfg);
    t.BM = C::BM;
    t.BN = C::BN;
    t.slots = 256 * (163840 / C::LDS_BYTES > 4 ? 4 : 163840 / C::LDS_BYTES);
  });
  return t;
}

hipError_t launch_head_rows(const HeadTile& k, const void* H, const void* W, int T, int d, int V, const HeadRows& rows,
                            int row0, float* ztok, float4* part, int n_splits, int tiles_per_split, hipStream_t st) {
  const int n_vtiles = (V + k.BM - 1) / k.BM, n_tblocks = (T + k.BN - 1) / k.BN;
  auto go = [&](auto cfg) {
    using C = decltype(cfg);
    using TIn = typename C::TIn;
    head_rows_kernel<C><<<n_tblocks * n_splits, C::NTHREADS, 0, st>>>((const TIn*)H, (const TIn*)W, T, d, V, rows, row0,
                                                                      ztok, part, n_vtiles, tiles_per_split, n_tblocks,
                                                                      n_splits);
  };
  by_tile(k.kind, go);
  CKL_LAUNCH_CHECK();
  return hipSuccess;
}

hipError_t launch_head_finish(const float4* part, int S, int count, int V, const HeadRows& rows, int row0,
                              const float* ztok, float* logprob, float* entropy, float* lse, hipStream_t st) {
  if (S > 64)
    head_finish_kernel<64><<<(count + 3) / 4, 256, 0, st>>>(part, S, count, V, rows, row0, ztok, logprob, entropy, lse);
  else
    head_finish_kernel<16><<<(count + 15) / 16, 256, 0, st>>>(part, S, count, V, rows, row0, ztok, logprob, entropy,
                                                             lse);
  CKL_LAUNCH_CHECK();
  return hipSuccess;
}

hipError_t launch_head_consts(const HeadRows& rows, int T, int Tp, int V, const float* lse, const float* entropy,
                              const float* dlogprob, const float* dentropy, float4* consts, int* tok, hipStream_t st) {
  head_consts_kernel<<<(Tp + 255) / 256, 256, 0, st>>>(rows, T, Tp, V, lse, entropy, dlogprob, dentropy, consts, tok);
  CKL_LAUNCH_CHECK();
  return hipSuccess;
}

hipError_t launch_head_buckets(const int* tok, int T, int Tc, const int* n, int tiles, int* order, int* start,
                               hipStream_t st) {
  head_buckets_kernel<<<dim3(tiles, (T + Tc - 1) / Tc), 256, 0, st>>>(tok, T, Tc, n, order, start);
  CKL_LAUNCH_CHECK();
  return hipSuccess;
}

hipError_t launch_head_dh(const float* part, int64_t stride, int S, const float* sums, int row0, int count, int d,
                          const int* tok, const float* gtok, const void* W, const HeadRows& rows, void* out,
                          int out_bf16, hipStream_t st) {
  const unsigned blocks = (unsigned)(((int64_t)count * (d / 8) + 255) / 256);
  if (out_bf16)
    head_dh_kernel<<<blocks, 256, 0, st>>>(part, stride, S, sums, row0, count, d / 8, tok, gtok, (const bf16_t*)W, rows,
                                           (bf16_t*)out);
  else
    head_dh_kernel<<<blocks, 256, 0, st>>>(part, stride, S, sums, row0, count, d / 8, tok, gtok, (const bf16_t*)W, rows,
                                           (float*)out);
  CKL_LAUNCH_CHECK();
  return hipSuccess;
}

hipError_t launch_head_dh_t(const float* part, int64_t stride, int64_t ldt, int S, int T, int d, const int* tok,
                            const float* gtok, const void* W, const HeadRows& rows, void* dH, int dh_bf16,
                            hipStream_t st) {
  const dim3 grid((T + 31) / 32, d / 8);
  if (dh_bf16)
    head_dh_t_kernel<<<grid, 256, 0, st>>>(part, stride, ldt, S, T, d, tok, gtok, (const bf16_t*)W, rows, (bf16_t*)dH);
  else
    head_dh_t_kernel<<<grid, 256, 0, st>>>(part, stride, ldt, S, T, d, tok, gtok, (const bf16_t*)W, rows, (float*)dH);
  CKL_LAUNCH_CHECK();
  return hipSuccess;
}

hipError_t launch_head_grad(int in_bf16, const void* H, const void* W, int T, int d, int V, const float4* consts,
                            const int* tok, float* gtok, int tb0, int t_rows, int vb0, int v_rows, int tiles_per_split,
                            void* G, int64_t ldG, void* Gt, int64_t ldGt, const int* nrows, hipStream_t st) {
  auto go = [&](auto cfg, int tps) {
    using C = decltype(cfg);
    using TIn = typename C::TIn;
    const int n_vtiles = v_rows / C::BM, n_tblocks = t_rows / C::BN, splits = (n_vtiles + tps - 1) / tps;
    head_grad_kernel<C><<<n_tblocks * splits, C::NTHREADS, 0, st>>>(
        (const TIn*)H, (const TIn*)W, T, d, V, consts, tok, gtok, tb0, vb0, n_vtiles, tps, n_tblocks, splits, (TIn*)G,
        ldG, (TIn*)Gt, ldGt, nrows);
  };
  // (fp32 by 64 x 64, us, against 128 x 128: 226 rows of 520, 5003 words 30 and 48; 1000 of 512, 2000 words 44 and 93;
  // 2048 of 1024, 32000 words 1274 and 1282)
  if (in_bf16)
    go(CfgWide{}, tiles_per_split);
  else
    go(CfgF32Small{}, 1);
  CKL_LAUNCH_CHECK();
  return hipSuccess;
}

}  // namespace ckl
