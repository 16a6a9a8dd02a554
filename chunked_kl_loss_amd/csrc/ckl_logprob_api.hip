// Host side of the log probabilities of given tokens, from logits and from hidden
// states and the output head: argument checks, workspaces and launch sequences
// behind the C ABI declared in include/ckl.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/ckl.h"
#include "ckl_head.hpp"
#include "ckl_host.hpp"
#include "ckl_kernels.hpp"
#include "ckl_ops.hpp"

using namespace ckl::host;

namespace {

ckl_status check_logprob(int64_t T, int64_t V, int64_t top) {
  ckl_status s = check_rows(T);
  if (s == CKL_OK) s = check_vocab(V);
  if (s != CKL_OK) return s;
  if (top < 0 || top > V) return fail(CKL_ERR_INVALID_ARG, "top=%lld must satisfy 0 <= top <= V", (long long)top);
  if (top > kMaxK) return fail(CKL_ERR_UNSUPPORTED, "top=%lld exceeds %lld", (long long)top, (long long)kMaxK);
  if (T * top >= ((int64_t)1 << 31)) return fail(CKL_ERR_UNSUPPORTED, "T*top must stay below 2^31");
  if (T * ceil_div(V + 7, 8192) >= ((int64_t)1 << 31)) return fail(CKL_ERR_UNSUPPORTED, "T*V is too large");
  return CKL_OK;
}
ckl_status check_tokens(const void* tokens, int32_t token_bytes) {
  if (token_bytes != 4 && token_bytes != 8) return fail(CKL_ERR_INVALID_ARG, "token_bytes must be 4 or 8");
  if ((uintptr_t)tokens & (uintptr_t)(token_bytes - 1))
    return fail(CKL_ERR_INVALID_ARG, "tokens must be aligned to their size");
  return CKL_OK;
}
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// Words and sums of the row segments.
struct LogprobWs {
  size_t cand, state, state_e, total;
};
LogprobWs logprob_layout(int64_t T, int64_t V, int64_t top) {
  LogprobWs w{};
  int segments = 1;
  int64_t cols = 0;
  if (T > 0 && top > 0 && !ckl::logprob_in_registers(V, top)) ckl::topk_plan(T, V, &segments, &cols);
  if (segments > 1) {
    const size_t n = (size_t)T * segments;
    w.state = align256(n * ckl::topk_segment_words(top) * 8);
    w.state_e = w.state + align256(n * 8);
    w.total = w.state_e + align256(n * 4);
  }
  return w;
}

// ---------------------------------------------------------- states and head --
// Row padding (elements) of the matrices whose leading dimension is chosen here:
// 256 bytes keep the rows of a load on different memory channels.
constexpr int64_t kLdPad = 128;
constexpr int64_t kTileElements = (int64_t)1 << 30;  // of bf16, what a tile's byte offsets reach
// Rows a launch of the forward takes (8192 rows of 512, 1000 words, bf16, in launches of 2048 97 us, in one 25;
// 32768 of 1024, 50264 words, in 16 3048, in two 2700).
constexpr int64_t kForwardRows = 16384;
// Columns of W whose transpose costs as much as one more tile of dH (its transpose against dH, us, with dW, 201088
// words of 2880: 16 rows 1090 and 1540, 300 1650 and 2190, 1024, of 12 more tiles, 3660 and 3920, 2048, of 12 more,
// 6550 and 6890; 100000 words: 512 rows of 264, 2 more, 263 and 288, 1024 of 520, 4 more, 598 and 590, 2048 of 1544,
// 9 more, 2090 and 2065, 1024 of 264, 4 more, 431 and 390).
constexpr int64_t kTurnedTile = 230;
// Rows up to which dH's transpose takes tiles of 256 x 64, in a launch of its own, instead of 256 x 320 beside dW's (us, dH
// with dW and alone: 16 rows of 2880, 201088 words 1027 and 500, against 1089 and 623; 64 of 2048, 32000 words 167 and
// 84, 193 and 110; 64 of 64, 100000 words 88 and 49, 95 and 60; 64 of 512, 1000 words 63 and 35, 58 and 48, where the
// second launch costs more than the wide tiles: the one of these that a rule by rows alone loses).
constexpr int64_t kNarrowRows = 64;
constexpr int64_t kGradSlots = 256;  // workgroups of head_grad at once: one to a compute unit

// Vocabulary splits of a launch over row blocks: the count that finishes in the
// fewest rounds of tiles, and among equals the fewest splits.
void pick_splits(int64_t row_blocks, int64_t vtiles, int64_t slots, int64_t* splits, int64_t* tps) {
  int64_t best = -1;
  for (int64_t s = 1; s <= vtiles; ++s) {
    const int64_t t = ceil_div(vtiles, s), sp = ceil_div(vtiles, t);
    if (sp != s) continue;  // the same as fewer
    const int64_t cost = ceil_div(row_blocks * sp, slots) * t;
    if (best < 0 || cost < best) {
      best = cost;
      *splits = sp;
      *tps = t;
    }
  }
}

struct HeadPlan {
  int bf16;
  size_t esz;
  int64_t T, d, V;
  // forward: chunks of Cs rows
  ckl::HeadTile tile;
  int64_t Cs, nS, splits, tps;
  // backward: G blocks of Tc rows x Vc columns; dH as Sh sums over Vs columns of a block each
  int64_t BM, BN, Tp, Vp, Tc, Vc, nT, nV, Sh, Vs;
  int64_t dh_rows;  // rows (turned: columns) of a part of dH: a block's
  bool carried;  // rows and words are both cut: dH's sums go from one block of words to the next in fp32 [T][d]
  bool narrow;  // turned, and of so few rows that narrow tiles hold them
  bool turned;  // the sums are of dH's transpose, which needs no transpose of W
};
ckl_status head_plan(int64_t T, int64_t d, int64_t V, int64_t chunk, int32_t in_dtype, int32_t dh_dtype,
                     int32_t dw_dtype, HeadPlan* q) {
  if (T < 0) return fail(CKL_ERR_INVALID_ARG, "T=%lld must be >= 0", (long long)T);
  chunk = std::min(chunk, kMaxRows);
  ckl_problem p{};
  p.T = std::max<int64_t>(T, 1);
  p.d = d;
  p.V = V;
  p.K = 1;
  // (the plan takes half its budget for bf16, which keeps no transpose: all of it here, and the vocabulary's padding
  // to whole tiles, so that a chunk of rows is one block.)
  const int64_t bm = ckl::tile_rows_m(1);
  p.chunk = in_dtype == CKL_BF16 && V > 0 ? ceil_div(2 * chunk * round_up(V, bm), V) : chunk;
  p.in_dtype = in_dtype;
  p.dh_dtype = dh_dtype;
  p.dw_dtype = dw_dtype;
  int64_t blocks[5];
  ckl_status s = ckl_backward_plan(&p, blocks);  // (checks the sizes)
  if (s != CKL_OK) return s;
  q->bf16 = in_dtype == CKL_BF16;
  q->esz = esize(in_dtype);
  q->T = T;
  q->d = d;
  q->V = V;
  q->BM = ckl::tile_rows_m(q->bf16);
  q->BN = ckl::tile_rows_n(q->bf16);
  q->Tp = round_up(p.T, q->BN);
  q->Vp = round_up(V, q->BM);
  q->Tc = blocks[0];
  q->Vc = blocks[1];
  q->nT = blocks[2];
  q->nV = blocks[3];
  // dH has few tiles of a long sum, dW many of a short one: dH is cut into parts of about a quarter of a compute
  // unit's share of both (but not below the 512 columns that cost as much as storing a part's tile)
  const int64_t gm = ckl::gemm_tile_m(q->bf16), gn = ckl::gemm_tile_n(q->bf16);
  int64_t dh_tiles = ceil_div(q->Tc, gm) * ceil_div(d, gn);
  const int64_t dw_tiles = ceil_div(q->Vc, gm) * ceil_div(d, gn);
  // One block of rows, bf16: dH^T = W^T G^T reads W as it lies, at the price of tiles the other way round.  (More blocks
  // share one transpose of W.)
  const int64_t turned_tiles = ceil_div(d, gm) * ceil_div(p.T, gn);
  q->turned = q->bf16 && q->nT == 1 && (turned_tiles - dh_tiles) * kTurnedTile <= d &&
              std::min(p.T, gn) * (q->Vc + kLdPad) < kTileElements;
  if (q->turned) dh_tiles = turned_tiles;
  q->dh_rows = q->turned ? round_up(T, 8) : std::min(q->Tc, T);
  q->carried = q->nT > 1 && q->nV > 1;
  // (twice that share where a block's sums pass through memory: half the parts, us, against a quarter's and all of a
  // unit's share: 65536 rows of 1024, 32000 words, chunk 1024 20400, 22000 and 21700; 32768, 50264 words, 2048 12920,
  // 13170 and 13280; 1024 14490, 15150 and 15870; 256 27960, 28700 and 23790)
  const int64_t share = (dh_tiles * q->Vc + dw_tiles * q->Tc) / (kGradSlots * (q->carried ? 2 : 4));
  q->narrow = q->turned && T <= kNarrowRows;
  if (q->narrow)  // (one round of the two workgroups that a compute unit holds of these tiles)
    q->Vs = std::max<int64_t>(ceil_div(q->Vc, std::max<int64_t>(2 * kGradSlots / dh_tiles, 1)), 512);
  else
    q->Vs = std::max<int64_t>(share, 512);
  q->Vs = std::min(round_up(q->Vs, 64), q->Vc);
  q->Sh = ceil_div(q->turned ? std::min(q->Vc, V) : q->Vc, q->Vs);
  // (the forward keeps 16 bytes a row and split: its blocks of rows need not be short)
  q->Cs = std::min(std::max(round_up(chunk, 256), kForwardRows), round_up(p.T, 256));
  q->nS = ceil_div(p.T, q->Cs);
  const int64_t rows = std::min(q->Cs, p.T);
  q->tile = ckl::head_tile(q->bf16, rows, V);
  pick_splits(ceil_div(rows, q->tile.BN), ceil_div(V, q->tile.BM), q->tile.slots, &q->splits, &q->tps);
  return CKL_OK;
}

struct Layout {
  size_t o = 0;
  size_t take(size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  }
};
// Packed rows of a mask: kept positions, ranks, their number, their states.
struct PackWs {
  size_t perm, rank, N, H;
};
PackWs pack_layout(const HeadPlan& q, Layout* l) {
  PackWs w{};
  w.perm = l->take(q.T * 4);
  w.rank = l->take(q.T * 4);
  w.N = l->take(4);
  w.H = l->take((size_t)q.T * q.d * q.esz);
  return w;
}
struct HeadFwdWs {
  size_t ztok, part, total;
  PackWs pk;
};
HeadFwdWs head_fwd_layout(const HeadPlan& q, bool masked) {
  HeadFwdWs w{};
  Layout l;
  w.ztok = l.take(q.Cs * 4);
  w.part = l.take((size_t)q.splits * q.Cs * 16);
  if (masked) w.pk = pack_layout(q, &l);
  w.total = l.o;
  return w;
}
struct HeadBwdWs {
  size_t consts, tok, gtok, order, start, Ht, Wt, G, Gt, parts, sums, dW, total;
  PackWs pk;
};
// Whether dH is finished from fp32 sums, or is them.
bool dh_summed(const HeadPlan& q, bool masked, int32_t dh_dtype) {
  return q.bf16 || dh_dtype == CKL_BF16 || masked || q.Sh > 1;
}
HeadBwdWs head_bwd_layout(const HeadPlan& q, bool masked, int32_t dh_dtype, int32_t dw_dtype) {
  HeadBwdWs w{};
  Layout l;
  w.consts = l.take(q.Tp * 16);
  w.tok = l.take(q.Tp * 4);
  if (q.bf16) {
    w.gtok = l.take(q.Tp * 4);
    w.order = l.take(q.Tp * 4);
    w.start = l.take(q.nT * (q.Vp / 64 + 1) * 4);
  }
  w.Ht = l.take((size_t)q.d * (q.Tp + kLdPad) * q.esz);
  w.Wt = q.turned ? 0 : l.take((size_t)q.d * (q.Vc + kLdPad) * q.esz);
  w.G = l.take((size_t)q.Tc * (q.Vc + kLdPad) * q.esz);
  w.Gt = q.bf16 ? 0 : l.take((size_t)q.Vc * (q.Tc + kLdPad) * q.esz);
  // dH: one block's parts, which a plan's choice of Vs holds near a tile for each quarter of a compute unit's share,
  // whatever T; and, where it is carried and dH itself cannot hold them, all rows' sums
  if (dh_summed(q, masked, dh_dtype)) {
    if (!q.carried || q.Sh > 1) w.parts = l.take((size_t)q.Sh * q.dh_rows * q.d * 4);
    if (q.carried && (dh_dtype == CKL_BF16 || masked)) w.sums = l.take((size_t)q.T * q.d * 4);
  }
  // fp32 sums of a bf16 dW (bf16 inputs: needed only between blocks of rows)
  w.dW = dw_dtype == CKL_BF16 && (!q.bf16 || q.nT > 1) ? l.take((size_t)q.V * q.d * 4) : 0;
  if (masked) w.pk = pack_layout(q, &l);
  w.total = l.o;
  return w;
}

// Packs the kept rows of a mask: *H and *rows become theirs.
hipError_t head_pack(const HeadPlan& q, char* b, const PackWs& w, const uint8_t* mask, const void** H,
                     ckl::HeadRows* rows, hipStream_t st) {
  int *perm = (int*)(b + w.perm), *rank = (int*)(b + w.rank), *n = (int*)(b + w.N);
  hipError_t e =
      timed(CKL_KERNEL_OTHER, st, [&] { return ckl::launch_compact_rows(mask, (int)q.T, perm, rank, n, st); });
  if (e != hipSuccess) return e;
  rows->perm = perm;
  rows->rank = rank;
  rows->n = n;
  const void* from = *H;
  *H = b + w.H;
  return timed(CKL_KERNEL_OTHER, st,
               [&] { return ckl::launch_gather_rows(from, (int)q.T, q.d * (int64_t)q.esz, perm, n, b + w.H, st); });
}

}  // namespace

extern "C" {

ckl_status ckl_logprob_workspace_size(int64_t T, int64_t V, int64_t top, size_t* bytes) {
  ckl_status s = check_logprob(T, V, top);
  if (s != CKL_OK) return s;
  if (!bytes) return fail(CKL_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = logprob_layout(T, V, top).total;
  return CKL_OK;
}

ckl_status ckl_token_logprobs(const void* logits, int32_t dtype, int64_t T, int64_t V, const void* tokens,
                              int32_t token_bytes, int64_t top, const uint8_t* mask, float* logprob, float* entropy,
                              float* lse, int32_t* top_idx, float* top_logprob, void* ws, size_t ws_bytes,
                              void* stream) {
  ckl_status s = check_logprob(T, V, top);
  if (s == CKL_OK) s = check_tokens(tokens, token_bytes);
  if (s != CKL_OK) return s;
  if (!dtype_ok(dtype)) return fail(CKL_ERR_INVALID_ARG, "dtype must be CKL_F32 (0) or CKL_BF16 (1)");
  if (T == 0) return CKL_OK;
  if (!logits || !tokens || !logprob || !entropy || !lse || (top > 0 && (!top_idx || !top_logprob)))
    return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(logits) || !aligned16(ws)) return fail(CKL_ERR_INVALID_ARG, "logits and ws must be 16-byte aligned");
  if (!aligned4(logprob) || !aligned4(entropy) || !aligned4(lse) || !aligned4(top_idx) || !aligned4(top_logprob))
    return fail(CKL_ERR_INVALID_ARG, "the outputs must be 4-byte aligned");
  const LogprobWs w = logprob_layout(T, V, top);
  if (w.total && (!ws || ws_bytes < w.total))
    return fail(CKL_ERR_WORKSPACE, "the workspace needs %zu bytes, got %zu", w.total, ws ? ws_bytes : (size_t)0);
  const size_t row = (size_t)T * 4, tops = (size_t)T * top * 4;
  s = check_disjoint({{logprob, row, "logprob"}, {entropy, row, "entropy"}, {lse, row, "lse"},
                      {top_idx, tops, "top_idx"}, {top_logprob, tops, "top_logprob"}, {ws, w.total, "ws"}},
                     {{logits, (size_t)T * V * esize(dtype), "logits"}, {tokens, (size_t)T * token_bytes, "tokens"},
                      {mask, (size_t)T, "mask"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  char* b = (char*)ws;
  const ckl::TokenRows t{tokens, token_bytes == 8, mask, logprob, entropy};
  HIP_TRY(timed(CKL_KERNEL_TOPK, st,
                [&] {
                  return ckl::launch_token_logprobs(logits, dtype == CKL_BF16, T, V, (int)top, t, lse, top_idx,
                                                    top_logprob, (uint64_t*)(b + w.cand), (float2*)(b + w.state),
                                                    (float*)(b + w.state_e), st);
                }),
          "token_logprobs");
  return CKL_OK;
}

ckl_status ckl_token_logprobs_backward(const void* logits, int32_t dtype, int64_t T, int64_t V, const void* tokens,
                                       int32_t token_bytes, const uint8_t* mask, const float* lse,
                                       const float* entropy, const float* dlogprob, const float* dentropy,
                                       void* dlogits, void* stream) {
  ckl_status s = check_logprob(T, V, 0);
  if (s == CKL_OK) s = check_tokens(tokens, token_bytes);
  if (s != CKL_OK) return s;
  if (!dtype_ok(dtype)) return fail(CKL_ERR_INVALID_ARG, "dtype must be CKL_F32 (0) or CKL_BF16 (1)");
  if (T == 0) return CKL_OK;
  if (!logits || !tokens || !lse || !entropy || !dlogits)
    return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(logits) || !aligned16(dlogits))
    return fail(CKL_ERR_INVALID_ARG, "logits and dlogits must be 16-byte aligned");
  if (!aligned4(lse) || !aligned4(entropy) || !aligned4(dlogprob) || !aligned4(dentropy))
    return fail(CKL_ERR_INVALID_ARG, "lse, entropy, dlogprob and dentropy must be 4-byte aligned");
  const size_t row = (size_t)T * 4, all = (size_t)T * V * esize(dtype);
  s = check_disjoint({{dlogits, all, "dlogits"}},
                     {{logits, all, "logits"}, {tokens, (size_t)T * token_bytes, "tokens"}, {mask, (size_t)T, "mask"},
                      {lse, row, "lse"}, {entropy, row, "entropy"}, {dlogprob, row, "dlogprob"},
                      {dentropy, row, "dentropy"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  const ckl::TokenRows t{tokens, token_bytes == 8, mask, nullptr, const_cast<float*>(entropy)};
  HIP_TRY(timed(CKL_KERNEL_TOPK, st,
                [&] {
                  return ckl::launch_token_logprobs_backward(logits, dtype == CKL_BF16, T, V, t, lse, dlogprob,
                                                             dentropy, dlogits, st);
                }),
          "token_logprobs_backward");
  return CKL_OK;
}

ckl_status ckl_head_workspace_size(int64_t T, int64_t d, int64_t V, int64_t chunk, int32_t in_dtype, int32_t dh_dtype,
                                   int32_t dw_dtype, int32_t masked, int which, size_t* bytes) {
  HeadPlan q;
  ckl_status s = head_plan(T, d, V, chunk, in_dtype, dh_dtype, dw_dtype, &q);
  if (s != CKL_OK) return s;
  if (!bytes) return fail(CKL_ERR_INVALID_ARG, "bytes is NULL");
  if (masked != 0 && masked != 1) return fail(CKL_ERR_INVALID_ARG, "masked must be 0 or 1");
  if (which != 0 && which != 1) return fail(CKL_ERR_INVALID_ARG, "which must be 0 (forward) or 1 (backward)");
  *bytes = T == 0 ? 0 : which == 0 ? head_fwd_layout(q, masked).total
                                   : head_bwd_layout(q, masked, dh_dtype, dw_dtype).total;
  return CKL_OK;
}

ckl_status ckl_head_logprobs(const void* H, const void* W, int32_t in_dtype, int64_t T, int64_t d, int64_t V,
                             const void* tokens, int32_t token_bytes, const uint8_t* mask, int64_t chunk,
                             float* logprob, float* entropy, float* lse, void* ws, size_t ws_bytes, void* stream) {
  HeadPlan q;
  ckl_status s = head_plan(T, d, V, chunk, in_dtype, in_dtype, CKL_F32, &q);
  if (s == CKL_OK) s = check_tokens(tokens, token_bytes);
  if (s != CKL_OK) return s;
  if (T == 0) return CKL_OK;
  if (!H || !W || !tokens || !logprob || !entropy || !lse)
    return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned16(H) || !aligned16(W) || !aligned16(ws))
    return fail(CKL_ERR_INVALID_ARG, "H, W and ws must be 16-byte aligned");
  if (!aligned4(logprob) || !aligned4(entropy) || !aligned4(lse))
    return fail(CKL_ERR_INVALID_ARG, "logprob, entropy and lse must be 4-byte aligned");
  const HeadFwdWs w = head_fwd_layout(q, mask != nullptr);
  if (!ws || ws_bytes < w.total)
    return fail(CKL_ERR_WORKSPACE, "the workspace needs %zu bytes, got %zu", w.total, ws ? ws_bytes : (size_t)0);
  const size_t row = (size_t)T * 4;
  s = check_disjoint({{logprob, row, "logprob"}, {entropy, row, "entropy"}, {lse, row, "lse"}, {ws, w.total, "ws"}},
                     {{H, (size_t)T * d * q.esz, "H"}, {W, (size_t)V * d * q.esz, "W"},
                      {tokens, (size_t)T * token_bytes, "tokens"}, {mask, (size_t)T, "mask"}});
  if (s != CKL_OK) return s;
  hipStream_t st = (hipStream_t)stream;
  char* b = (char*)ws;
  float* ztok = (float*)(b + w.ztok);
  float4* part = (float4*)(b + w.part);
  ckl::HeadRows r{tokens, token_bytes == 8, nullptr, nullptr, nullptr};
  const void* Hs = H;
  if (mask) HIP_TRY(head_pack(q, b, w.pk, mask, &Hs, &r, st), "packing kept rows");
  for (int64_t c = 0; c < q.nS; ++c) {
    const int64_t r0 = c * q.Cs;
    const int rows = (int)std::min(q.Cs, T - r0);
    HIP_TRY(timed(CKL_KERNEL_FWD_LSE, st,
                  [&] {
                    return ckl::launch_head_rows(q.tile, (const char*)Hs + r0 * d * q.esz, W, rows, (int)d, (int)V, r,
                                                 (int)r0, ztok, part, (int)q.splits, (int)q.tps, st);
                  }),
            "head_rows");
    HIP_TRY(timed(CKL_KERNEL_FWD_FINALIZE, st,
                  [&] {
                    return ckl::launch_head_finish(part, (int)q.splits, rows, (int)V, r, (int)r0, ztok, logprob,
                                                   entropy, lse, st);
                  }),
            "head_finish");
  }
  return CKL_OK;
}

ckl_status ckl_head_logprobs_backward(const void* H, const void* W, int32_t in_dtype, int64_t T, int64_t d, int64_t V,
                                      const void* tokens, int32_t token_bytes, const uint8_t* mask, int64_t chunk,
                                      const float* lse, const float* entropy, const float* dlogprob,
                                      const float* dentropy, void* dH, int32_t dh_dtype, void* dW, int32_t dw_dtype,
                                      void* ws, size_t ws_bytes, void* stream) {
  HeadPlan q;
  ckl_status s = head_plan(T, d, V, chunk, in_dtype, dh_dtype, dw_dtype, &q);
  if (s == CKL_OK) s = check_tokens(tokens, token_bytes);
  if (s != CKL_OK) return s;
  if (!W || (T > 0 && (!H || !tokens || !lse || !entropy)))
    return fail(CKL_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!dW && (T > 0 && !dH)) return fail(CKL_ERR_INVALID_ARG, "dH and dW are both NULL");
  if (!aligned16(H) || !aligned16(W) || !aligned16(dH) || !aligned16(dW) || !aligned16(ws))
    return fail(CKL_ERR_INVALID_ARG, "H, W, dH, dW and ws must be 16-byte aligned");
  if (!aligned4(lse) || !aligned4(entropy) || !aligned4(dlogprob) || !aligned4(dentropy))
    return fail(CKL_ERR_INVALID_ARG, "lse, entropy, dlogprob and dentropy must be 4-byte aligned");
  const size_t dw_bytes = (size_t)V * d * esize(dw_dtype);
  hipStream_t st = (hipStream_t)stream;
  if (T == 0) {
    if (dW)
      HIP_TRY(timed(CKL_KERNEL_OTHER, st,
                    [&] { return ckl::launch_fill_f32((float*)dW, (int64_t)(dw_bytes / 4), 0.f, st); }),
              "zero dW");
    return CKL_OK;
  }
  const HeadBwdWs w = head_bwd_layout(q, mask != nullptr, dh_dtype, dw_dtype);
  if (!ws || ws_bytes < w.total)
    return fail(CKL_ERR_WORKSPACE, "the workspace needs %zu bytes, got %zu", w.total, ws ? ws_bytes : (size_t)0);
  const size_t row = (size_t)T * 4;
  s = check_disjoint({{dH, (size_t)T * d * esize(dh_dtype), "dH"}, {dW, dw_bytes, "dW"}, {ws, w.total, "ws"}},
                     {{H, (size_t)T * d * q.esz, "H"}, {W, (size_t)V * d * q.esz, "W"},
                      {tokens, (size_t)T * token_bytes, "tokens"}, {mask, (size_t)T, "mask"}, {lse, row, "lse"},
                      {entropy, row, "entropy"}, {dlogprob, row, "dlogprob"}, {dentropy, row, "dentropy"}});
  if (s != CKL_OK) return s;
  char* b = (char*)ws;
  float4* consts = (float4*)(b + w.consts);
  int* tok = (int*)(b + w.tok);
  float* gtok = (float*)(b + w.gtok);  // (bf16)
  int *order = (int*)(b + w.order), *start = (int*)(b + w.start);
  char* Ht = b + w.Ht;
  void* Wt = b + w.Wt;
  void* G = b + w.G;
  void* Gt = q.bf16 ? nullptr : b + w.Gt;
  ckl::HeadRows r{tokens, token_bytes == 8, nullptr, nullptr, nullptr};
  const void* Hs = H;
  if (mask) HIP_TRY(head_pack(q, b, w.pk, mask, &Hs, &r, st), "packing kept rows");
  // fp32 sums in the outputs themselves, or in the workspace where the output is bf16 or its rows are packed
  const bool summed = dh_summed(q, mask != nullptr, dh_dtype);
  float* parts = (float*)(b + w.parts);
  float* sums = !summed || (dh_dtype == CKL_F32 && !mask) ? (float*)dH : (float*)(b + w.sums);
  const bool in_sums = !summed || (q.carried && q.Sh == 1);  // the contraction adds to them itself
  const int64_t dh_stride = q.dh_rows * d;
  // bf16 inputs and dW: the last block of rows writes the rounded sums
  const bool dw16 = q.bf16 && dw_dtype == CKL_BF16;
  float* dWacc = dw_dtype != CKL_BF16 ? (float*)dW : w.dW ? (float*)(b + w.dW) : nullptr;
  HIP_TRY(timed(CKL_KERNEL_OTHER, st,
                [&] {
                  return ckl::launch_head_consts(r, (int)T, (int)q.Tp, (int)V, lse, entropy, dlogprob, dentropy, consts,
                                                 tok, st);
                }),
          "head_consts");
  if (dW && q.bf16)
    HIP_TRY(timed(CKL_KERNEL_OTHER, st,
                  [&] {
                    return ckl::launch_head_buckets(tok, (int)T, (int)q.Tc, r.n, (int)(q.Vp / 256), order, start, st);
                  }),
            "head_buckets");
  if (dW)
    HIP_TRY(timed(CKL_KERNEL_TRANSPOSE, st,
                  [&] {
                    return ckl::launch_transpose_pad(q.bf16, Hs, (int)T, (int)d, (int)q.Tp, Ht, q.Tp + kLdPad, st);
                  }),
            "transpose H");
  const int64_t ldWt = q.Vc + kLdPad;
  for (int64_t vb = 0; vb < q.nV; ++vb) {
    const int64_t vb0 = vb * q.Vc, vrows = std::min(q.Vc, q.Vp - vb0);
    if (dH && !q.turned)
      HIP_TRY(timed(CKL_KERNEL_TRANSPOSE, st,
                    [&] {
                      return ckl::launch_transpose_pad(q.bf16, (const char*)W + vb0 * d * q.esz,
                                                       (int)std::min(q.Vc, V - vb0), (int)d, (int)vrows, Wt, ldWt, st);
                    }),
              "transpose W block");
    for (int64_t tb = 0; tb < q.nT; ++tb) {
      const int64_t tb0 = tb * q.Tc, trows = std::min(q.Tc, q.Tp - tb0);
      int64_t splits, tps;
      pick_splits(trows / q.BN, vrows / q.BM, kGradSlots, &splits, &tps);
      HIP_TRY(timed(CKL_KERNEL_BWD_GRAD, st,
                    [&] {
                      return ckl::launch_head_grad(q.bf16, Hs, W, (int)T, (int)d, (int)V, consts, tok, gtok, (int)tb0,
                                                   (int)trows, (int)vb0, (int)vrows, (int)tps, G,
                                                   vrows + kLdPad, Gt, trows + kLdPad, r.n, st);
                    }),
              "head_grad");
      // dH[tb0 ..) (+)= G W[vb0 ..) by parts of the vocabulary block (the longer sums: scheduled first),
      // dW[vb0 ..) (+)= G^T H[tb0 ..) (bf16: G read k-major)
      const int rows_here = (int)std::min(trows, T - tb0);
      ckl::GemmArgs gdh{G, vrows + kLdPad, Wt, ldWt, !dH ? nullptr : in_sums ? sums + tb0 * d : parts, d,
                        dH ? rows_here : 0, (int)d, (int)std::min(q.Vs, vrows),
                        vb > 0 && (in_sums || !q.carried)};
      const int gdh_parts = gdh.batches = (int)ceil_div(vrows, q.Vs);
      gdh.kdim_last = (int)(vrows - (gdh.batches - 1) * q.Vs);
      gdh.xb = gdh.yb = q.Vs;
      gdh.ob = dh_stride;
      if (q.turned) {
        const int64_t cols = std::min(vrows, V - vb0);  // (W's rows)
        gdh.batches = (int)ceil_div(cols, q.Vs);
        gdh.kdim = (int)std::min(q.Vs, cols);
        gdh.kdim_last = (int)(cols - (gdh.batches - 1) * q.Vs);
        gdh.X = (const char*)W + vb0 * d * 2;
        gdh.ldx = d;
        gdh.xt = 1;
        gdh.xb = q.Vs * d;
        gdh.Y = G;
        gdh.ldy = vrows + kLdPad;
        gdh.ldo = q.dh_rows;
        gdh.M = dH ? (int)d : 0;
        gdh.N = (int)T;
      }
      ckl::GemmArgs gdw{q.bf16 ? G : Gt, q.bf16 ? vrows + kLdPad : trows + kLdPad, Ht + tb0 * q.esz, q.Tp + kLdPad,
                        dWacc ? dWacc + vb0 * d : nullptr, d, dW ? (int)std::min(vrows, V - vb0) : 0, (int)d,
                        (int)std::min(trows, round_up(T - tb0, 64)), tb > 0};
      gdw.xt = q.bf16;
      // (the contraction, us, fp32 by 64 x 64 against 128 x 128: 226 rows of 520, 5003 words 41 and 53; 1000 of 512,
      // 2000 words 80 and 164; 2048 of 1024, 32000 words 2437 and 2427)
      if (dW && dw16 && tb == q.nT - 1) gdw.out16 = (char*)dW + vb0 * d * 2;
      if (dW && q.bf16) {
        gdw.rows.order = order;
        gdw.rows.start = start + tb * (q.Vp / 64 + 1);
        gdw.rows.col = tok;
        gdw.rows.scale = gtok;
        gdw.rows.rows = Hs;
        gdw.rows.col0 = (int)vb0;
      }
      if (r.n) {
        gdw.lim = r.n;
        gdw.lim_base = (int)tb0;
        gdw.lim_kind = 2;
        gdw.lim_round = 64;  // (G's rows are formed in blocks of as many or more)
        if (!q.turned) {
          gdh.lim = r.n;
          gdh.lim_base = (int)tb0;
          gdh.lim_kind = 1;
        }
      }
      if (q.narrow && dH) {
        HIP_TRY(timed(CKL_KERNEL_GEMM_DHDW, st, [&] { return ckl::launch_gemm_pair(1, gdh, ckl::GemmArgs{}, st, 1); }),
                "gemm dH");
        gdh.M = 0;
      }
      if (!q.narrow || dW)
        HIP_TRY(timed(CKL_KERNEL_GEMM_DHDW, st,
                      [&] { return ckl::launch_gemm_pair(q.bf16, gdh, gdw, st, !q.bf16); }),
                "gemm dH + dW");
      // the block's rows of dH: finished behind the last block of words, until then kept where they are carried
      const bool last = vb == q.nV - 1;
      if (dH && summed && (last || (q.carried && !in_sums)))
        HIP_TRY(timed(CKL_KERNEL_OTHER, st,
                      [&] {
                        if (q.turned)
                          return ckl::launch_head_dh_t(parts, dh_stride, q.dh_rows, (int)q.Sh, (int)T, (int)d, tok,
                                                       gtok, W, r, dH, dh_dtype == CKL_BF16, st);
                        const int n = in_sums ? 0 : q.carried ? gdh_parts : (int)q.Sh;
                        const float* before = in_sums || (q.carried && vb > 0) ? sums : nullptr;
                        if (last)
                          return ckl::launch_head_dh(parts, dh_stride, n, before, (int)tb0, rows_here, (int)d, tok,
                                                     q.bf16 ? gtok : nullptr, W, r, dH, dh_dtype == CKL_BF16, st);
                        return ckl::launch_head_dh(parts, dh_stride, n, before, (int)tb0, rows_here, (int)d, nullptr,
                                                   nullptr, nullptr, {nullptr, 0, nullptr, nullptr, r.n}, sums, 0, st);
                      }),
                "sum dH");
    }
  }
  if (dW && dw_dtype == CKL_BF16 && !dw16)
    HIP_TRY(timed(CKL_KERNEL_OTHER, st, [&] { return ckl::launch_cast_f32_bf16(dWacc, dW, V * d, st); }), "cast dW");
  return CKL_OK;
}

}  // extern "C"
