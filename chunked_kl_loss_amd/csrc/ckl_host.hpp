// What the entry points share on the host: error reporting, timing records,
// size helpers and the checks of buffers (internal; not part of the ABI).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include "../../include/ckl.h"

namespace ckl {
namespace host {

inline thread_local std::string g_last_error;

inline ckl_status fail(ckl_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline ckl_status fail(ckl_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

inline ckl_status hip_fail(hipError_t e, const char* what) {
  return fail(CKL_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

#define HIP_TRY(expr, what)                         \
  do {                                              \
    hipError_t e__ = (expr);                        \
    if (e__ != hipSuccess) return hip_fail(e__, what); \
  } while (0)

constexpr int64_t kMaxK = 4096;
// Rows of H and W: the contraction loads address a 256-row tile of H^T, W^T,
// G or G^T with 32-bit byte offsets (256 * (rows + padding) * 2 < 2^31).
constexpr int64_t kMaxRows = 4000000;

// ------------------------------------------------------------------ timing --
struct TimingState {
  std::mutex mu;
  bool on = false;
  struct Rec { int cls; hipEvent_t a, b; };
  std::vector<Rec> pending;
  std::vector<std::pair<hipEvent_t, hipEvent_t>> pool;
  double total_ms[CKL_KERNEL_CLASSES] = {};
  int64_t launches[CKL_KERNEL_CLASSES] = {};
};
inline TimingState g_timing;

// Launch `fn` (returning hipError_t), bracketed by timing events when enabled.
// Set while ckl_forward_noalloc runs: its launches record no timing events
// (creating events would allocate).
inline thread_local bool g_no_events = false;

template <class Fn>
hipError_t timed(int cls, hipStream_t st, Fn&& fn) {
  if (!g_timing.on || g_no_events) return fn();
  std::pair<hipEvent_t, hipEvent_t> ev{};
  {
    std::lock_guard<std::mutex> lk(g_timing.mu);
    if (!g_timing.pool.empty()) { ev = g_timing.pool.back(); g_timing.pool.pop_back(); }
  }
  hipError_t e;
  if (!ev.first) {
    if ((e = hipEventCreate(&ev.first)) != hipSuccess) return e;
    if ((e = hipEventCreate(&ev.second)) != hipSuccess) return e;
  }
  if ((e = hipEventRecord(ev.first, st)) != hipSuccess) return e;
  if ((e = fn()) != hipSuccess) return e;
  if ((e = hipEventRecord(ev.second, st)) != hipSuccess) return e;
  std::lock_guard<std::mutex> lk(g_timing.mu);
  g_timing.pending.push_back({cls, ev.first, ev.second});
  return hipSuccess;
}

inline hipError_t timing_drain() {
  std::lock_guard<std::mutex> lk(g_timing.mu);
  for (auto& r : g_timing.pending) {
    hipError_t e = hipEventSynchronize(r.b);
    if (e != hipSuccess) return e;
    float ms = 0.f;
    e = hipEventElapsedTime(&ms, r.a, r.b);
    if (e != hipSuccess) return e;
    g_timing.total_ms[r.cls] += ms;
    g_timing.launches[r.cls] += 1;
    g_timing.pool.push_back({r.a, r.b});
  }
  g_timing.pending.clear();
  return hipSuccess;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

inline bool aligned16(const void* ptr) { return ((uintptr_t)ptr & 15u) == 0; }

// A buffer of an entry point: where it starts, its bytes, its name.
struct Span {
  const void* p;
  size_t n;
  const char* name;
};
inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + b.n && b0 < a0 + a.n;
}
// Every buffer the call writes (outputs, the used part of the workspace) must
// be disjoint from every other buffer of the call: an output that aliases an
// input or the workspace would be read after the library overwrote it.
inline ckl_status check_disjoint(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  for (auto w = written.begin(); w != written.end(); ++w) {
    for (auto o = w + 1; o != written.end(); ++o)
      if (overlap(*w, *o)) return fail(CKL_ERR_INVALID_ARG, "%s and %s overlap", w->name, o->name);
    for (const Span& r : read)
      if (overlap(*w, r)) return fail(CKL_ERR_INVALID_ARG, "%s overlaps %s", w->name, r.name);
  }
  return CKL_OK;
}

}  // namespace host
}  // namespace ckl
