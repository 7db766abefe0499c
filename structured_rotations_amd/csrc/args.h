// What the C entry points of the operators share: errors, and the checks of
// their arguments, which run on the host before any HIP call.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "harp.h"
#include "kernels.h"
#include "plan.h"

namespace harp {

inline harp_status fail(harp_status st, const char* fmt, ...) {
  char buf[240];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return st;
}

inline harp_status launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return HARP_OK;
  return fail(HARP_ERR_LAUNCH, "%s: %s", what, hipGetErrorString(e));
}

inline bool io_ok(harp_dtype t) { return t == HARP_F32 || t == HARP_BF16; }
inline int size_of(harp_dtype t) { return t == HARP_F32 ? 4 : t == HARP_BF16 ? 2 : 1; }
inline DT dt(harp_dtype t) { return static_cast<DT>(t); }

// A matrix argument: its name, base, leading dimension (elements), extent and
// element size.
struct Mat {
  const char* name;
  const void* p;
  int64_t ld, rows, cols;
  int eb;
  uintptr_t at() const { return reinterpret_cast<uintptr_t>(p); }
  uint64_t bytes() const { return (uint64_t)((rows - 1) * ld + cols) * (uint64_t)eb; }
};

// Base, alignment, leading dimension and extent of a matrix with rows >= 1.
inline harp_status check(const Mat& m) {
  if (m.p == nullptr) return fail(HARP_ERR_INVALID_ARG, "%s is NULL", m.name);
  if (m.at() % m.eb) return fail(HARP_ERR_INVALID_ARG, "%s is not aligned to its element size", m.name);
  if (m.ld < m.cols)
    return fail(HARP_ERR_INVALID_ARG, "%s: leading dimension %lld is smaller than the row length %lld", m.name,
                (long long)m.ld, (long long)m.cols);
  if (m.rows > 1 && m.ld > (INT64_MAX / m.eb - m.cols) / (m.rows - 1))
    return fail(HARP_ERR_INVALID_ARG, "%s: rows x leading dimension exceeds the address space", m.name);
  if (m.at() > UINT64_MAX - m.bytes())
    return fail(HARP_ERR_INVALID_ARG, "%s: rows x leading dimension exceeds the address space", m.name);
  return HARP_OK;
}

// An output against another argument: no common byte, unless `same` allows the
// same buffer with the same leading dimension.  Rows may lie side by side in one
// buffer: matrices whose rows are the same distance apart (a single row goes with
// any distance) have no common byte if a row of one fits between the other's.
// Other matrices have to be apart as a whole.
inline harp_status check_apart(const Mat& out, const Mat& in, bool same) {
  if (out.p == nullptr || in.p == nullptr) return HARP_OK;
  if (same && out.p == in.p && out.eb == in.eb && out.ld == in.ld) return HARP_OK;
  if (out.at() >= in.at() + in.bytes() || in.at() >= out.at() + out.bytes()) return HARP_OK;
  const uint64_t lo = (uint64_t)out.ld * out.eb, li = (uint64_t)in.ld * in.eb;
  if ((out.rows > 1 || in.rows > 1) && (out.rows == 1 || in.rows == 1 || lo == li)) {
    const uint64_t step = out.rows > 1 ? lo : li;
    // where a row of `in` begins after the beginning of one of `out`
    const uint64_t d = (in.at() >= out.at() ? in.at() - out.at() : step - (out.at() - in.at()) % step) % step;
    if (d >= (uint64_t)out.cols * out.eb && step - d >= (uint64_t)in.cols * in.eb) return HARP_OK;
  }
  return fail(HARP_ERR_INVALID_ARG, "%s overlaps %s", out.name, in.name);
}

// Sizes fit an int with room for a tile beyond the last row or column.
constexpr int64_t kMaxSize = 1LL << 30;

inline harp_status check_size(const char* name, int64_t v, int64_t lo, int64_t hi) {
  if (v < lo || v > hi)
    return fail(HARP_ERR_INVALID_ARG, "%s = %lld is outside %lld..%lld", name, (long long)v, (long long)lo,
                (long long)hi);
  return HARP_OK;
}

inline harp_status check_workspace(int64_t need, const void* ws, size_t bytes, int align) {
  if (need <= 0) return HARP_OK;
  if (ws == nullptr || bytes < (uint64_t)need)
    return fail(HARP_ERR_INVALID_ARG, "workspace of %lld bytes is needed, got %lld", (long long)need,
                (long long)(ws ? bytes : 0));
  if (reinterpret_cast<uintptr_t>(ws) % align)
    return fail(HARP_ERR_INVALID_ARG, "workspace is not %d-byte aligned", align);
  return HARP_OK;
}

#define TRY(expr)                          \
  do {                                     \
    const harp_status st_ = (expr);        \
    if (st_ != HARP_OK) return st_;        \
  } while (0)

}  // namespace harp
