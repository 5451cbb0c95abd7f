// Argument checks that the operators' entry points share (host only).
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "kda.h"
#include "kda_internal.h"

namespace kda {
namespace {

kda_status bad(kda_status st, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return report_error(st, msg);
}

kda_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return KDA_OK;
  return bad(e == cudaErrorMemoryAllocation ? KDA_ERR_OUT_OF_MEMORY : KDA_ERR_CUDA, "%s: %s", what,
             cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int64_t size_of(kda_dtype t) { return t == KDA_BF16 ? 2 : t == KDA_E4M3 ? 1 : 4; }

// Rows of `width` bytes, `pitch` bytes apart.  A null pointer has no rows.
struct Rows {
  const char* name;
  const void* p;
  int64_t rows, pitch, width;
};

Rows rows_of(const char* name, const void* p, int64_t rows, int64_t ld, int64_t cols, int64_t esize) {
  return Rows{name, p, p ? rows : 0, ld * esize, cols * esize};
}

bool same_rows(const Rows& a, const Rows& b) {
  return a.p == b.p && a.width == b.width && (a.pitch == b.pitch || a.rows <= 1);
}

// Whether two sets of rows share a byte.  Rows of one pitch may interleave
// (column slices of one buffer); rows of different pitches count as
// overlapping where their spans do.
bool overlap(const Rows& a, const Rows& b) {
  if (a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t a1 = a0 + static_cast<uintptr_t>((a.rows - 1) * a.pitch + a.width);
  const uintptr_t b1 = b0 + static_cast<uintptr_t>((b.rows - 1) * b.pitch + b.width);
  if (a1 <= b0 || b1 <= a0) return false;
  if (a.pitch == b.pitch && a.pitch > 0) {
    const int64_t pitch = a.pitch;
    int64_t d = static_cast<int64_t>(b0 - a0) % pitch;  // b's first column in a's rows
    if (d < 0) d += pitch;
    if (d >= a.width && pitch - d >= b.width) return false;
  }
  return true;
}

// An output against inputs and the other outputs; `may_be`: the one it may equal exactly.
kda_status check_output(const Rows& out, const Rows* others, int n, const Rows* may_be,
                        const Rows* may_be2 = nullptr) {
  for (int i = 0; i < n; ++i) {
    if (!overlap(out, others[i])) continue;
    const bool allowed = (&others[i] == may_be || &others[i] == may_be2) && same_rows(out, others[i]);
    if (!allowed) return bad(KDA_ERR_INVALID_ARGUMENT, "%s overlaps %s", out.name, others[i].name);
  }
  return KDA_OK;
}

bool float_type(kda_dtype t) { return t == KDA_BF16 || t == KDA_F32; }

// Pointer alignment to its element, and a leading dimension that holds a row.
kda_status check_rows(const char* name, const void* p, int64_t ld, int64_t cols, int64_t esize) {
  if (!aligned(p, static_cast<uintptr_t>(esize)))
    return bad(KDA_ERR_INVALID_ARGUMENT, "%s is not aligned to its element", name);
  if (p && ld < cols)
    return bad(KDA_ERR_INVALID_ARGUMENT, "%s: leading dimension %lld is less than the %lld columns",
               name, (long long)ld, (long long)cols);
  if (p && ld > (1LL << 40))
    return bad(KDA_ERR_INVALID_ARGUMENT, "%s: leading dimension %lld", name, (long long)ld);
  return KDA_OK;
}

#define KDA_TRY(call)                      \
  do {                                     \
    const kda_status st_ = (call);         \
    if (st_ != KDA_OK) return st_;         \
  } while (0)

}  // namespace
}  // namespace kda
