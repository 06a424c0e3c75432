// checks.h -- what the exported calls of include/mnb_ops.h and include/mnb_decode.h check their arguments with.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mnb_ops.h"
#include "ops.h"

namespace mnb {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool bad_dtype(int d, bool f32) { return d < MNB_F16 || d > (f32 ? MNB_F32 : MNB_BF16); }
inline int elem_size(int dtype) { return dtype == MNB_F32 ? 4 : 2; }
inline bool off16(const void *p) { return ((uintptr_t)p & 15u) != 0; }
inline bool off16(int64_t bytes) { return (bytes & 15) != 0; }

// bytes of an MX row and of its scales as they are read
inline int64_t mx_row(int fmt, int K) { return fmt == MNB_MX_FP4 ? K / 2 : K; }
inline int64_t scale_row(int K) { return cdiv(K, kMxScaleK) * 16; }

// rows of `row` bytes, `ld` apart
struct Span {
  const void *p;
  int64_t rows, ld, row;
};
inline uintptr_t end_of(const Span &s) {
  uintptr_t d, e;
  if (__builtin_mul_overflow((uintptr_t)(s.rows - 1), (uintptr_t)s.ld, &d) || __builtin_add_overflow(d, (uintptr_t)s.row, &d) ||
      __builtin_add_overflow((uintptr_t)s.p, d, &e))
    return UINTPTR_MAX;
  return e;
}
// Do they share a byte?  Rows between each other's rows (columns of one buffer) do not; where the row
// distances differ, whole ranges count.
inline bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.row <= 0 || b.row <= 0) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  if (a0 >= end_of(b) || b0 >= end_of(a)) return false;
  const int64_t ld = a.rows > 1 ? a.ld : b.ld;
  if (ld <= 0 || (a.rows > 1 && b.rows > 1 && a.ld != b.ld) || (a.rows == 1 && b.rows == 1)) return true;
  // b's columns, counted from a's
  const int64_t d = b0 >= a0 ? (int64_t)((b0 - a0) % (uintptr_t)ld) : (int64_t)((ld - (int64_t)((a0 - b0) % (uintptr_t)ld)) % ld);
  return d < a.row || d + b.row > ld;
}
inline bool same(const Span &a, const Span &b) { return a.p == b.p && (a.ld == b.ld || a.rows == 1) && a.row == b.row; }

// a row distance in elements: any real one is far below 2^40
inline bool bad_ld(int64_t ld, int64_t least) { return ld < least || ld > (1ll << 40); }

inline hipStream_t as_stream(void *s) { return static_cast<hipStream_t>(s); }
inline int status(hipError_t e) { return e == hipSuccess ? MNB_OK : MNB_ERR_HIP; }

}  // namespace mnb
