// rows.h -- rows of memory that lie a stride apart, and whether two sets of them
// share a byte (host only).
#pragma once

#include <stdint.h>

namespace pkv {

struct Rows {
  uintptr_t at;                // the first row
  int64_t n, stride, bytes;    // rows, bytes between their starts, bytes of each (<= stride, or n is 1)

  uintptr_t end() const { return at + (uintptr_t)((n - 1) * stride + bytes); }
};

inline bool rows_overlap(Rows a, Rows b) {
  if (a.n <= 0 || b.n <= 0 || a.at >= b.end() || b.at >= a.end()) return false;
  for (Rows* r : {&a, &b})
    if (r->stride == r->bytes) {                      // without gaps: one row
      r->bytes *= r->n;
      r->n = 1;
    }
  if (a.n > 1 && b.n > 1 && a.stride == b.stride) {
    // parts of the same rows: b's row j starts `in` bytes into a's row j + k
    const int64_t d = (int64_t)(b.at - a.at), k = d >= 0 ? d / a.stride : -((-d + a.stride - 1) / a.stride);
    const int64_t in = d - k * a.stride;
    auto meet = [&](int64_t shift) { return shift > -b.n && shift < a.n; };      // some j has both
    return (in < a.bytes && meet(k)) || (in + b.bytes > a.stride && meet(k + 1));
  }
  if (a.n > b.n) {
    const Rows t = a;
    a = b;
    b = t;
  }
  for (int64_t i = 0; i < a.n; ++i) {                 // a's rows one by one against b's
    const uintptr_t lo = a.at + (uintptr_t)(i * a.stride), hi = lo + (uintptr_t)a.bytes;
    // b's first row that ends behind lo
    int64_t j = 0;
    if (lo >= b.at + (uintptr_t)b.bytes) {
      if (b.n == 1) continue;
      j = (int64_t)(lo - b.at - (uintptr_t)b.bytes) / b.stride + 1;
    }
    if (j < b.n && b.at + (uintptr_t)(j * b.stride) < hi) return true;
  }
  return false;
}

}  // namespace pkv
