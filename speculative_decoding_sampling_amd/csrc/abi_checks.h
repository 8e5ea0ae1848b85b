// Checks that the C ABIs of the operators share.
#pragma once

#include <cstddef>
#include <cstdint>

#include "specverify.h"

namespace specv {

inline bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

inline bool known(specv_dtype_t t) { return t == SPECV_F32 || t == SPECV_BF16; }
inline size_t size_of(specv_dtype_t t) { return t == SPECV_BF16 ? 2 : 4; }

// An array by its bytes (null or empty: none).
struct Span {
  const void* p;
  size_t n;
};
inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.n && y < x + a.n;
}

// The rows of a probability tensor: nk for each of B requests, n bytes each,
// at strides of sb and sk bytes (null: none).
struct Rows {
  const void* p;
  size_t sb, sk;
  int B, nk;
  size_t n;
};
// Whether an array lies over one of the rows (between them it may lie).  Few
// calls get past the first comparison.
inline bool overlaps_rows(const Span& a, const Rows& r) {
  if (!r.p || r.nk == 0) return false;
  const size_t last = (size_t)(r.B - 1) * r.sb + (size_t)(r.nk - 1) * r.sk;
  if (!overlap(a, Span{r.p, last + r.n})) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(r.p);
  for (int b = 0; b < r.B; ++b) {
    const uintptr_t first = y + (size_t)b * r.sb;
    size_t k = 0;                                  // the request's first row that ends past x
    if (x >= first + r.n) {
      if (r.sk == 0) continue;
      k = (x - first - r.n) / r.sk + 1;
    }
    if (k < (size_t)r.nk && first + k * r.sk < x + a.n) return true;
  }
  return false;
}

// Whether an output lies over an input or over another output.
template <size_t NO, size_t NI>
bool clash(const Span (&out)[NO], const Span (&in)[NI]) {
  for (size_t i = 0; i < NO; ++i) {
    for (size_t j = 0; j < NI; ++j)
      if (overlap(out[i], in[j])) return true;
    for (size_t j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

inline specv_status_t status(hipError_t e) { return e == hipSuccess ? SPECV_OK : SPECV_EHIP; }

}  // namespace specv
