// Whether two matrices in memory share a byte: the binding refuses outputs over its inputs with it.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moelora {

// Bytes of a matrix: `rows` runs of `width`, `step` apart.
struct Bytes {
  const char* p;
  int64_t rows, width, step;
  const char* end() const { return p + (rows - 1) * step + width; }
};

inline Bytes dense_bytes(const void* p, int64_t n) { return {(const char*)p, p && n > 0 ? 1 : 0, n, n}; }

inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); }

// Whether two matrices share a byte.
inline bool overlap(const Bytes& a, const Bytes& b) {
  if (!a.rows || !b.rows || a.p >= b.end() || b.p >= a.end()) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  if (a.rows > b.rows) return overlap(b, a);
  if (a.rows > 1 && a.step == b.step) {
    // row j of b begins (j - i) step + d after row i of a: the first j - i with b's row past the start of a's
    const int64_t d = b.p - a.p, m = std::max(floor_div(-b.width - d, a.step) + 1, 1 - a.rows);
    return m < b.rows && m * a.step + d < a.width;
  }
  for (int64_t i = 0; i < a.rows; ++i) {  // the first row of b that ends past the start of a's
    const char* q = a.p + i * a.step;
    const int64_t j = std::max(floor_div(q - b.width - b.p, b.step) + 1, (int64_t)0);
    if (j < b.rows && b.p + j * b.step < q + a.width) return true;
  }
  return false;
}

}  // namespace moelora
