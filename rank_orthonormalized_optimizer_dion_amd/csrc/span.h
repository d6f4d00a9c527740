// The memory of a row-major matrix with a row pitch (host side of the training
// operators' argument checks).
#pragma once
#include <cstddef>
#include <cstdint>

namespace dion {

struct Span {
  const void* p;
  int64_t rows, cols, ld;   // ld >= cols
  int64_t esize;
  bool misplaced() const { return reinterpret_cast<uintptr_t>(p) % esize != 0; }
  size_t bytes() const { return rows > 0 ? static_cast<size_t>(((rows - 1) * ld + cols) * esize) : 0; }
};

// Whether two matrices share an element.  Column blocks of one buffer lie
// within each other's address range and share none: with one pitch for both,
// b's rows start at the same offset d in every row of a, and the blocks are
// apart where b starts past a's columns and ends before a's next row.  (A
// matrix of one row has every pitch.)  Interleaved matrices of different
// pitches count as sharing.
inline bool spans_overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.rows < 1 || b.rows < 1) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  if (x >= y + b.bytes() || y >= x + a.bytes()) return false;
  const uint64_t wa = a.cols * a.esize, wb = b.cols * b.esize;
  const uint64_t pa = a.ld * a.esize, pb = b.ld * b.esize;
  if (pa != pb && a.rows > 1 && b.rows > 1) return true;
  const uint64_t pitch = a.rows > 1 ? pa : pb;
  const uint64_t d = y >= x ? (y - x) % pitch : (pitch - (x - y) % pitch) % pitch;
  return d < wa || d + wb > pitch;
}

}  // namespace dion
