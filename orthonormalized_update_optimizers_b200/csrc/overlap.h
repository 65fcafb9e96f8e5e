// Whether two strided matrices share bytes.  Plain C++: no CUDA needed.
#pragma once

#include <stdint.h>

namespace ouo {

struct Span {
  uintptr_t p;
  int64_t rows, width, pitch;  // bytes of a row, bytes from row to row
  uintptr_t end() const { return p + (uintptr_t)((rows - 1) * pitch + width); }
  bool empty() const { return rows <= 0 || width <= 0; }
  bool solid() const { return rows == 1 || pitch == width; }
};

// Bytes [lo, hi), which reach into s's range, against s's rows.
inline bool hits_row(const Span& s, uintptr_t lo, uintptr_t hi) {
  if (lo <= s.p) return true;
  const int64_t off = (int64_t)(lo - s.p), r = off / s.pitch;
  if (off - r * s.pitch < s.width) return true;
  return r + 1 < s.rows && hi > s.p + (uintptr_t)((r + 1) * s.pitch);
}

// Exact where one of them is without gaps or both have the same pitch (columns
// of one wider matrix, say).  Two matrices with gaps and different pitches
// inside one range are taken to be apart: nothing short of a search tells.
inline bool overlap(const Span& a, const Span& b) {
  if (a.empty() || b.empty() || a.p >= b.end() || b.p >= a.end()) return false;
  if (a.solid()) return b.solid() || hits_row(b, a.p, a.end());
  if (b.solid()) return hits_row(a, b.p, b.end());
  if (a.pitch != b.pitch) return false;
  const Span &first = a.p <= b.p ? a : b, &second = a.p <= b.p ? b : a;
  const int64_t d = (int64_t)(second.p - first.p) % first.pitch;
  return d < first.width || d + second.width > first.pitch;
}

}  // namespace ouo
