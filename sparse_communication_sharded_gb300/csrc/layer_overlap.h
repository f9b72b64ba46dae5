// layer_overlap.h -- whether two matrices share memory.  Host code without CUDA's
// headers, so that a test can compare it with a count of bytes.
#pragma once

#include <cstdint>

namespace scapek {
namespace layer {

// `rows` pieces of `width` bytes, `pitch` (at least width) bytes apart.
struct Span {
  uintptr_t p = 0;
  int64_t pitch = 0, width = 0, rows = 0;

  Span() = default;
  Span(const void* at, int64_t pitch_, int64_t width_, int64_t rows_)
      : p(reinterpret_cast<uintptr_t>(at)), pitch(pitch_), width(width_), rows(at ? rows_ : 0) {
    if (rows <= 0 || width <= 0) rows = width = 0;
    if (pitch == width || rows == 1) width *= rows, pitch = width, rows = rows ? 1 : 0;
  }
  bool same(const Span& o) const { return p == o.p && pitch == o.pitch && width == o.width && rows == o.rows; }
  uintptr_t end() const { return rows ? p + (rows - 1) * pitch + width : p; }
};

// Pieces of b that share bytes with [from, to): those j with j pitch < to and
// j pitch + width > from, counted from b's start.
inline bool meets(int64_t from, int64_t to, const Span& b) {
  int64_t first = from < b.width ? 0 : (from - b.width) / b.pitch + 1;
  int64_t last = to <= 0 ? -1 : (to - 1) / b.pitch;
  if (last > b.rows - 1) last = b.rows - 1;
  return first <= last;
}

// Slices of one wider buffer lie between each other without sharing a byte, so
// where the ranges of memory meet the pieces are compared: two of them stand for
// all where the pitches are equal, else every piece of the matrix that has fewer.
inline bool overlap(const Span& x, const Span& y) {
  if (!x.rows || !y.rows || x.end() <= y.p || y.end() <= x.p) return false;
  const Span &a = x.rows <= y.rows ? x : y, &b = x.rows <= y.rows ? y : x;
  const int64_t apart = (int64_t)(a.p - b.p);
  if (a.rows > 1 && a.pitch == b.pitch) {
    // a lies q pitches and r bytes after b: piece i of a starts r bytes into pitch
    // i + q of b's, and may reach into the one after
    int64_t q = apart / a.pitch, r = apart % a.pitch;
    if (r < 0) r += a.pitch, --q;
    const bool same_pitch = r < b.width && q < b.rows && q + a.rows > 0;
    const bool next_pitch = r + a.width > a.pitch && q + 1 < b.rows && q + 1 + a.rows > 0;
    return same_pitch || next_pitch;
  }
  for (int64_t i = 0; i < a.rows; ++i)
    if (meets(apart + i * a.pitch, apart + i * a.pitch + a.width, b)) return true;
  return false;
}

}  // namespace layer
}  // namespace scapek
