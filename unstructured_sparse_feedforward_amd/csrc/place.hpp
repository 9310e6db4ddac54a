// Whether a call's matrices share memory (host).
#pragma once

#include <stdint.h>

namespace sffn {

// rows of `width` bytes, one every `pitch` >= width, of elements of elem bytes
// (no rows: no memory)
struct Place {
  const void* p;
  int64_t rows, pitch, width;
  int elem;
};

// kSame: every row and element in the place of the other's, which a kernel whose
// lanes write what they have read may do in place; kMixed: some bytes otherwise,
// so that one row's result would lie over another's operand.
enum Meeting { kApart, kSame, kMixed };

// of two matrices of as many rows, or none
inline Meeting meeting(const Place& a, const Place& b) {
  const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
  const int64_t last = a.rows - 1;
  if (a.rows == 0 || b.rows == 0 || pa >= pb + (uint64_t)(last * b.pitch + b.width) ||
      pb >= pa + (uint64_t)(last * a.pitch + a.width))
    return kApart;
  if (pa == pb && a.elem == b.elem && a.width == b.width && (last == 0 || a.pitch == b.pitch))
    return kSame;
  if (last == 0) return kMixed;
  // Row i of the one with the longer pitch from byte t of the other's first row
  // on, and the first row of the other that does not end before it.
  const bool swap = b.pitch > a.pitch;
  const Place &l = swap ? b : a, &s = swap ? a : b;
  const int64_t d = (int64_t)((uintptr_t)l.p - (uintptr_t)s.p);
  const auto meets = [&](int64_t i) {
    const int64_t t = d + i * l.pitch, over = t - s.width;
    const int64_t j = over < 0 ? 0 : over / s.pitch + 1;
    return j <= last && j * s.pitch < t + l.width;
  };
  if (l.pitch == s.pitch) {
    // all rows meet as the first one that has rows of the other beside it, and
    // the last
    const int64_t i = d < 0 ? -d / l.pitch : 0;
    return meets(i) || (i < last && meets(i + 1)) ? kMixed : kApart;
  }
  for (int64_t i = 0; i <= last; ++i)
    if (meets(i)) return kMixed;
  return kApart;
}

}  // namespace sffn
