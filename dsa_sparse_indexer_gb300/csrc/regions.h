// Host-side check that what a call writes lies apart from what it reads.
#pragma once

#include <cstdint>
#include <initializer_list>

namespace dsa {

// Bytes [first, end) of an argument; none where there is no pointer.
struct Region {
  uintptr_t first = 0, end = 0;
};
inline Region bytes_of(const void* p, int64_t n) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  return p && n > 0 ? Region{at, at + (uintptr_t)n} : Region{};
}
// T x H rows of `width` values of `size` bytes, strides in values: the first byte to the
// last, with whatever lies between the rows.
inline Region rows_of(const void* p, int64_t T, int64_t token, int64_t H, int64_t head, int64_t width, int size) {
  if (T < 1 || H < 1) return {};
  const __int128 n = ((__int128)(T - 1) * token + (__int128)(H - 1) * head + width) * size;
  return bytes_of(p, n > INT64_MAX / 2 ? INT64_MAX / 2 : (int64_t)n);
}
inline bool apart(const Region& a, const Region& b) { return a.end <= b.first || b.end <= a.first; }

// Each of `written` apart from the others and from all that is read.
inline bool apart(std::initializer_list<Region> written, std::initializer_list<Region> read) {
  for (const Region* w = written.begin(); w != written.end(); ++w) {
    for (const Region* o = written.begin(); o != w; ++o)
      if (!apart(*w, *o)) return false;
    for (const Region& r : read)
      if (!apart(*w, r)) return false;
  }
  return true;
}

}  // namespace dsa
