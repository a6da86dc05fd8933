// Host check of csrc/regions.h: prints "ok" when every case holds.
#include <cstdio>

#include "regions.h"

using namespace dsa;

int main() {
  const void* p = reinterpret_cast<const void*>(4096);
  const void* q = reinterpret_cast<const void*>(4096 + 64);
  const void* last = reinterpret_cast<const void*>(4096 + 63);
  int bad = 0;
  auto is = [&](bool got, bool want, const char* what) {
    if (got != want) bad = 1, std::printf("%s\n", what);
  };
  is(apart(bytes_of(p, 64), bytes_of(q, 64)), true, "neighbours");
  is(apart(bytes_of(p, 65), bytes_of(q, 64)), false, "a byte");
  is(apart(bytes_of(last, 1), bytes_of(p, 64)), false, "the last byte");
  is(apart(bytes_of(p, 64), bytes_of(p, 64)), false, "the same");
  is(apart(bytes_of(nullptr, 64), bytes_of(nullptr, 64)), true, "no pointers");
  is(apart(bytes_of(p, 0), bytes_of(p, 64)), true, "no bytes");
  // Rows: [2][3][8] 16-bit values, tokens 64 and heads 16 apart, end at (64 + 32 + 8) * 2.
  is(rows_of(p, 2, 64, 3, 16, 8, 2).end == 4096 + 208, true, "rows' end");
  is(rows_of(p, 2, 16, 3, 64, 8, 2).end == 4096 + (16 + 128 + 8) * 2, true, "heads outside");
  is(rows_of(p, 1, 1ll << 40, 1, 1ll << 40, 8, 2).end == 4096 + 16, true, "one row's strides");
  is(rows_of(p, 0, 64, 3, 16, 8, 2).end == 0, true, "no rows");
  is(rows_of(p, 1ll << 31, 1ll << 37, 128, 1ll << 37, 192, 2).end > (1ull << 61), true, "past 64 bits");
  is(apart({bytes_of(p, 64), bytes_of(q, 64)}, {}), true, "two outputs");
  is(apart({bytes_of(p, 64), bytes_of(q, 64), bytes_of(last, 4)}, {}), false, "three outputs");
  is(apart({bytes_of(p, 64)}, {bytes_of(q, 64), bytes_of(last, 1)}), false, "an input");
  is(apart({bytes_of(p, 64)}, {bytes_of(q, 64), bytes_of(q, 8)}), true, "inputs may overlap");
  if (!bad) std::printf("ok\n");
  return bad;
}
