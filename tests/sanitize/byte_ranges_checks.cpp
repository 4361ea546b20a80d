// overlap() of csrc/byte_ranges.h against a map of the bytes (test infrastructure), over small
// matrices of every start, width and step around each other. Exit status 0 = clean.
#include <stdint.h>
#include <stdio.h>

#include <vector>

#include "byte_ranges.h"

using moelora::Bytes;

static char memory[256];

static bool shared(const Bytes& a, const Bytes& b) {
  std::vector<bool> in(sizeof memory, false);
  for (int64_t i = 0; i < a.rows; ++i)
    for (int64_t c = 0; c < a.width; ++c) in[a.p - memory + i * a.step + c] = true;
  for (int64_t i = 0; i < b.rows; ++i)
    for (int64_t c = 0; c < b.width; ++c)
      if (in[b.p - memory + i * b.step + c]) return true;
  return false;
}

int main() {
  std::vector<Bytes> all;
  for (int start = 0; start < 40; start += 3)
    for (int rows = 0; rows <= 4; ++rows)
      for (int width = 1; width <= 13; width += 3)
        for (int step = width; step <= width + 17; step += 2) all.push_back({memory + start, rows, width, step});
  int64_t yes = 0, no = 0;
  for (const Bytes& a : all)
    for (const Bytes& b : all) {
      const bool want = shared(a, b);
      if (moelora::overlap(a, b) != want) {
        fprintf(stderr, "start %d rows %d width %d step %d, start %d rows %d width %d step %d: expected %d\n",
                (int)(a.p - memory), (int)a.rows, (int)a.width, (int)a.step, (int)(b.p - memory), (int)b.rows,
                (int)b.width, (int)b.step, (int)want);
        return 1;
      }
      ++(want ? yes : no);
    }
  const Bytes none = moelora::dense_bytes(nullptr, 0), one = moelora::dense_bytes(memory, 1);
  if (moelora::overlap(none, one) || moelora::overlap(one, none) || !moelora::overlap(one, one)) return 1;
  printf("byte ranges: ok, %lld share a byte, %lld do not\n", (long long)yes, (long long)no);
  return 0;
}
