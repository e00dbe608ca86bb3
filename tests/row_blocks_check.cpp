// Row arithmetic of the weight gradients against plain 64-bit arithmetic; prints OK.  Built with
// overflow checks, so that a sum past 2^31 ends the program.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "row_blocks.h"

using namespace muon;

#define CHECK(x)                                                              \
  do {                                                                        \
    if (!(x)) {                                                               \
      std::printf("rows %lld: %s\n", (long long)rows, #x);                    \
      std::exit(1);                                                           \
    }                                                                         \
  } while (0)

void check(int64_t rows) {
  const int64_t blocks = (rows + 63) / 64;
  CHECK(row_blocks((int32_t)rows) == blocks);
  for (int shift = 0; shift <= 3; ++shift) {
    int64_t next = 0;
    for (int i = 0; i < 1 << shift; ++i) {
      const RowShare s = row_share((int32_t)rows, i, shift);
      // Shares follow one another, start on blocks, and differ by at most one block.
      CHECK(s.rows >= 0 && s.first % 64 == 0 && (s.rows == 0 || s.first == next));
      CHECK((s.rows + 63LL) / 64 >= (blocks >> shift) && (s.rows + 63LL) / 64 <= (blocks >> shift) + 1);
      next += s.rows;
    }
    CHECK(next == rows);
  }
  for (int most : {4, 6, 8, 11})
    for (int sub : {1, 2}) {
      if (sub == 2 && most % 2) continue;
      const int64_t seg = segment_blocks((int32_t)blocks, most, sub);
      CHECK(blocks == 0 ? seg == 0 : seg >= 1 && seg <= most && seg % sub == 0);
      // The loop over the segments ends, with no more of them than needed but for whole stages.
      if (blocks > 0) CHECK((blocks + seg - 1) / seg <= (blocks + most - 1) / most);
    }
}

int main() {
  for (int64_t rows = 0; rows < 20000; ++rows) check(rows);
  for (int64_t rows = INT32_MAX - 20000LL; rows <= INT32_MAX; ++rows) check(rows);
  uint64_t r = 1;
  for (int i = 0; i < 200000; ++i) {
    r = r * 6364136223846793005u + 1442695040888963407u;
    check((int64_t)(r >> 33));
  }
  std::printf("OK\n");
}
