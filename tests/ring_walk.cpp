// For each number of rows, stages and row k at which a walk is left (k = rows: at
// its end) a line with what it asked for, counted as norm_rows_kernel issues its
// copies, and what RowRing says of it:
//   rows stages k issued: parity of each stage that is waited for
#include <cstdio>

#include "ring.h"

int main() {
  for (int rows = 1; rows <= 24; ++rows)
    for (int stages = 2; stages <= 6; ++stages)
      for (int left = 0; left <= rows; ++left) {
        int copies = 0, k = 0;
        for (int i = 0; i < stages && i < rows; ++i) ++copies;
        for (; k < rows; ++k) {
          if (k == left) break;                  // a wait gave up
          if (k + stages < rows) ++copies;
        }
        const hb::RowRing ring(stages, rows, k);
        std::printf("%d %d %d %d:", rows, stages, left, copies);
        for (int s = 0; s < ring.used(); ++s) std::printf(" %u", ring.last_parity(s));
        std::printf("\n");
      }
  return 0;
}
