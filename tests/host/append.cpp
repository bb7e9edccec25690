// The pieces of the paged append (paged_common.cuh): the rows below R fall to the CTAs once, row by row, and no CTA takes a
// piece past them, up to the most rows and the widest rows that the interface accepts.
//   argv: rows_max, pieces of a row, pieces of a CTA at once, R [, "wrapped"]: the product in 32 bits for every CTA
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "host_warp.h"

#include "paged_common.cuh"

namespace {

// The product as it must not be: also formed where the CTA's rows begin past the last one.
int wrapped(const ec::paged::RowSplit& s, int r0, int rows) {
  return static_cast<int>(static_cast<uint32_t>(min(s.rows_per_cta, rows - r0)) * static_cast<uint32_t>(s.pieces));
}

}  // namespace

int main(int argc, char** argv) {
  const int rows_max = std::atoi(argv[1]), pieces = std::atoi(argv[2]), at_once = std::atoi(argv[3]), R = std::atoi(argv[4]);
  const bool planted = argc > 5 && std::strcmp(argv[5], "wrapped") == 0;
  ec::paged::RowSplit s;
  s.set(rows_max, pieces, at_once);
  int64_t next = 0;  // row
  for (int64_t r0 = 0; r0 < rows_max; r0 += s.rows_per_cta) {
    const int n = planted ? wrapped(s, static_cast<int>(r0), R) : s.count(static_cast<int>(r0), R);
    if (n <= 0) continue;
    if (n % pieces != 0) return std::printf("part of a row: %d pieces at row %lld\n", n, (long long)r0), 1;
    const int rows = n / pieces;
    if (r0 != next || r0 + rows > R) return std::printf("row %lld, %d pieces\n", (long long)r0, n), 1;
    // the first and the last piece of a row as the kernel finds them
    for (int i = 0; i < rows; ++i)
      for (const int u : {i * pieces, (i + 1) * pieces - 1})
        if (s.per_row(u) != i) return std::printf("piece %d is of row %d\n", u, s.per_row(u)), 1;
    next = r0 + rows;
  }
  if (next != R) return std::printf("rows from %lld on are left out\n", (long long)next), 1;
  std::puts("ok");
  return 0;
}
