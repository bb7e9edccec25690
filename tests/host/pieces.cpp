// The pieces of a line of rows (quant_common.cuh): every piece falls to one CTA once, and no row index
// leaves the line, up to the longest line that the interface accepts.
//   argv: rows, piece, ctas [, "signed"]: the same loop with a signed counter, whose last step wraps
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "host_warp.h"

#include "quant_common.cuh"

namespace {

// The loop as it must not be: 32-bit arithmetic with a sign.
struct SignedPieces {
  int32_t at, n, step;
  SignedPieces(int32_t rows, uint32_t piece, uint32_t cta, uint32_t ctas)
      : at(static_cast<int32_t>(cta * piece)), n(rows), step(static_cast<int32_t>(ctas * piece)) {}
  bool more() const { return at < n; }
  void next() { at = static_cast<int32_t>(static_cast<uint32_t>(at) + static_cast<uint32_t>(step)); }
};

template <class P>
int check(int32_t rows, uint32_t piece, uint32_t ctas) {
  const int64_t pieces = (static_cast<int64_t>(rows) + piece - 1) / piece;
  std::vector<uint8_t> seen(static_cast<size_t>(pieces), 0);
  for (uint32_t c = 0; c < ctas; ++c) {
    int64_t turns = 0;
    for (P line(rows, piece, c, ctas); line.more(); line.next()) {
      const int64_t at = line.at;
      if (at < 0 || at >= rows || at % piece != 0 || ++turns > pieces) return std::printf("row %lld\n", (long long)at), 1;
      if (seen[static_cast<size_t>(at / piece)]++ != 0) return std::printf("twice: row %lld\n", (long long)at), 1;
      // the rows of the piece past the line's end are told from those within
      for (uint32_t i = 0; i < piece; ++i)
        if ((line.at + i < line.n) != (at + i < rows)) return std::printf("row %lld + %u\n", (long long)at, i), 1;
    }
  }
  for (int64_t i = 0; i < pieces; ++i)
    if (seen[static_cast<size_t>(i)] != 1) return std::printf("left out: piece %lld\n", (long long)i), 1;
  std::puts("ok");
  return 0;
}

}  // namespace

int main(int argc, char** argv) {
  const int32_t rows = std::atoi(argv[1]);
  const uint32_t piece = std::atoi(argv[2]), ctas = std::atoi(argv[3]);
  return argc > 4 && std::strcmp(argv[4], "signed") == 0 ? check<SignedPieces>(rows, piece, ctas)
                                                         : check<ec::Pieces>(rows, piece, ctas);
}
