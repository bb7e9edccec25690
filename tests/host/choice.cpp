// Which form a paged attention takes (paged_choice.h) on a GB300, with the clusters that one has there.
//   argv: B L Hq Hkv rows_max left right sinks (left -2: no window) places ("idx", "start", "none") lengths (0, 1)
//   prints "rows" or "tiles", and the CTAs of a cluster (0: shares of the line)
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "paged_choice.h"

using namespace ec;

int main(int, char** argv) {
  ec_params p{};
  p.B = std::atoi(argv[1]), p.L = std::atoi(argv[2]), p.Hq = std::atoi(argv[3]), p.Hkv = std::atoi(argv[4]), p.D = 128;
  const int rows_max = std::atoi(argv[5]), left = std::atoi(argv[6]), right = std::atoi(argv[7]);
  constexpr int kAll = 1 << 20;
  const Window w{left < 0 ? kAll : left, right < 0 ? kAll : right, std::atoi(argv[8])};
  const int32_t here = 0;
  RowPlaces at{};
  if (std::strcmp(argv[9], "idx") == 0) at.idx = &here;
  if (std::strcmp(argv[9], "start") == 0) at.start = &here;
  const paged::Device d{152, {0, 152, 76, 46, 36, 28, 23, 15, 15}};
  const Window* window = left == -2 ? nullptr : &w;
  const bool lengths = std::atoi(argv[10]) != 0;
  if (paged::few_rows(p, rows_max))
    std::printf("rows %d\n", paged::few_rows_cluster(p, rows_max, window, at, lengths, d));
  else
    std::printf("tiles %d\n", paged::tiles_cluster(p, rows_max, paged::tile_positions(p, rows_max), window, at, lengths, d));
  return 0;
}
