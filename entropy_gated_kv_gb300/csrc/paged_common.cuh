// paged_common.cuh — what the kernels over a paged K/V cache share: where a call's rows stand, which
// keys they see, the line of work that the CTAs cut into shares, and the partial rows that a cut leaves.
#pragma once

#include <cuda.h>

#include <algorithm>

#include "ec_common.cuh"
#include "ec_internal.h"
#include "paged_choice.h"

namespace ec {
namespace paged {

constexpr int kMaxCtas = 160;  // bound of the attention grids, for the workspace
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.f;  // the running maximum is moved when it grows by more than 2^8
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per pipeline wait

// An item that is cut between CTAs, as the CTA that begins it leaves it for the merge: parts 0 (nothing to merge) or
// the number of CTAs from this one on that hold partial rows of it.
struct Record {
  int32_t parts, b, kvh, row0, rows;  // packed rows row0 .. row0 + rows - 1 of (b, kvh)
  int32_t pad[3];
};

struct Shape {
  int32_t B, L, Hq, Hkv, g, rows_max, scope_hi, windowed, page_shift, n_pages;
  int64_t table_stride;
  float scale_log2;
  FastDiv by_g;
  Window w;
  RowPlaces at;
  const int32_t *R, *kv_len, *table;
  int32_t* dev_err;
};

struct Args {
  CUtensorMap tk, tv, tq;
  Shape s;
  const uint16_t* q;
  uint16_t* out;
  float* part_o;      // [slots][16][D] (few rows), [slots][D / 4][128][4] (tiles)
  float2* part_stat;  // [slots][rows of a slot]: running maximum (base 2, scaled; NaN: the row is not written) and sum
  Record* records;    // [CTAs]
};

// How the append's rows fall to its CTAs: rows of `pieces` pieces each, as many to a CTA as make `at_once` pieces, one at
// least.
struct RowSplit {
  int32_t pieces, rows_per_cta;
  FastDiv per_row;
  void set(int32_t rows_max, int32_t row_pieces, int32_t at_once) {
    pieces = row_pieces;
    rows_per_cta = std::min(rows_max, std::max(1, at_once / row_pieces));
    per_row.set(row_pieces);
  }
  // Pieces of the CTA whose rows begin at r0, of `rows` in all; at most pieces or at_once. A CTA past the last row has none:
  // rows - r0 times pieces would leave 32 bits there.
  EC_DEV int count(int r0, int rows) const { return r0 < rows ? min(rows_per_cta, rows - r0) * pieces : 0; }
};

// Position of row r of sequence b; it may lie outside [0, L).
EC_DEV int64_t raw_position(const RowPlaces& at, int b, int r) {
  if (at.idx != nullptr) return __ldg(at.idx + b * at.stride + r);
  return at.start != nullptr ? static_cast<int64_t>(__ldg(at.start + b)) + r : r;
}
EC_DEV bool inside(int64_t pos, int L) { return pos >= 0 && pos < L; }

// Rows and keys of sequence b; rows 0 where a size is bad (`tell`: reported).
EC_DEV void sizes_of(const Shape& s, int b, bool tell, int& rows, int& keys) {
  rows = __ldg(s.R + b);
  keys = s.kv_len == nullptr ? s.scope_hi : __ldg(s.kv_len + b);
  if (rows < 0 || rows > s.rows_max) {
    if (tell) report_error(s.dev_err, EC_DEVERR_BAD_R);
    rows = 0;
  }
  if (keys < 0 || keys > s.L) {
    if (tell) report_error(s.dev_err, EC_DEVERR_BAD_LEN);
    rows = keys = 0;
  }
  keys = min(keys, s.scope_hi);
}

// The keys that rows r0 .. r1 - 1 of a sequence of n keys see between them: j < near, or lo <= j < hi.
struct Hull {
  int near, lo, hi;
};
// first: the position of row r0, which a caller may ask for before it knows the sizes.
EC_DEV Hull hull_of(const Shape& s, int b, int r0, int r1, int n, int64_t first) {
  if (!s.windowed) return {0, 0, n};
  int64_t p0 = first, p1 = r1 - 1 == r0 ? first : raw_position(s.at, b, r1 - 1);
  while (!inside(p0, s.L) && r0 + 1 < r1) p0 = raw_position(s.at, b, ++r0);  // rows at bad positions are not written
  while (!inside(p1, s.L) && r0 + 1 < r1) p1 = raw_position(s.at, b, --r1 - 1);
  if (!inside(p0, s.L) || !inside(p1, s.L)) return {0, 0, 0};
  Hull h;
  h.near = min(s.w.sinks, n);
  h.lo = min(max(static_cast<int>(p0) - s.w.left, 0), n);
  h.hi = max(min(static_cast<int>(p1) + s.w.right + 1, n), h.lo);
  return h;
}

// The hull's blocks of 2^shift keys in order: first those of the keys below near, then the others.
struct Blocks {
  int near, first, count;
  EC_DEV int block(int v) const { return v < near ? v : v - near + first; }
};
EC_DEV Blocks blocks_of(const Hull& h, int shift) {
  const int up = (1 << shift) - 1;
  Blocks k;
  k.near = (h.near + up) >> shift;
  k.first = max(h.lo >> shift, k.near);
  const int end = h.hi > h.lo ? (h.hi + up) >> shift : 0;
  k.count = k.near + max(0, end - k.first);
  return k;
}

// The page of position j of sequence b; a bad number is reported and reads as n_pages, past the
// tensor map's end, where a load fills in zeros.
EC_DEV int page_of(const Shape& s, int b, int j) {
  const int page = __ldg(s.table + b * s.table_stride + (j >> s.page_shift));
  if (page >= 0 && page < s.n_pages) return page;
  report_error(s.dev_err, EC_DEVERR_BAD_PAGE);
  return s.n_pages;
}

// Sizes, page numbers and first positions into L2, each line by one thread of the grid, before the wait for the kernel in
// front: a prefetch into L2, where that kernel's writes go too, reads nothing stale. The chain of sizes, first
// position, page number, keys has a DRAM access less at each step.
EC_DEV void prefetch_lines(const void* p, int64_t bytes, int64_t line) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p) / 128 * 128 + line * 128;
  if (at < reinterpret_cast<uintptr_t>(p) + bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(at) : "memory");
}
EC_DEV void prefetch_small(const Shape& s, int threads) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * threads + threadIdx.x;
  prefetch_lines(s.R, s.B * 4ll, i);
  if (s.kv_len != nullptr) prefetch_lines(s.kv_len, s.B * 4ll, i);
  prefetch_lines(s.table, ((s.B - 1) * s.table_stride + ((s.L + (1 << s.page_shift) - 1) >> s.page_shift)) * 4, i);
  if (s.windowed && s.at.idx != nullptr && i < s.B) prefetch_lines(s.at.idx + i * s.at.stride, 4, 0);
  if (s.windowed && s.at.start != nullptr) prefetch_lines(s.at.start, s.B * 4ll, i);
}

EC_DEV int warp_inclusive(int x) {
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, i);
    if ((threadIdx.x & 31) >= i) x += y;
  }
  return x;
}

EC_DEV uint4 ld_shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}
EC_DEV float4 ld_dsmem16(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
EC_DEV float2 ld_dsmem8(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
EC_DEV void st_shared16(uint32_t dst, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// cluster 0: shares of the line, partial rows where items are cut; else a cluster of so many CTAs for each item.
cudaError_t launch_few_rows(const Args& a, int D, int ctas, int cluster, cudaStream_t s);
cudaError_t launch_tiles(const Args& a, int D, int nr, int ctas, int cluster, cudaStream_t s);
cudaError_t setup_few_rows(Device* d);  // the kernels' shared memory, and d->clusters
cudaError_t setup_tiles();
// A CTA leaves two cut items at most, one that goes on in it and one that begins there: slots
// 2 tiles cta + tile and 2 tiles cta + tiles + tile, with one tile or two beside each other.
EC_DEV int64_t part_slot(int first_cta, int i, int tiles, int tile) {
  return static_cast<int64_t>(first_cta + i) * 2 * tiles + (i == 0 ? tiles : 0) + tile;
}
EC_DEV float kNotWritten() { return __int_as_float(0x7fffffff); }

}  // namespace paged
}  // namespace ec
