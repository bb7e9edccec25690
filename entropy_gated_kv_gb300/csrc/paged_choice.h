// paged_choice.h — which form a paged attention takes, from what the host knows of a call: sizes, the window, whether
// lengths and positions come from the device.
#pragma once

#include <algorithm>

#include "ec_internal.h"

namespace ec {
namespace paged {

// attention_paged_rows.cu: at most kFewRows packed rows (positions times the heads of a KV head) a sequence, the rows of
// one mma.sync tile. (With two such tiles a warp the products bound it: 8 x 32 rows of 32 heads behind 2048 keys, ragged,
// 66 us there and 46 as tiles of 128; 4 rows of 28/4 heads behind 2048 keys 12.0 and 8.8.)
constexpr int kFewRows = 16;
// attention_paged_tiles.cu: tiles of nr positions, nr times the heads of a KV head at most 128 packed rows.
constexpr int kTileRows = 128;
constexpr int kStepKeys = 128;  // of a CTA's step in either

inline bool few_rows(const ec_params& p, int32_t rows_max) { return static_cast<int64_t>(rows_max) * (p.Hq / p.Hkv) <= kFewRows; }
// Positions of a tile.
inline int tile_positions(const ec_params& p, int32_t rows_max) { return std::min(kTileRows / (p.Hq / p.Hkv), rows_max); }

constexpr int kMaxCluster = 8;
// What the launches ask of a device, found once: its SMs, and clusters of S CTAs, one an SM, that are on it at once (a part
// of the GPU need not have a multiple of S SMs: 15 clusters of 8 on 152).
struct Device {
  int sms, clusters[kMaxCluster + 1];
};
// CTAs of a cluster that `items` clusters can have at once.
inline int cluster_for(const Device& d, int64_t items) {
  int S = kMaxCluster;
  while (S > 1 && d.clusters[S] < items) --S;
  return S;
}

// The keys of an item, in steps: `likely` ones, and as many as it may have where its rows may lie apart (all of the sequence; where
// there is one sequence only, its `groups` of rows share it out). `ragged`: only the device knows which items have them and
// which have few.
struct Reach {
  int64_t likely, most;
  bool ragged;
};
inline Reach reach_of(const ec_params& p, int32_t rows_max, const Window* w, const RowPlaces& at, bool lengths, int64_t groups, int slack) {
  const int64_t scope = scope_hi(p);
  auto steps = [](int64_t keys) { return (keys + kStepKeys - 1) / kStepKeys; };
  if (w == nullptr) return {steps(scope), steps(scope), p.B > 1 && lengths};
  // Rows beside each other, as a start has them and a block's idx too. A window that is less than half of the scope bounds
  // what a long sequence reads; one without a bound on a side does not.
  const int64_t keys = std::min<int64_t>(scope, static_cast<int64_t>(w->left) + w->right + w->sinks + rows_max + slack);
  const bool vary = p.B > 1 && (lengths || at.idx != nullptr || at.start != nullptr);
  const int64_t most = at.idx != nullptr && rows_max > 1 ? std::max(keys, p.B > 1 ? scope : scope / groups) : keys;
  return {steps(keys), steps(most), vary && 2 * keys > scope};
}

// Whether each of `items` items goes to a cluster of S CTAs and is joined there, or all stand in the line, at the cost of a second launch and
// its join, `join` steps of a full GPU. `full` CTAs and more share the HBM's rate, fewer take their own. One item with many
// keys may be all that a cluster's call waits for: where items may differ, clusters only where that is no more than `ragged`
// such steps, and where rows may lie apart, no more than `apart`.
struct Cost {
  int64_t full, join, ragged, apart;
};
inline bool cluster_pays(const Device& d, int64_t items, int S, const Reach& r, const Cost& c) {
  auto alone = [&](int64_t steps) { return (steps + S - 1) / S * c.full; };
  if (r.most > r.likely && alone(r.most) > c.apart * d.sms) return false;
  if (r.ragged) return alone(r.likely) <= c.ragged * d.sms;
  return (r.likely + S - 1) / S * std::max(items * S, c.full) <= items * r.likely + c.join * d.sms;
}

// CTAs of a cluster for each item, 0: shares of the line.
// Few rows: a step takes a CTA 0.7 us by itself and 1.5 in a full GPU; a second launch and its join 1 to 4 us. Line and clusters measured: one token
// of 28/4 heads behind 4096 keys 9.9 and 9.0 us, behind 8192 11.3 and 11.8, behind 16384 13.7 and 17.6; 3 tokens of 32 heads (clusters
// of one CTA) behind 2048 24.2 and 20.7, behind 4096 39.3 and 37.1; 12 of 28/4 behind 8192 40.9 and 37.9.
// Windows plan longer in the line (positions are read too), so more is left to clusters there. Tokens of 28/4 heads that see
// all keys before them, line and clusters, every sequence long and one of them (in brackets a long item's own cost): 4 x 8192 keys
// (5 steps) 21.7 and 17.2, 12.7 and 14.5; 16 x 8192 (15) 51.5 and 46.8, 17.4 and 29.2; 16 x 32768 (61) 170 and 169, 27 and 97; the last 16384 of
// 32768: 92 and 87, 23 and 53; the last 8192: 52 and 47, 20 and 31. Two rows with 512 keys to either side, beside each other and all over
// the sequence: 4 x 32768 (20) 11 and 8, 17 and 15; 16 x 16384 (30) 17 and 9, 42 and 49, one sequence's alone apart 19 and 38; 16 x 32768 (61)
// 17 and 9, 82 and 87, one long sequence of 16 with its rows apart 26 and 77.
inline int few_rows_cluster(const ec_params& p, int32_t rows_max, const Window* w, const RowPlaces& at, bool lengths, const Device& d) {
  const int64_t items = static_cast<int64_t>(p.B) * p.Hkv;
  if (items > d.sms) return 0;
  const int S = cluster_for(d, items);
  const Cost cost{72, 2, w != nullptr ? 8 : 4, 32};
  return cluster_pays(d, items, S, reach_of(p, rows_max, w, at, lengths, 1, 32), cost) ? S : 0;
}
// Tiles: a second launch costs some six blocks. Line and clusters measured: 95 rows of 28/4 heads
// behind 16384 keys 44 and 40 us, behind 24576 47 and 53; 512 rows behind 8192 61 and 67; 95 rows of 32 heads behind 32768 95 and 86; 18 rows
// of 28/4 behind 16384 30 and 27, behind 32768 38 and 43. Pairs in clusters of one CTA are off: 1024 rows of 32 heads 25 and 33.
// 32 rows of 28/4 heads that see all keys before them, every sequence long and one of them: 4 x 8192 keys (11 steps) 36 and 31, 35 and 29;
// 16 x 4096 (16) 45 and 41, 27 and 40. Rows with 512 keys to either side, beside each other, all over their sequences, one
// sequence's alone apart: 4 rows, one tile, 4 x 32768 (24) 14 and 9, 45 and 47, 28 and 31, 16 x 16384 (36) 15 and 11, 73 and 77, 26 and 54; 95
// rows, pairs, 2 x 8192 (13) 22 and 16, 33 and 28, 31 and 27, 4 x 8192 (22) 24 and 21, 40 and 49, 31 and 45, 4 x 32768 (86) 22 and 21, 77 and
// 126, 44 and 106; of one sequence 1 x 32768 (11) 21 and 14, 44 and 43, 32 rows (32) 17 and 13, 43 and 69.
inline int tiles_cluster(const ec_params& p, int32_t rows_max, int nr, const Window* w, const RowPlaces& at, bool lengths, const Device& d) {
  const bool pair = rows_max > nr;
  const int64_t step = pair ? 2 * nr : nr, groups = (rows_max + step - 1) / step, items = static_cast<int64_t>(p.B) * p.Hkv * groups;
  if (items > d.sms) return 0;
  const int S = cluster_for(d, items);
  if (S == 1 && pair) return 0;
  // the split form's blocks take a CTA 0.8 us by itself: more than 85 share the HBM's rate
  const Cost cost{pair ? d.sms : 85, 6, 12, pair ? 15 : 30};
  return cluster_pays(d, items, S, reach_of(p, rows_max, w, at, lengths, groups, 2 * kStepKeys), cost) ? S : 0;
}

}  // namespace paged
}  // namespace ec
