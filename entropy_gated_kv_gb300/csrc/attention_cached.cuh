// attention_cached.cuh — work plan of the cached attentions (attention_cached.cu), made on the
// device from the recompute-set sizes and key lengths, by the attention kernel and by its merge.
//
// A tile is 128 packed query rows (a row of a sequence and one of the g query heads of a KV head)
// of one KV head; a unit is a tile times one block of 128 keys. All units stand in one line, tile
// after tile, and CTA c takes the units [c chunk, (c + 1) chunk): every SM gets the same number
// of key blocks whatever the batch, heads and lengths are. The part of a tile that falls to one CTA
// is an item; a tile with one item is finished by it, one with several leaves partial rows in the
// workspace for the merge.
//   separate  a tile holds rows of one sequence and runs over the prefix's blocks, then the sequence's own
//   shared    rows of all sequences are packed into tiles for the prefix's blocks, each sequence's
//             rows into tiles for its own blocks, and every row is merged. Taken when it saves
//             more than an eighth of the units (tiles that were mostly padding), which pays for
//             the merge of every row.
#pragma once

#include <cstdint>

#include "ec_common.cuh"

namespace ec {
namespace cached {

constexpr int kBlockM = 128;  // packed query rows per tile (TMEM lanes)
constexpr int kBlockN = 128;  // keys per block

struct Shape {
  const int32_t *R, *kv_len;
  int32_t B, L, Lk, Lp, Hkv, g;  // own keys [0, Lk) without kv_len; Lp prefix positions
  int32_t ctas, slots;           // CTAs of the attention grid, partial tiles that the workspace holds
};

struct Plan {
  int64_t units;    // all units
  int64_t own0;     // shared: units of the prefix tiles, which come first
  int64_t rows;     // packed rows of one KV head over all sequences
  int64_t chunk;    // units per CTA
  int32_t nbp;      // key blocks of the prefix
  int32_t ptiles;   // shared: prefix tiles (KV head major), 0 otherwise
  int32_t otiles;   // tiles of single sequences
  bool shared;
  int32_t rows_l, len_l;  // B <= 32: rows and keys of sequence `lane`
};

struct Item {
  int32_t b, kvh;    // b = -1: rows of several sequences (a shared prefix tile)
  int64_t row0;      // first packed row: within the sequence, or over all of them (b = -1)
  int32_t nrows;     // valid rows, 1 .. 128
  int32_t np;        // the tile's blocks [0, np) are the prefix's, the rest the sequence's own
  int32_t units;     // blocks of the whole tile
  int32_t j0, nblk;  // this item's blocks [j0, j0 + nblk)
  int32_t tile;      // index over all tiles
  int32_t len;       // own keys of the sequence
};

EC_DEV int64_t div_fast(int64_t a, int64_t b) {  // a >= 0, b > 0; the 32-bit form when both fit
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

template <typename T>
EC_DEV T warp_total(T v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

template <typename T>
EC_DEV T warp_inclusive(T v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += u;
  }
  return v;
}

// Rows and own keys of sequence b. A bad R or length leaves the sequence out (no rows).
EC_DEV void load_seq(const Shape& s, int b, int32_t& rows, int32_t& len, int32_t* dev_err, bool report) {
  rows = 0;
  len = 0;
  if (b >= s.B) return;
  const int r = __ldcg(s.R + b);
  const int n = s.kv_len != nullptr ? __ldcg(s.kv_len + b) : s.Lk;
  const bool bad_r = r < 0 || r > s.L, bad_n = n < 0 || n > s.L;
  if (report && bad_r) report_error(dev_err, EC_DEVERR_BAD_R);
  if (report && bad_n) report_error(dev_err, EC_DEVERR_BAD_LEN);
  if (bad_r || bad_n) return;
  rows = r;
  len = min(n, s.Lk);
}

EC_DEV void seq_of(const Shape& s, const Plan& pl, int b, int32_t& rows, int32_t& len) {
  if (s.B <= 32) {
    rows = pl.rows_l;
    len = pl.len_l;
  } else {
    load_seq(s, b, rows, len, nullptr, false);
  }
}

EC_DEV int tiles_of(const Shape& s, int32_t rows) {
  return static_cast<int>((static_cast<int64_t>(rows) * s.g + kBlockM - 1) / kBlockM);
}
EC_DEV int blocks_of(int32_t len) { return (len + kBlockN - 1) / kBlockN; }

// Blocks of one tile of a sequence. A sequence without any key still has one, all of it masked,
// so that its rows are written (as zeros).
EC_DEV int tile_units(const Plan& pl, int32_t len) {
  return pl.shared ? blocks_of(len) : max(1, pl.nbp + blocks_of(len));
}

// Whole warp; every warp of both kernels computes the same plan.
EC_DEV Plan make_plan(const Shape& s, int32_t* dev_err, bool report) {
  const int lane = threadIdx.x & 31;
  Plan pl;
  pl.nbp = blocks_of(s.Lp);
  pl.rows_l = pl.len_l = 0;
  int64_t rows = 0, apart = 0, own = 0;
  int32_t tiles = 0;
  for (int b = lane; b < s.B; b += 32) {
    int32_t r, n;
    load_seq(s, b, r, n, dev_err, report);
    if (b == lane) {
      pl.rows_l = r;
      pl.len_l = n;
    }
    const int t = s.Hkv * tiles_of(s, r);
    rows += static_cast<int64_t>(r) * s.g;
    tiles += t;
    apart += static_cast<int64_t>(t) * max(1, pl.nbp + blocks_of(n));
    own += static_cast<int64_t>(t) * blocks_of(n);
  }
  pl.rows = warp_total(rows);
  pl.otiles = warp_total(tiles);
  apart = warp_total(apart);
  own = warp_total(own);
  const int64_t ptiles = static_cast<int64_t>(s.Hkv) * ((pl.rows + kBlockM - 1) / kBlockM);
  const int64_t together = ptiles * pl.nbp + own;
  pl.shared = pl.nbp > 0 && ptiles + pl.otiles + s.ctas <= s.slots && 8 * together <= 7 * apart;
  pl.ptiles = pl.shared ? static_cast<int32_t>(ptiles) : 0;
  pl.own0 = pl.shared ? ptiles * pl.nbp : 0;
  pl.units = pl.shared ? together : apart;
  pl.chunk = max(int64_t(1), div_fast(pl.units + s.ctas - 1, s.ctas));
  return pl;
}

// Whole warp: the tile that holds unit u, from its block u on.
EC_DEV Item item_at(const Shape& s, const Plan& pl, int64_t u) {
  const int lane = threadIdx.x & 31;
  Item it;
  if (u < pl.own0) {
    const int t = static_cast<int>(div_fast(u, pl.nbp)), per_head = pl.ptiles / s.Hkv;
    it.b = -1;
    it.kvh = t / per_head;
    it.row0 = static_cast<int64_t>(t - it.kvh * per_head) * kBlockM;
    it.nrows = static_cast<int32_t>(min(static_cast<int64_t>(kBlockM), pl.rows - it.row0));
    it.np = it.units = pl.nbp;
    it.j0 = static_cast<int32_t>(u - static_cast<int64_t>(t) * pl.nbp);
    it.tile = t;
    it.len = 0;
    return it;
  }
  int64_t base = pl.own0;
  int32_t tbase = pl.ptiles;
  for (int b0 = 0; b0 < s.B; b0 += 32) {
    int32_t r, n;
    seq_of(s, pl, b0 + lane, r, n);
    const int32_t t = s.Hkv * tiles_of(s, r), tu = tile_units(pl, n);
    const int64_t incl = warp_inclusive(static_cast<int64_t>(t) * tu);
    const int64_t total = __shfl_sync(0xffffffffu, incl, 31);
    if (u < base + total) {
      const int src = __ffs(__ballot_sync(0xffffffffu, base + incl > u)) - 1;
      const int64_t before = __shfl_sync(0xffffffffu, incl - static_cast<int64_t>(t) * tu, src);
      const int32_t tincl = warp_inclusive(t);
      const int32_t tbefore = __shfl_sync(0xffffffffu, tincl - t, src);
      const int32_t rsel = __shfl_sync(0xffffffffu, r, src);
      it.len = __shfl_sync(0xffffffffu, n, src);
      it.units = __shfl_sync(0xffffffffu, tu, src);
      it.b = b0 + src;
      const int64_t w = u - base - before;
      const int32_t tl = static_cast<int32_t>(div_fast(w, it.units));
      const int32_t per_head = tiles_of(s, rsel);
      it.kvh = tl / per_head;
      it.row0 = static_cast<int64_t>(tl - it.kvh * per_head) * kBlockM;
      it.nrows = static_cast<int32_t>(min(static_cast<int64_t>(kBlockM), static_cast<int64_t>(rsel) * s.g - it.row0));
      it.np = pl.shared ? 0 : pl.nbp;
      it.j0 = static_cast<int32_t>(w - static_cast<int64_t>(tl) * it.units);
      it.tile = tbase + tbefore + tl;
      return it;
    }
    base += total;
    tbase += warp_total(t);
  }
  it.nrows = it.units = it.nblk = 0;  // not reached: u is below pl.units
  it.b = it.kvh = it.j0 = it.np = it.len = it.tile = 0;
  it.row0 = 0;
  return it;
}

// The item of CTA c that starts at unit u (u below its end).
EC_DEV Item cta_item(const Shape& s, const Plan& pl, int64_t u, int64_t end) {
  Item it = item_at(s, pl, u);
  it.nblk = static_cast<int32_t>(min(static_cast<int64_t>(it.units - it.j0), end - u));
  return it;
}

EC_DEV bool item_complete(const Plan& pl, const Item& it) { return !pl.shared && it.nblk == it.units; }

// Where an incomplete item of CTA c leaves its partial rows. Shared: tile + c grows from item to
// item, so no two share a slot. Separate: a CTA has at most two incomplete items, one that began
// before it and one that ends after it.
EC_DEV int64_t item_slot(const Plan& pl, const Item& it, int c) {
  return pl.shared ? static_cast<int64_t>(it.tile) + c : 2 * static_cast<int64_t>(c) + (it.j0 == 0 ? 1 : 0);
}

}  // namespace cached
}  // namespace ec
