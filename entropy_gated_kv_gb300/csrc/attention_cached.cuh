// attention_cached.cuh — work plan of the cached attentions (attention_cached.cu), made on the
// device from the recompute-set sizes and key lengths by one warp of every CTA of the attention
// kernel. It hands the CTA's items to the other warps through shared memory, and leaves what the
// merge kernel needs in the workspace. (Straight-line code that a CTA runs once costs about ten
// cycles an instruction, its fetch from the cold instruction cache: with the plan made by every
// warp, and again by the merge, a one-block call took 24.6 us, 12 of them before the first score.)
//
// A tile is 128 packed query rows (a row of a sequence and one of the g query heads of a KV head)
// of one KV head; a unit is a tile times one block of 128 keys. Each tile is followed by kTileCost
// units without a block, for the time between one tile and the next (its queries, the join, the
// rows' way out). All units stand in one line, tile after tile, and CTA c takes the units
// [c chunk, (c + 1) chunk): every SM gets about the same time whatever the batch, heads and lengths
// are. (Without the cost, a batch with a long shared prefix gave the last CTAs tens of two-block
// tiles for the others' 140 blocks: 602 us, of which half was waiting for them.) The part of a tile
// that falls to one CTA is an item; a tile with one item is finished by it, one with several leaves
// partial rows in the workspace for the merge.
//   separate  a tile holds rows of one sequence and runs over the prefix's blocks, then the sequence's own
//   shared    rows of all sequences are packed into tiles for the prefix's blocks, each sequence's
//             rows into tiles for its own blocks, and every row is merged. Taken when it saves
//             more than an eighth of the units (tiles that were mostly padding), which pays for
//             the merge of every row, and the workspace has a place for every tile's partial rows.
//   whole     as separate, with a tile to a CTA: taken when there are CTAs enough and the longest
//             tile is not kWholeExtra units above an equal share, as the partial rows and their merge
//             cost more than that (a ragged batch of 148 tiles of 9 to 16 blocks: 38 us cut into
//             equal shares, 9 of them the merge).
#pragma once

#include <cstdint>

#include "ec_common.cuh"

namespace ec {
namespace cached {

constexpr int kBlockM = 128;  // packed query rows per tile (TMEM lanes)
constexpr int kBlockN = 128;  // keys per block
constexpr int kTileCost = 3;  // blocks whose time a tile takes beside its own
constexpr int kWholeExtra = 5;  // units that a merge of all tiles costs

// Floor of x / d, 0 <= x < 2^31, quotients up to a few thousand: `inv` is 1 / d rounded, so the
// product's floor is at most one off.
EC_DEV int div_near(int x, int d, float inv) {
  int q = static_cast<int>(static_cast<float>(x) * inv);
  const int r = x - q * d;
  if (r < 0) --q;
  if (r >= d) ++q;
  return q;
}

struct Shape {
  const int32_t *R, *kv_len;
  int32_t B, L, Lk, Lp, Hkv, g;  // own keys [0, Lk) without kv_len; Lp prefix positions
  int32_t ctas, slots;           // CTAs of the attention grid, partial tiles that the workspace holds
  FastDiv div_g, div_h, div_ctas;  // by g, by Hkv and by ctas
};

// Units, packed rows of a KV head and rows of q are counted in 32 bits: the host checks that q has
// fewer than 2^31 rows, and a call of 2^31 units or more (seconds of work on every SM) is not run.
struct Plan {
  int32_t units;   // all units
  int32_t own0;    // shared: units of the prefix tiles, which come first
  int32_t rows;    // packed rows of one KV head over all sequences
  int32_t chunk;   // units per CTA
  int32_t nbp;     // key blocks of the prefix
  int32_t ptiles;  // shared: prefix tiles (KV head major), 0 otherwise
  int32_t otiles;  // tiles of single sequences
  int32_t whole;   // whole tiles: units of every tile's place in the line, 0 otherwise
  bool shared;
  int32_t rows_l, len_l;  // B <= 32: rows and keys of sequence `lane`
};

struct Item {
  int32_t b, kvh;    // b = -1: rows of several sequences (a shared prefix tile)
  int32_t row0;      // first packed row: within the sequence, or over all of them (b = -1)
  int32_t nrows;     // valid rows, 1 .. 128
  int32_t np;        // the tile's blocks [0, np) are the prefix's, the rest the sequence's own
  int32_t j0, nblk;  // this item's blocks [j0, j0 + nblk); nblk = 0 ends the CTA's work
  int32_t len;       // own keys of the sequence
  int32_t slot;      // where its partial rows go, -1: the tile is complete
  int32_t blocks;    // of the whole tile
  int32_t tile;      // index over all tiles
  int32_t before;    // packed rows of the sequences before b
};
static_assert(sizeof(Item) == 48, "three 16-byte words");

// What the merge reads: one record per tile of a single sequence (shared), or per CTA, for the tile
// that begins in it and does not end there (separate; nrows = 0 where there is none). A row's
// partials lie in n1 slots from a1 on and n2 slots from a2 on; shared, the first ones are those of
// the row's prefix tile, which the merge works out from the header.
struct Record {
  int32_t b, kvh, row0, nrows;
  int32_t a1, a2, n2, before;
};
struct Header {
  int32_t records, shared, prefix_units, chunk;  // units of a prefix tile, units of a CTA
  int32_t ptiles_head, nbp, rows, pad;           // of a KV head: prefix tiles, blocks of each, packed rows
};

// Quotients of numbers below 2^31 by a divisor that is known on the device only: the compiler's unsigned
// 32-bit division.
EC_DEV int div_down(int a, int b) { return static_cast<int>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)); }

EC_DEV int warp_total(int v) { return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v))); }

EC_DEV int warp_inclusive(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int off = 1; off < 32; off <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, off);
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

EC_DEV int tiles_of(const Shape& s, int32_t rows) { return (rows * s.g + kBlockM - 1) / kBlockM; }
EC_DEV int blocks_of(int32_t len) { return (len + kBlockN - 1) / kBlockN; }

// Blocks of one tile of a sequence. A tile without any key still has one block, all of it masked, so
// that its rows are written (as zeros) or, shared, so that a CTA leaves its record.
EC_DEV int tile_blocks(const Plan& pl, int32_t len) { return max(1, (pl.shared ? 0 : pl.nbp) + blocks_of(len)); }
// The units of its place in the line.
EC_DEV int tile_units(const Plan& pl, int blocks) { return pl.whole != 0 ? pl.whole : blocks + kTileCost; }

// Whole warp.
EC_DEV Plan make_plan(const Shape& s, int32_t* dev_err, bool report) {
  const int lane = threadIdx.x & 31;
  Plan pl;
  pl.nbp = blocks_of(s.Lp);
  pl.rows_l = pl.len_l = 0;
  int rows = 0, apart = 0, own = 0, tiles = 0, longest = 0;
  float most = 0.f;  // units as a float: 2^31 and more are seen there
#pragma unroll 1
  for (int b = lane; b < s.B; b += 32) {
    int32_t r, n;
    load_seq(s, b, r, n, dev_err, report);
    if (b == lane) {
      pl.rows_l = r;
      pl.len_l = n;
    }
    const int t = s.Hkv * tiles_of(s, r), nb = blocks_of(n);
    rows += r * s.g;
    tiles += t;
    apart += t * (max(1, pl.nbp + nb) + kTileCost);
    own += t * (max(1, nb) + kTileCost);
    if (t > 0) longest = max(longest, max(1, pl.nbp + nb) + kTileCost);
    most += static_cast<float>(t) * static_cast<float>(pl.nbp + nb + 1 + 2 * kTileCost);
  }
  pl.rows = warp_total(rows);
  pl.otiles = warp_total(tiles);
  apart = warp_total(apart);
#pragma unroll 1
  for (int off = 16; off > 0; off >>= 1) most += __shfl_xor_sync(0xffffffffu, most, off);
  if (most > 2.1e9f) {
    if (report && lane == 0) report_error(dev_err, EC_DEVERR_BAD_R);
    apart = 0;
  }
  pl.shared = false;
  pl.ptiles = pl.own0 = 0;
  pl.units = apart;
  pl.whole = 0;
  if (pl.nbp > 0 && s.B > 1) {
    const int ptiles = s.Hkv * ((pl.rows + kBlockM - 1) / kBlockM);
    const int together = ptiles * (pl.nbp + kTileCost) + warp_total(own);
    pl.shared = apart > 0 && ptiles + pl.otiles + s.ctas <= s.slots && together <= apart - apart / 8;
    if (pl.shared) {
      pl.ptiles = ptiles;
      pl.own0 = ptiles * (pl.nbp + kTileCost);
      pl.units = together;
    }
  }
  pl.chunk = s.div_ctas(max(1, pl.units) - 1) + 1;
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (!pl.shared && pl.otiles <= s.ctas && longest <= pl.chunk + kWholeExtra) {
    pl.whole = pl.chunk = max(1, longest);
    pl.units = pl.otiles * longest;
  }
  return pl;
}

// Whole warp: the item of CTA c that starts at unit u (u below `end`, its last one's successor), and
// the units `span` that it takes; nblk = 0 when those are a tile's cost only.
EC_DEV Item cta_item(const Shape& s, const Plan& pl, int u, int end, int c, int& span) {
  const int lane = threadIdx.x & 31;
  Item it;
  it.before = 0;
  if (u < pl.own0) {
    const int t = div_down(u, pl.nbp + kTileCost), per_head = s.div_h(pl.ptiles);
    it.b = -1;
    it.kvh = div_down(t, per_head);
    it.row0 = (t - it.kvh * per_head) * kBlockM;
    it.nrows = min(kBlockM, pl.rows - it.row0);
    it.np = it.blocks = pl.nbp;
    it.j0 = u - t * (pl.nbp + kTileCost);
    it.tile = t;
    it.len = 0;
  } else {
    int base = pl.own0, tbase = pl.ptiles, rsel = 0;
#pragma unroll 1
    for (int b0 = 0;; b0 += 32) {
      int32_t r, n;
      seq_of(s, pl, b0 + lane, r, n);
      const int t = s.Hkv * tiles_of(s, r), tu = tile_units(pl, tile_blocks(pl, n));
      int incl = t * tu, src = 0;
      if (s.B > 1) {
        incl = warp_inclusive(incl);
        const int total = __shfl_sync(0xffffffffu, incl, 31);
        const int nt = warp_total(t), nr = warp_total(r * s.g);
        if (u >= base + total && b0 + 32 < s.B) {
          base += total;
          tbase += nt;
          it.before += nr;
          continue;
        }
        src = __ffs(__ballot_sync(0xffffffffu, base + incl > u)) - 1;
        base += __shfl_sync(0xffffffffu, incl - t * tu, src);
        tbase += warp_total(lane < src ? t : 0);
        it.before += warp_total(lane < src ? r * s.g : 0);
      }
      rsel = __shfl_sync(0xffffffffu, r, src);
      it.len = __shfl_sync(0xffffffffu, n, src);
      it.b = b0 + src;
      break;
    }
    it.blocks = tile_blocks(pl, it.len);
    const int units = tile_units(pl, it.blocks);
    const int w = u - base, tl = div_down(w, units), per_head = tiles_of(s, rsel);
    it.kvh = per_head == 1 ? tl : div_down(tl, per_head);
    it.row0 = (tl - it.kvh * per_head) * kBlockM;
    it.nrows = min(kBlockM, rsel * s.g - it.row0);
    it.np = pl.shared ? 0 : pl.nbp;
    it.j0 = w - tl * units;
    it.tile = tbase + tl;
  }
  span = min(tile_units(pl, it.blocks) - it.j0, end - u);
  it.nblk = max(0, min(it.blocks - it.j0, span));
  // Partial rows. Shared: tile + c grows from item to item, so no two share a slot. Separate: a CTA
  // has at most two incomplete items, one that began before it and one that ends after it.
  it.slot = pl.shared ? it.tile + c : it.nblk == it.blocks ? -1 : 2 * c + (it.j0 == 0 ? 1 : 0);
  return it;
}

// The record of an item of CTA c that begins a cut tile of one sequence; u is the unit past the item.
// False for any other item.
EC_DEV bool tile_record(const Plan& pl, const Item& it, int u, int c, Record& rec) {
  if (it.slot < 0 || it.j0 != 0 || it.b < 0) return false;
  rec.b = it.b;
  rec.kvh = it.kvh;
  rec.row0 = it.row0;
  rec.nrows = it.nrows;
  rec.before = it.before;
  // the CTA that ends the tile: u is past this item and, if that is in here, the tile's cost
  const int last = it.nblk == it.blocks ? c : div_down(u + it.blocks - it.nblk - 1, pl.chunk);
  rec.a1 = it.slot;
  rec.a2 = pl.shared ? it.slot : 2 * (c + 1);
  rec.n2 = last - c + (pl.shared ? 1 : 0);
  return true;
}

// Whole warp, shared: the records of all tiles that begin in CTA c. For a CTA that gave up before it
// came to them: the merge reads the record of every tile, and one that no one wrote in this call would send
// it to rows and slots of whatever the workspace held before.
EC_DEV void write_records(const Shape& s, const Plan& pl, int c, Record* records) {
  const int end = min(pl.units, (c + 1) * pl.chunk);
#pragma unroll 1
  for (int u = min(pl.units, c * pl.chunk), span; u < end;) {
    const Item it = cta_item(s, pl, u, end, c, span);
    u += span;
    Record rec;
    if (it.nblk > 0 && tile_record(pl, it, u, c, rec) && (threadIdx.x & 31) == 0) records[it.tile - pl.ptiles] = rec;
  }
}

}  // namespace cached
}  // namespace ec
