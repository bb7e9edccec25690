// The work plan of the cached attentions (attention_cached.cuh) on the CPU: the items of every CTA cover
// every block of every tile once, partial rows have places of their own, and the merge finds a
// record of every cut tile, also when a CTA gave up before it handed anything out.
//   stdin: B L Lk Lp Hkv g ctas slots has_len, then R[B] and, with has_len, kv_len[B]
//   argv[1] "lost": the records of a CTA that gave up are left out
//   prints the mode (separate, shared, whole), the tiles and the units
#include <cstdio>
#include <cstring>
#include <iostream>
#include <map>
#include <string>

#include "host_warp.h"

#include "attention_cached.cuh"

using namespace ec::cached;

namespace {

int fail(const char* what, long long a = 0, long long b = 0) {
  std::printf("%s %lld %lld\n", what, a, b);
  return 1;
}

bool same(const Record& a, const Record& b) { return std::memcmp(&a, &b, sizeof a) == 0; }

struct Cover {
  int32_t b, kvh, row0, nrows, blocks, len;
  std::vector<int> seen;
  std::vector<int32_t> slots;  // of its items, in order
};

}  // namespace

int main(int argc, char** argv) {
  const bool lost = argc > 1 && std::strcmp(argv[1], "lost") == 0;
  Shape s{};
  int has_len = 0;
  std::cin >> s.B >> s.L >> s.Lk >> s.Lp >> s.Hkv >> s.g >> s.ctas >> s.slots >> has_len;
  std::vector<int32_t> R(s.B), len(s.B);
  for (auto& x : R) std::cin >> x;
  if (has_len)
    for (auto& x : len) std::cin >> x;
  s.R = R.data();
  s.kv_len = has_len ? len.data() : nullptr;
  s.div_g.set(s.g);
  s.div_h.set(s.Hkv);
  s.div_ctas.set(s.ctas);

  Plan plan{};
  std::map<int, Cover> tiles;
  std::map<int32_t, int> places;  // slot -> the tile whose partial rows it holds
  const Record none{-7, -7, -7, -7, -7, -7, -7, -7};
  std::vector<Record> handed(std::max(s.slots, s.ctas), none), rewritten(handed);
  int32_t err = 0;
  int bad = 0;
  host_warp::warp([&](int lane) {
    const Plan pl = make_plan(s, &err, true);
    if (lane == 0) plan = pl;
    for (int c = 0; c < s.ctas; ++c) {
      const int end = min(pl.units, (c + 1) * pl.chunk);
      Record rec{};
      for (int u = min(pl.units, c * pl.chunk), span; u < end;) {
        const Item it = cta_item(s, pl, u, end, c, span);
        u += span;
        if (lane != 0 || it.nblk == 0) continue;
        if (span <= 0 || it.j0 < 0 || it.j0 + it.nblk > it.blocks || it.nrows < 1 || it.nrows > kBlockM) bad |= 1;
        auto [at, fresh] = tiles.try_emplace(it.tile, Cover{it.b, it.kvh, it.row0, it.nrows, it.blocks, it.len, {}, {}});
        Cover& t = at->second;
        if (fresh) t.seen.assign(it.blocks, 0);
        if (t.b != it.b || t.kvh != it.kvh || t.row0 != it.row0 || t.nrows != it.nrows || t.blocks != it.blocks) bad |= 2;
        for (int j = it.j0; j < it.j0 + it.nblk && j < t.blocks; ++j) ++t.seen[j];
        if (it.slot >= 0 && (it.slot >= s.slots || !places.emplace(it.slot, it.tile).second)) bad |= 4;
        t.slots.push_back(it.slot);
        if (tile_record(pl, it, u, c, rec) && pl.shared) handed[it.tile - pl.ptiles] = rec;
      }
      if (lane == 0 && !pl.shared) handed[c] = rec;
      if (pl.shared && !lost) write_records(s, pl, c, rewritten.data());
    }
  });
  if (bad) return fail("bad item", bad);

  // every row of every sequence and head, and every key block, once
  int expect = 0;
  if (plan.shared) expect += s.Hkv * ((plan.rows + kBlockM - 1) / kBlockM);
  for (int b = 0; b < s.B; ++b) {
    const bool ok = R[b] >= 0 && R[b] <= s.L && (!has_len || (len[b] >= 0 && len[b] <= s.L));
    if (ok) expect += s.Hkv * tiles_of(s, R[b]);
  }
  if (static_cast<int>(tiles.size()) != expect) return fail("tiles", tiles.size(), expect);
  std::map<std::pair<int, int>, std::map<int, int>> rows;  // (b, head) -> first row -> rows
  for (auto& [n, t] : tiles) {
    for (int x : t.seen)
      if (x != 1) return fail("blocks of tile", n, x);
    if (!rows[{t.b, t.kvh}].emplace(t.row0, t.nrows).second) return fail("rows twice in tile", n);
  }
  for (auto& [who, m] : rows) {
    int next = 0;
    for (auto& [r0, n] : m) {
      if (r0 != next) return fail("rows of", who.first, who.second);
      next = r0 + n;
    }
    if (next != (who.first < 0 ? plan.rows : R[who.first] * s.g)) return fail("row count of", who.first, who.second);
  }

  // what the merge reads
  auto matches = [&](const Record& r, const Cover& t) {
    if (r.b != t.b || r.kvh != t.kvh || r.row0 != t.row0 || r.nrows != t.nrows) return false;
    std::vector<int32_t> want;
    if (!plan.shared) want.push_back(r.a1);
    for (int i = 0; i < r.n2; ++i) want.push_back(r.a2 + i * (plan.shared ? 1 : 2));
    return want == t.slots;
  };
  if (plan.shared) {
    for (int i = 0; i < plan.otiles; ++i) {
      if (!matches(handed[i], tiles.at(plan.ptiles + i))) return fail("record of tile", plan.ptiles + i);
      if (!same(handed[i], rewritten[i])) return fail("no record after giving up: tile", plan.ptiles + i);
    }
  } else if (plan.whole == 0) {
    std::map<int, int> recs;
    for (int c = 0; c < s.ctas; ++c)
      if (handed[c].nrows > 0) ++recs[c];
    size_t cut = 0;
    for (auto& [n, t] : tiles) {
      if (t.slots.size() == 1 && t.slots[0] == -1) continue;
      ++cut;
      const int c = t.slots[0] / 2;
      if (c >= s.ctas || !matches(handed[c], t)) return fail("record of cut tile", n, c);
    }
    if (cut != recs.size()) return fail("records", recs.size(), cut);
  }
  std::printf("%s %d %d %d\n", plan.shared ? "shared" : plan.whole ? "whole" : "separate", plan.ptiles, plan.otiles, plan.units);
  return 0;
}
