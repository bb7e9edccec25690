// attention_paged_tiles.cu — attention over a paged K/V cache for more rows than a few: tiles of 128 packed query rows (a
// sequence's positions times the g query heads of a KV head) on the 5th-generation tensor cores.
//
//   out[x] = sum_j p_xj v_j / sum_j p_xj, p_xj = 2^(s_xj - m_x), s_xj = scale log2(e) <q_x, k_j>, m_x a running maximum
// Two streams run through a CTA, each with its issuer, its softmax warps, a score buffer of 128 keys and an O
// accumulator in tensor memory: while one stream is in its softmax, the tensor cores do the other's P V and next scores.
// The weights are handed over in two halves of 64 keys, so that P V of the first runs beside the exponentials of the
// second. Two forms:
//   - pair (a sequence may have more rows than a tile): a stream a tile, two tiles side by side on the same K/V, so that
//     a byte brought to shared memory feeds 256 rows;
//   - split (every sequence has one tile): the streams take the even and the odd key blocks of the tile and are
//     joined at the item's end.
// The streams take turns at the tensor cores, P V and next scores in one piece: left to themselves they
// fall into step, both in the softmax, then both at the tensor cores (4 full steps of 2048 rows, 28/4 heads, 210 us for 182).
// 4 such steps take 172 us now, 1390 TFLOP/s, a pair of blocks 3010 cycles. What bounds them: a stream's own chain, softmax 1690
// cycles (64 exponentials of a row take a lone warp 490, two warps of a scheduler 590 together), then 1330 until the next
// scores are there, of which P V and scores are 1000, as a wait takes 120 to 200 cycles also when it is over; and an item's end
// and begin, another 6000. Tried when they took 182: score buffers of 64 keys, two a stream (210 us: as many waits for half the product), one
// issuer for both streams (222 us), sixteen softmax warps (204 us, with 104 registers each), all 128 scores in registers (180 us, but 3 to
// 5% slower in the split form). An L2 prefetch of the next item's queries took 1.5 us off 172 and cost windows 3 of 398.
// For the 172 also tried: the weights of the first half in two quarters (177: a wait more), waits that poll (182), every fourth
// exponential by a polynomial of degree 3 (177: issue slots bind, not the exponentials' unit).
// Blocks are 128 keys, brought in by TMA: one box of 128 rows, or of a smaller page, from the page that the table
// names. The blocks of all items (sequence, group of tiles, KV head) stand in one line of
// which the CTAs, one an SM, take equal shares; an item cut between CTAs leaves fp32 partial rows, which a second
// launch joins in a fixed order. Where items are few, each goes to a cluster of up to eight CTAs
// instead, a CTA an equal part of its blocks, joined over distributed shared memory: one launch and no line (paged_choice.h).
// A window leaves only the blocks that a group's rows see between them.
// Roles (12 warps):
//   warp 0      plan, items, TMA producer        warps 4..7    softmax and epilogue of stream 0
//   warps 1, 2  issuers of the two streams       warps 8..11   of stream 1
//   warp 3      zeroes V rows that no row of the group may see (a page's rest may hold NaN, and 0 x NaN is NaN)
// A waiter on an mbarrier sees a phase's parity only, so whoever waits on a barrier follows every one of its
// phases or has seen by another way that the one before is complete.
#include <algorithm>
#include <type_traits>

#include "paged_common.cuh"

namespace ec {
namespace paged {
namespace {

constexpr int kThreads = 384;
constexpr int kBlockM = kTileRows;
constexpr int kBlockN = kStepKeys;
constexpr int kHalf = 64;  // keys whose weights are handed over at once
constexpr int kItems = 4;  // items handed out and not yet finished
// What the partial rows of cut items cost, in blocks, where the choice is whole items in the line: with 3, 8 x 95 rows of 28/4 heads behind
// 2048 keys 40.0 us for 37.5; with 8, 2048 rows of 28/4 heads 67.5 for 59.7.
constexpr int kCutCost = 5;
// An item takes a CTA two blocks' time beside its own, for the first scores, the last weights and O. In the line it counts so many units
// more, in front of its blocks: 16384 rows in windows, where the first groups see half as many blocks as the others, 409 us without and 401 so,
// 8 x 95 rows of 28/4 heads, ragged, 32.0 and 30.5; with three 31.8.
constexpr int kItemCost = 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 256;  // stream t: scores at columns [128 t, + 128), O at [256 + 128 t, + D)
constexpr uint32_t kDescHi = sdesc_hi(1024);
constexpr int kAtomBytes = 128 * 128;  // 128 rows x 128 bytes (64 bf16)
__host__ __device__ constexpr uint32_t step_k(int kk) { return (kk >> 2) * (kAtomBytes / 16) + (kk & 3) * 2; }
constexpr uint32_t kStepPV = 16 * 128 / 16;

// Work of a CTA on one (sequence, group of tiles, KV head): blocks v0 .. v0 + nblk - 1 of the group's; nblk 0: the end.
// part -1: the whole item; else the CTA's partial rows stand in its slots of an item that goes on here (0) or
// begins here (1).
struct __align__(16) Item {
  int b, kvh, nblk, v0, near_blocks, first, near, lo, hi, n, r0, rows0, rows1, part, pad[2];
};
static_assert(sizeof(Item) == 64, "four 16-byte pieces");

template <int P>
struct Bars {
  uint64_t q_full, q_empty;
  uint64_t unit_full[P], unit_empty[P];  // K or V of a block
  uint64_t v_ok[P];
  uint64_t s_full[2], p_full[2][2], pv_half[2], pv_done[2];  // [stream][half]
  uint64_t join, o_free, turn[2];
  uint64_t item_full[kItems], item_empty[kItems];
  uint32_t tmem_base;
  int abort;
  int scan[kThreads / 32], most[kThreads / 32];
  int begin[4], share;  // b, group, KV head, unit of the CTA's first item
};

template <int D, bool PAIR>
struct Layout {
  static constexpr int kAtoms = D / 64;
  static constexpr int kTileBytes = kAtoms * kAtomBytes;
  // Rings of places, K's and V's of the blocks in turn: one ring in the pair form; one for each stream in the split
  // form, as a waiter that does not follow every use of a place could take one use for another.
  static constexpr int kRings = PAIR ? 1 : 2;
  static constexpr int kRing = (PAIR ? 5 : 3) * (D == 128 ? 1 : 2);
  static constexpr int kPlaces = kRing * kRings;
  static constexpr int kUnitOff = (PAIR ? 2 : 1) * kTileBytes;
  static constexpr int kJoinPitch = D * 4 + 16;  // bytes of a row for a cluster's join, over the places: 8 rows fall to all banks
  static_assert(kPlaces * kTileBytes >= (PAIR ? 2 : 1) * kBlockM * kJoinPitch, "join");
  static constexpr int kStatOff = kUnitOff + kPlaces * kTileBytes;
  static constexpr int kItemOff = kStatOff + (PAIR ? 0 : 2 * kBlockM * 8);
  static constexpr int kBarOff = kItemOff + kItems * static_cast<int>(sizeof(Item));
  static constexpr int kBytes = kBarOff + static_cast<int>(sizeof(Bars<kPlaces>));
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

EC_DEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}

// tcgen05.wait::ld that names the loaded registers, so that no use of them moves before it.
#define EC_TMEM_WAIT32(r)                                                                                    \
  asm volatile("tcgen05.wait::ld.sync.aligned;"                                                              \
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),         \
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),     \
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]),  \
                 "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),  \
                 "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory")

#define EC_TMEM_ST16(taddr, r)                                                                              \
  asm volatile(                                                                                             \
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" \
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), \
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])          \
      : "memory")

EC_DEV uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
EC_DEV void unpack_f32x2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
EC_DEV uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
EC_DEV uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
EC_DEV uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
EC_DEV float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The rest of a wait that is not over at first sight.
EC_DEV bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* dev_err) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort, dev_err, kWaitLimitNs)) != 0;
}

// A group of tiles of a sequence: its positions (at most `step`), what they see, its blocks.
struct Group {
  int rows, n, blocks;
  Hull h;
  Blocks k;
};
EC_DEV Group load_group(const Shape& s, int b, int grp, int step, bool tell) {
  Group q;
  const int r0 = grp * step;  // below rows_max
  const int64_t first = s.windowed ? raw_position(s.at, b, r0) : 0;
  sizes_of(s, b, tell, q.rows, q.n);
  q.rows = min(step, q.rows - r0);
  q.h = q.rows > 0 ? hull_of(s, b, r0, r0 + q.rows, q.n, first) : Hull{0, 0, 0};
  q.k = blocks_of(q.h, 7);
  q.blocks = q.rows > 0 ? max(1, q.k.count) : 0;  // rows without a key are written too
  return q;
}

EC_DEV int units_of(const Group& g) { return g.blocks > 0 ? g.blocks + kItemCost : 0; }

// Keys j0 .. j0 + count - 1 are all of the hull, or some of them. (Rows past the last key have an empty one, lo = hi = n, that
// may lie inside a box.)
EC_DEV bool all_in(int near, int lo, int hi, int j0, int count) { return j0 + count <= near || (j0 >= lo && j0 + count <= hi); }
EC_DEV bool some_in(int near, int lo, int hi, int j0, int count) { return j0 < near || max(j0, lo) < min(j0 + count, hi); }

// Four lanes beside each other hold a row each, in four pieces of 16 bytes; after it lane q of them holds piece q of the
// four rows. A store of 16 bytes then goes to 64 together in each of 8 rows. (A piece of a row of its own from each lane: 178 us for 172 on
// 4 full steps of 2048 rows, 444 for 405 on 16384 rows in windows.)
EC_DEV void turn_quads(uint32_t (&w)[4][4], int lane) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & bit) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[i][e] : w[i | bit][e], bit);
        if (up) w[i][e] = got;
        else w[i | bit][e] = got;
      }
    }
  }
}

// CLUSTER: an item a cluster; else shares of the line.
template <int D, bool PAIR, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1) tiles_kernel(const __grid_constant__ Args a, int nr, int groups) {
  using LY = Layout<D, PAIR>;
  constexpr int kTiles = PAIR ? 2 : 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  auto* bars = reinterpret_cast<Bars<LY::kPlaces>*>(smem + LY::kBarOff);
  const Shape& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int step = nr * kTiles;  // positions of a group

  if (warp == 0) {  // the lanes share the barriers
    if (lane < LY::kPlaces) {
      mbar_init(&bars->unit_full[lane], 1);
      mbar_init(&bars->unit_empty[lane], kTiles + 1);  // released by the issuers that read it and by warp 3
      mbar_init(&bars->v_ok[lane], 1);
    }
    if (lane < 4) mbar_init(&bars->p_full[lane >> 1][lane & 1], 4);
    if (lane < 2) {
      mbar_init(&bars->s_full[lane], 1);
      mbar_init(&bars->pv_half[lane], 1);
      mbar_init(&bars->pv_done[lane], 1);
      mbar_init(&bars->turn[lane], 1);
    }
    if (lane < kItems) {
      mbar_init(&bars->item_full[lane], 1);
      mbar_init(&bars->item_empty[lane], 11);  // all that read the items
    }
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 2);
    mbar_init(&bars->join, 8);
    mbar_init(&bars->o_free, 8);
    bars->abort = (smem_u32(smem) & 1023u) != 0u;  // the swizzled tiles need the alignment that dynamic shared memory has here
    if (bars->abort) report_error(s.dev_err, EC_DEVERR_TIMEOUT);
    bars->begin[3] = -1;
    fence_mbar_init();
    prefetch_tmap(&a.tq);
    prefetch_tmap(&a.tk);
    prefetch_tmap(&a.tv);
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  prefetch_small(s, kThreads);
  pdl_wait();  // everything above overlaps the previous kernel
  pdl_launch_dependents();

  int share = 0, left = 0, place[4] = {0, 0, 0, 0};  // the CTA's first item: sequence, group, KV head, unit; units from there on
  bool whole = false;
  if constexpr (CLUSTER) {
    const int item = blockIdx.x / cluster_size(), pair = item / s.Hkv;
    place[0] = pair / groups, place[1] = pair % groups, place[2] = item % s.Hkv;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  } else {
    // The line: each thread adds up the blocks of its (sequence, group) pairs, the CTA their sum, and the thread whose pairs
    // hold the first block of this CTA's share finds it.
    const int pairs = s.B * groups, per = (pairs + kThreads - 1) / kThreads, p0 = threadIdx.x * per;
    int mine = 0, longest = 0;
#pragma unroll 2
    for (int i = p0; i < min(p0 + per, pairs); ++i) {
      const int b = i / groups, units = units_of(load_group(s, b, i - b * groups, step, blockIdx.x == 0));
      mine += units * s.Hkv;
      longest = max(longest, units);
    }
    int incl = warp_inclusive(mine);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 31) bars->scan[warp] = incl, bars->most[warp] = longest;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) incl += bars->scan[w];
      total += bars->scan[w];
      longest = max(longest, bars->most[w]);
    }
    share = (total + gridDim.x - 1) / gridDim.x;
    const int begin = blockIdx.x * share;
    // Whole items, each to the CTA whose share holds its first block, where that costs little more than the cuts' partial
    // rows do.
    whole = (share + longest - 1) / max(longest, 1) * longest <= share + kCutCost;
    if (begin < total && begin >= incl - mine && begin < incl) {
      int off = begin - (incl - mine);
      for (int i = p0;; ++i) {
        const int b = i / groups, units = units_of(load_group(s, b, i - b * groups, step, false));
        if (off < units * s.Hkv) {
          bars->begin[0] = b, bars->begin[1] = i - b * groups, bars->begin[2] = off / units, bars->begin[3] = off % units;
          break;
        }
        off -= units * s.Hkv;
      }
    }
    __syncthreads();
    left = bars->begin[3] >= 0 ? min(share, total - begin) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) place[i] = bars->begin[i];
  }
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort;
  auto wait_w = [&](uint64_t* bar, uint32_t parity) {  // whole warp
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return wait_on(bar, parity, &bars->abort, s.dev_err);
  };
  // The n-th item of this CTA, once the producer has made it; nblk = 0 at the end and after a wait that gave up.
  Item* const items_s = reinterpret_cast<Item*>(smem + LY::kItemOff);
  auto next_item = [&](int n) {
    Item it;
    const bool ok = wait_w(&bars->item_full[n % kItems], (n / kItems) & 1);
    const uint32_t src = smem_u32(items_s + n % kItems);
    uint4* dst = reinterpret_cast<uint4*>(&it);
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = ld_shared16(src + 16 * i);
    if (!ok) it.nblk = 0;
    return it;
  };
  // Place and use of K or V of a ring's next block.
  struct Place {
    uint32_t at, use;
    EC_DEV void next() {
      at += 2;
      if (at >= LY::kRing) at -= LY::kRing, ++use;
    }
  };
  auto ring_of = [](int i) { return PAIR ? 0 : i & 1; };  // of block i of an item
  auto block_of = [](const Item& it, int i) {
    const int v = it.v0 + i;
    return v < it.near_blocks ? v : v - it.near_blocks + it.first;
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ items and loads
    const int box = min(kBlockN, 1 << s.page_shift);   // rows of a TMA box
    const int boxes = kBlockN / box;                   // boxes of a block's rows: 1, 2, 4 or 8
    const int atoms = box < kBlockN ? LY::kAtoms : 1;  // boxes beside each other
    constexpr int kLead = CLUSTER ? 0 : kItemCost;
    int b = place[0], grp = place[1], kvh = place[2], u = place[3];
    Group g{};
    if constexpr (CLUSTER) {
      const int S = cluster_size(), rank = cluster_ctarank();
      g = load_group(s, b, grp, step, rank == 0 && kvh == 0 && grp == 0 && lane == 0);
      u = g.blocks * rank / S;
      left = g.blocks * (rank + 1) / S - u;
      if (lane == 0) bars->begin[0] = max(g.rows, 0), bars->begin[1] = left;
    } else {
      if (lane < kTiles) a.records[blockIdx.x * kTiles + lane].parts = 0;
      if (left > 0) g = load_group(s, b, grp, step, false);
    }
    if (*abort_flag) left = 0;
    auto next_group = [&]() {
      if (++kvh < s.Hkv) return;
      kvh = 0;
      do {
        if (++grp == groups) grp = 0, ++b;
        g = load_group(s, b, grp, step, false);
      } while (g.blocks == 0);
    };
    if (whole && u > 0) {  // an item of the CTA before
      left -= g.blocks + kLead - u;
      u = 0;
      if (left > 0) next_group();
    }
    Place k0{0, 0}, v0{1, 0}, k1{0, 0}, v1{1, 0};  // of the rings
    bool ok = true;
#pragma unroll 1
    for (int count = 0;; ++count) {
      Item it;
      const int size = g.blocks + kLead, take = whole ? size : min(size - u, left);
      it.v0 = max(u - kLead, 0);
      it.nblk = ok && left > 0 ? max(u + take - kLead, 0) - it.v0 : 0;  // 0, too, where the share ends before the item's first block
      if (it.nblk > 0) {
        it.b = b, it.kvh = kvh;
        it.near_blocks = g.k.near, it.first = g.k.first;
        it.near = g.h.near, it.lo = g.h.lo, it.hi = g.h.hi, it.n = g.n;
        it.r0 = grp * step, it.rows0 = min(nr, g.rows), it.rows1 = g.rows - it.rows0;
        it.part = it.nblk == g.blocks ? -1 : it.v0 == 0 ? 1 : 0;
      }
      ok = wait_w(&bars->item_empty[count % kItems], ((count / kItems) & 1) ^ 1);
      if (!ok) it.nblk = 0;
      if (lane == 0) {
        items_s[count % kItems] = it;
        mbar_arrive(&bars->item_full[count % kItems]);
      }
      if (it.nblk == 0) break;
      if (!CLUSTER && it.part == 1 && lane < kTiles) {  // the item begins here and goes on in the next CTAs
        const int rest = size - u - take;
        Record r{};
        r.rows = (lane == 0 ? it.rows0 : it.rows1) * s.g;
        r.parts = r.rows > 0 ? 1 + (rest + share - 1) / share : 0;
        r.b = b, r.kvh = kvh, r.row0 = (it.r0 + lane * nr) * s.g;
        a.records[blockIdx.x * kTiles + lane] = r;
      }
      // the queries, when the products of the item before have read theirs
      if (count > 0) ok = wait_w(&bars->q_empty, (count - 1) & 1);
      if (ok && lane == 0) {
        const int tiles = PAIR && it.rows1 > 0 ? 2 : 1;
        mbar_arrive_expect_tx(&bars->q_full, tiles * LY::kAtoms * nr * s.g * 128);
        for (int t = 0; t < tiles; ++t)
          for (int at = 0; at < LY::kAtoms; ++at)
            tma_load_5d(smem + t * LY::kTileBytes + at * kAtomBytes, &a.tq, &bars->q_full, at * 64, 0, kvh, it.r0 + t * nr, b);
      }
      // lane i: the page of the i-th box of a block's rows, one block ahead
      auto look = [&](int i) {
        const int j = block_of(it, i) * kBlockN + lane * box;
        return lane < boxes && some_in(it.near, it.lo, it.hi, j, box) ? page_of(s, b, j) : -1;
      };
      int next = look(0);
#pragma unroll 1
      for (int i = 0; ok && i < it.nblk; ++i) {
        const int page = next, j0 = block_of(it, i) * kBlockN;
        if (i + 1 < it.nblk) next = look(i + 1);
        const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
        const int ring = ring_of(i);
        const int r = lane % boxes, at = lane / boxes;
        const int pg = __shfl_sync(0xffffffffu, page, r);
#pragma unroll 1
        for (int n = 0; ok && n < 2; ++n) {
          const Place pl = n == 0 ? (ring == 0 ? k0 : k1) : ring == 0 ? v0 : v1;
          const int unit = ring * LY::kRing + pl.at;
          ok = wait_w(&bars->unit_empty[unit], (pl.use & 1u) ^ 1u);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&bars->unit_full[unit], __popc(have) * box * D * 2);
          __syncwarp();
          if (at < atoms && pg >= 0)
            tma_load_5d(smem + LY::kUnitOff + unit * LY::kTileBytes + at * kAtomBytes + r * box * 128, n == 0 ? &a.tk : &a.tv,
                        &bars->unit_full[unit], 0, (j0 + r * box) & ((1 << s.page_shift) - 1), at, kvh, pg);
        }
        if (ring == 0) k0.next(), v0.next();
        else k1.next(), v1.next();
      }
      left -= take;
      u = 0;
      if (CLUSTER) left = 0;
      if (left > 0) next_group();
    }
  } else if (warp <= 2) {
    // ------------------------------------------------------------------ issuer of one stream
    // The whole warp waits, one thread issues: the products' descriptors live in uniform registers.
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kBlockN, 0);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 1);
    const uint32_t st = __shfl_sync(0xffffffffu, warp - 1, 0);
    const uint32_t q_lo = sdesc_lo(smem_u32(smem) + (PAIR ? st * LY::kTileBytes : 0), 16), unit0 = smem_u32(smem + LY::kUnitOff);
    const uint32_t tmem_u = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t s_col = tmem_u + st * 128, o_col = tmem_u + kTmemO + st * 128;
    constexpr int kBy = PAIR ? 1 : 2;  // a stream takes every kBy-th block
    uint32_t used = 0;    // blocks of this stream whose P V is under way or done
    Place k{0, 0}, v{1, 0};  // of the next scores, of the next P V
    const uint32_t ring0 = PAIR ? 0 : st * LY::kRing;
    // Turns: a stream's P V and next scores go out in one piece, by turns with the other stream's.
    uint32_t turns = 0;
    auto my_turn = [&](bool by_turns) {
      if (!by_turns) return true;
      const uint32_t n = turns + st;  // stream 0's first turn waits for nothing
      return n == 0 || wait_w(&bars->turn[st], (n - 1) & 1u);
    };
    bool ok = true;
    for (int items = 0; ok; ++items) {
      const Item it = next_item(items);
      if (it.nblk == 0) break;
      const bool live = PAIR ? (st == 0 || it.rows1 > 0) : static_cast<int>(st) < it.nblk;
      const int i0 = PAIR ? 0 : st;
      const bool by_turns = !PAIR || it.rows1 > 0;  // else stream 0 is alone
      // A step of the stream: P V of block i (none before the first), then the scores of the block after it (none behind the
      // last). What can be waited for and worked out before the turn comes is.
      auto turn = [&](int i) {
        const bool weigh = i >= i0, more = i + kBy < it.nblk;
        const uint32_t v_unit = ring0 + v.at, k_unit = ring0 + k.at;
        const uint32_t v_lo = __shfl_sync(0xffffffffu, sdesc_lo(unit0 + v_unit * LY::kTileBytes, kAtomBytes), 0);
        const uint32_t k_lo = __shfl_sync(0xffffffffu, sdesc_lo(unit0 + k_unit * LY::kTileBytes, 16), 0);
        const uint32_t acc0 = __shfl_sync(0xffffffffu, i > i0 ? 1u : 0u, 0);
        if (more && !wait_w(&bars->unit_full[k_unit], k.use & 1u)) return false;
        if (weigh) {
          if (!wait_w(&bars->unit_full[v_unit], v.use & 1u)) return false;
          if (!all_in(it.near, it.lo, it.hi, block_of(it, i) * kBlockN, kBlockN) && !wait_w(&bars->v_ok[v_unit], v.use & 1u)) return false;
          if (!wait_w(&bars->p_full[st][1], used & 1u)) return false;
          // the item's first product starts O anew: the warps of both streams have read it
          if (!PAIR && items > 0 && i == i0 && !wait_w(&bars->o_free, (items - 1) & 1)) return false;
        }
        if (!my_turn(by_turns)) return false;
        tc_fence_after();
        if (weigh) {
#pragma unroll
          for (int h = 1; h >= 0; --h) {  // the half whose weights come first
            if (h == 0) {
              if (!wait_w(&bars->p_full[st][0], used & 1u)) return false;
              tc_fence_after();
            }
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kHalf / 16; ++kk)
                umma_ts(o_col, s_col + h * 64 + kk * 8, v_lo + (h * 4 + kk) * kStepPV, kDescHi, idesc_pv, h == 0 || kk > 0 ? 1u : acc0);
              umma_commit(h == 1 ? &bars->pv_half[st] : &bars->pv_done[st]);
              if (h == 0) umma_commit(&bars->unit_empty[v_unit]);
            }
            __syncwarp();
          }
          v.next();
          ++used;
        }
        if (more) {
          if (used != 0 && !wait_w(&bars->pv_done[st], (used - 1) & 1u)) return false;  // the buffer's last P has been read
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              umma_ss(s_col, q_lo + step_k(kk), k_lo + step_k(kk), kDescHi, idesc_qk, kk > 0 ? 1u : 0u);
              // the other stream's products may queue up behind these
              if (kk == D / 16 - 1 && by_turns) mbar_arrive(&bars->turn[st ^ 1]);
            }
            umma_commit(&bars->s_full[st]);
            umma_commit(&bars->unit_empty[k_unit]);
            if (i + 2 * kBy >= it.nblk) umma_commit(&bars->q_empty);  // the stream's last scores of the item
          }
          __syncwarp();
          k.next();
        } else if (by_turns && lane == 0) {
          mbar_arrive(&bars->turn[st ^ 1]);
        }
        turns += by_turns;
        return true;
      };
      ok = wait_w(&bars->q_full, items & 1);
      if (live) {
#pragma unroll 1
        for (int i = i0 - kBy; ok && i < it.nblk; i += kBy) ok = turn(i);
      } else {
        // Nothing of this item falls to the stream. (It leaves o_free alone: its next wait there comes after a P of its own,
        // and so after the join of this item, and that after the phase before.)
        if (lane == 0) mbar_arrive(&bars->q_empty);
        if constexpr (PAIR) {
#pragma unroll 1
          for (int i = 0; ok && i < it.nblk; ++i) {
#pragma unroll 1
            for (int n = 0; ok && n < 2; ++n) {
              const Place pl = n == 0 ? k : v;
              ok = wait_w(&bars->unit_full[pl.at], pl.use & 1u);
              if (ok && lane == 0) mbar_arrive(&bars->unit_empty[pl.at]);
            }
            k.next();
            v.next();
          }
        }
      }
      if (!PAIR && st == 1) {  // as many turns as stream 0, whose blocks may be one more
#pragma unroll 1
        for (int e = live ? it.nblk & 1 : 2; ok && e > 0; --e, ++turns) {
          ok = my_turn(true);
          if (ok && lane == 0) mbar_arrive(&bars->turn[0]);
        }
      }
      if (lane == 0) mbar_arrive(&bars->item_empty[items % kItems]);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------------ rows of V outside the hull
    Place k0{0, 0}, v0{1, 0}, k1{0, 0}, v1{1, 0};  // of the rings
    bool ok = true;
    for (int items = 0; ok; ++items) {
      const Item it = next_item(items);
      if (it.nblk == 0) break;
#pragma unroll 1
      for (int i = 0; ok && i < it.nblk; ++i) {
        const int j0 = block_of(it, i) * kBlockN;
        const int ring = ring_of(i);
#pragma unroll 1
        for (int n = 0; ok && n < 2; ++n) {
          const Place pl = n == 0 ? (ring == 0 ? k0 : k1) : ring == 0 ? v0 : v1;
          const int unit = ring * LY::kRing + pl.at;
          ok = wait_w(&bars->unit_full[unit], pl.use & 1u);
          if (!ok) break;
          if (n == 1 && !all_in(it.near, it.lo, it.hi, j0, kBlockN)) {
            const uint32_t base = smem_u32(smem + LY::kUnitOff) + unit * LY::kTileBytes;
#pragma unroll 1
            for (int r = lane >> 3; r < kBlockN; r += 4)  // eight lanes a row
              if (!some_in(it.near, it.lo, it.hi, j0 + r, 1))
#pragma unroll
                for (int at = 0; at < LY::kAtoms; ++at) st_shared16(base + at * kAtomBytes + r * 128 + (lane & 7) * 16, make_uint4(0, 0, 0, 0));
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) {
            mbar_arrive(&bars->v_ok[unit]);
            mbar_arrive(&bars->unit_empty[unit]);
          }
        }
        if (ring == 0) k0.next(), v0.next();
        else k1.next(), v1.next();
      }
      if (lane == 0) mbar_arrive(&bars->item_empty[items % kItems]);
    }
  } else {
    // ------------------------------------------------------------------ softmax and epilogue of one stream
    const int st = (warp - 4) >> 2;
    const int row = 32 * (warp & 3) + lane;  // TMEM lane = packed query row
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    float2* stat = reinterpret_cast<float2*>(smem + LY::kStatOff);
    constexpr int kBy = PAIR ? 1 : 2;
    const int i0 = PAIR ? 0 : st;
    uint32_t used = 0;  // blocks of this stream
    bool ok = true;
#pragma unroll 1
    for (int items = 0; ok; ++items) {
      const Item it = next_item(items);
      if (it.nblk == 0) break;
      const int rows = (PAIR && st ? it.rows1 : it.rows0) * s.g;  // packed rows of the tile
      const int r0 = it.r0 + (PAIR && st ? nr : 0);
      const bool live = 32 * (warp & 3) < rows;  // else the warp's rows are all padding
      const bool valid = row < rows;
      const int rl = s.by_g(row), r = r0 + rl;
      int r_lo = it.lo, r_hi = it.hi;  // what this row sees, beside the keys below near
      bool good = valid;
      if (s.windowed && valid) {
        const int64_t pos = raw_position(s.at, it.b, r);
        const int p = inside(pos, s.L) ? static_cast<int>(pos) : 0;
        r_lo = max(p - s.w.left, 0);
        r_hi = min(p + s.w.right + 1, it.n);
        // right, or not written: the row's keys are between those of the group's first and last row
        good = inside(pos, s.L) && min(r_lo, it.n) >= it.lo && r_hi <= it.hi;
        if (!good) {
          report_error(s.dev_err, EC_DEVERR_BAD_IDX);
          r_lo = r_hi = 0;
        }
      }
      float m_used = -INFINITY, l_sum = 0.f;
      if (!PAIR || rows > 0) {
#pragma unroll 1
        for (int i = i0; ok && i < it.nblk; i += kBy, ++used) {
          const int j = block_of(it, i) * kBlockN;
          const uint32_t s_addr = tmem + lane_off + st * 128;
          ok = wait_w(&bars->s_full[st], used & 1u);
          if (!ok) break;
          if (live) {
            tc_fence_after();
            // Two halves of 64 keys, the second first. P goes over the scores of its half, in bf16 as the products take it: each
            // weight is off by 2^-8 of itself at most. Their sum is that of the fp32 weights.
            const bool plain = __all_sync(0xffffffffu, !valid || all_in(it.near, r_lo, r_hi, j, kBlockN));
            const uint64_t scale2 = pack_f32x2(s.scale_log2, s.scale_log2);
            // (twice, with the masks and without: what is in the way of the plain blocks costs them 4%)
            auto halves = [&](auto masked) {
#pragma unroll 1
              for (int h = 1; h >= 0; --h) {
                if (masked && !__any_sync(0xffffffffu, valid && some_in(it.near, r_lo, r_hi, j + 64 * h, kHalf))) {
                  uint32_t none[16] = {};  // no row of the warp sees a key of the half
                  EC_TMEM_ST16(s_addr + 64 * h, none);
                  EC_TMEM_ST16(s_addr + 64 * h + 16, none);
                  tmem_wait_st();
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) mbar_arrive(&bars->p_full[st][h]);
                  continue;
                }
                uint32_t x[2][32];
                EC_TMEM_LD32(s_addr + 64 * h, x[0]);
                EC_TMEM_LD32(s_addr + 64 * h + 32, x[1]);
                EC_TMEM_WAIT32(x[0]);
                EC_TMEM_WAIT32(x[1]);
                if (masked) {  // keys that the row does not see
                  auto below = [](int y) { return y <= 0 ? 0u : y >= 32 ? ~0u : (1u << y) - 1u; };
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    const int jc = j + 64 * h + 32 * c;
                    const uint32_t see = below(it.near - jc) | (below(r_hi - jc) & ~below(r_lo - jc));
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                      if (!((see >> e) & 1u)) x[c][e] = __float_as_uint(-INFINITY);
                  }
                }
                // maximum (scale > 0 commutes with it), then p = 2^(s scale log2(e) - m)
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  m4[e & 2] = max3(m4[e & 2], __uint_as_float(x[0][e]), __uint_as_float(x[0][e + 1]));
                  m4[(e & 2) + 1] = max3(m4[(e & 2) + 1], __uint_as_float(x[1][e]), __uint_as_float(x[1][e + 1]));
                }
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * s.scale_log2;
                if (i == i0 && h == 1) {
                  m_used = mx;
                } else {
                  const bool rescale = mx > m_used + kRescaleLog2;
                  // (a row without a weight so far has zeros in O: a window's first half block may be all masked)
                  if (!__any_sync(0xffffffffu, rescale && (!masked || m_used != -INFINITY))) {
                    if (rescale) m_used = mx;
                  } else {
                    // O is at rest at a block's first half, as its scores came after the last P V; at its second half
                    // the first one's P V may be under way
                    if (h == 0) ok = wait_w(&bars->pv_half[st], used & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    const float alpha = rescale ? ex2_approx(m_used - mx) : 1.f;
                    if (rescale) m_used = mx;
                    l_sum *= alpha;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                      uint32_t o[32];
                      EC_TMEM_LD32(tmem + lane_off + kTmemO + st * 128 + c * 32, o);
                      EC_TMEM_WAIT32(o);
#pragma unroll
                      for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                      EC_TMEM_ST32(tmem + lane_off + kTmemO + st * 128 + c * 32, o);
                    }
                  }
                }
                // without a finite score so far, nothing is subtracted and p = 0
                const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
                const uint64_t neg_m2 = pack_f32x2(neg_m, neg_m);
                uint64_t sum2[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  uint32_t pk[16];
#pragma unroll
                  for (int e = 0; e < 32; e += 2) {
                    float p0, p1;
                    unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])), scale2, neg_m2), p0, p1);
                    p0 = ex2_approx(p0);
                    p1 = ex2_approx(p1);
                    sum2[(e >> 1) & 1] = add_f32x2(sum2[(e >> 1) & 1], pack_f32x2(p0, p1));
                    pk[e >> 1] = pack_bf16x2(p0, p1);
                  }
                  EC_TMEM_ST16(s_addr + 64 * h + 16 * c, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->p_full[st][h]);
                float sum_lo, sum_hi;
                unpack_f32x2(add_f32x2(sum2[0], sum2[1]), sum_lo, sum_hi);
                l_sum += sum_lo + sum_hi;
              }
            };
            if (plain) halves(std::false_type{});
            else halves(std::true_type{});
            if (!ok) break;
          } else if (lane == 0) {
            mbar_arrive(&bars->p_full[st][0]);
            mbar_arrive(&bars->p_full[st][1]);
          }
        }
        if (ok && (PAIR || st < it.nblk)) ok = wait_w(&bars->pv_done[st], (used - 1) & 1u);
      }
      const bool complete = !CLUSTER && it.part < 0;
      // slots of a CTA: [item goes on here, item begins here][tile]
      const int64_t slot = (static_cast<int64_t>(blockIdx.x) * 2 + (it.part > 0 ? 1 : 0)) * kTiles + (PAIR ? st : 0);
      // out's rows of the four lanes that trade pieces of their rows; -1: not written
      const int mine = good ? (it.b * s.rows_max + r) * s.Hq + it.kvh * s.g + (row - rl * s.g) : -1;
      int orow[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) orow[i] = __shfl_sync(0xffffffffu, mine, (lane & ~3) + i);
      // a slot is [D / 4][128] quads of columns, neighbouring rows side by side
      float4* const prow = reinterpret_cast<float4*>(a.part_o) + slot * (kBlockM * (D / 4)) + row;
      auto store = [&](const float (&y)[32], int col) {
        if (complete) {
          uint32_t w[4][4];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e >> 2][e & 3] = pack_bf16x2(y[2 * e], y[2 * e + 1]);
          turn_quads(w, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (orow[i] >= 0)
              *reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(orow[i]) * D + col + 8 * (lane & 3)) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
        } else if (CLUSTER && !complete) {
          const uint32_t dst = smem_u32(smem + LY::kUnitOff) + ((PAIR ? st * kBlockM : 0) + row) * LY::kJoinPitch + col * 4;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            st_shared16(dst + 16 * e, make_uint4(__float_as_uint(y[4 * e]), __float_as_uint(y[4 * e + 1]), __float_as_uint(y[4 * e + 2]), __float_as_uint(y[4 * e + 3])));
        } else if (!complete && valid) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            prow[(col / 4 + e) * kBlockM] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
        }
      };
      if constexpr (PAIR) {
        if constexpr (CLUSTER) {  // both streams are done with the places that the rows go to
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&bars->join);
          ok = ok && wait_w(&bars->join, items & 1);
        }
        if (!ok) break;
        tc_fence_after();
        if (live) {
          const float f = complete ? (l_sum == 0.f ? 0.f : 1.f / l_sum) : 1.f;
          if (!complete && valid) {
            const float2 mine = make_float2(good ? m_used : kNotWritten(), l_sum);
            if constexpr (CLUSTER) reinterpret_cast<float2*>(smem + st * LY::kTileBytes)[row] = mine;  // the queries have been read
            else a.part_stat[slot * kBlockM + row] = mine;
          }
          const bool empty = __any_sync(0xffffffffu, l_sum == 0.f);  // a row without a key, whose O may hold 0 x infinity
          const uint64_t f2 = pack_f32x2(f, f);
#pragma unroll 1
          for (int c = 0; c < D / 32; c += 2) {
            uint32_t o[2][32];
            EC_TMEM_LD32(tmem + lane_off + kTmemO + st * 128 + c * 32, o[0]);
            EC_TMEM_LD32(tmem + lane_off + kTmemO + st * 128 + c * 32 + 32, o[1]);
            EC_TMEM_WAIT32(o[0]);
            EC_TMEM_WAIT32(o[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float y[32];
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                unpack_f32x2(mul_f32x2(pack_f32x2(__uint_as_float(o[k][e]), __uint_as_float(o[k][e + 1])), f2), y[e], y[e + 1]);
              if (empty)
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = l_sum == 0.f ? 0.f : y[e];
              store(y, (c + k) * 32);
            }
          }
          tc_fence_before();
        }
        __syncwarp();
      } else {
        // join the two streams: each warpgroup takes half of the columns of both accumulators. Every warp is done with the
        // item before, so its statistics may be overwritten
        if (ok && items > 0) ok = wait_w(&bars->o_free, (items - 1) & 1);
        stat[st * kBlockM + row] = make_float2(m_used, l_sum);
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&bars->join);
        ok = ok && wait_w(&bars->join, items & 1);
        if (!ok) break;
        tc_fence_after();
        if (live) {
          const float2 s0 = stat[row], s1 = stat[kBlockM + row];
          const float M = fmaxf(s0.x, s1.x);
          // a stream without weight (no block, or no finite score) contributes nothing
          const bool has0 = s0.y != 0.f, has1 = it.nblk > 1 && s1.y != 0.f;
          const float w0 = has0 && s0.x != -INFINITY ? ex2_approx(s0.x - M) : has0 ? 1.f : 0.f;
          const float w1 = has1 && s1.x != -INFINITY ? ex2_approx(s1.x - M) : has1 ? 1.f : 0.f;
          const float L = (has0 ? w0 * s0.y : 0.f) + (has1 ? w1 * s1.y : 0.f);
          const float norm = complete ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
          const float f0 = w0 * norm, f1 = w1 * norm;
          if (!complete && st == 0 && valid) {
            const float2 mine = make_float2(good ? M : kNotWritten(), L);
            if constexpr (CLUSTER) reinterpret_cast<float2*>(smem)[row] = mine;  // the queries have been read
            else a.part_stat[slot * kBlockM + row] = mine;
          }
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c) {
            uint32_t o0[32], o1[32];
            EC_TMEM_LD32(tmem + lane_off + kTmemO + st * (D / 2) + c * 32, o0);
            EC_TMEM_LD32(tmem + lane_off + kTmemO + 128 + st * (D / 2) + c * 32, o1);
            EC_TMEM_WAIT32(o0);
            EC_TMEM_WAIT32(o1);
            float y[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              y[e] = has0 ? __uint_as_float(o0[e]) * f0 : 0.f;
              if (has1) y[e] = fmaf(__uint_as_float(o1[e]), f1, y[e]);
            }
            store(y, st * (D / 2) + c * 32);
          }
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->o_free);
      }
      if (lane == 0) mbar_arrive(&bars->item_empty[items % kItems]);
    }
  }

  // ---------------------------------------------------------------------- teardown
  if (*abort_flag) {  // copies and products may still be under way: they take microseconds
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 200000u) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if constexpr (CLUSTER) {
    // the cluster's CTAs share out the tile's rows and read all parts of theirs
    const int S = cluster_size(), rank = cluster_ctarank(), rows = bars->begin[0];
    const int rows0 = min(rows, nr) * s.g, packed = rows * s.g;  // of tile 0, of both
    if (bars->begin[1] == 0)
      for (int i = threadIdx.x; i < kTiles * kBlockM; i += kThreads)
        reinterpret_cast<float2*>(smem + i / kBlockM * LY::kTileBytes)[i % kBlockM] = make_float2(-INFINITY, 0.f);
    cluster_arrive_release();
    cluster_wait_acquire();
    const int x0 = packed * rank / S, n = (packed * (rank + 1) / S - x0) * (D / 4);
#pragma unroll 1
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int xx = x0 + i / (D / 4), c = i % (D / 4) * 4, t = PAIR && xx >= rows0, x = t ? xx - rows0 : xx;
      float2 st[kMaxCluster];
      float4 z[kMaxCluster];
      float top = -INFINITY, sum = 0.f;
      bool lost = false;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        st[r] = make_float2(-INFINITY, 0.f);
        z[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < S) {
          st[r] = ld_dsmem8(dsmem_map(smem_u32(smem) + t * LY::kTileBytes + x * 8, r));
          z[r] = ld_dsmem16(dsmem_map(smem_u32(smem + LY::kUnitOff) + (t * kBlockM + x) * LY::kJoinPitch + c * 4, r));
        }
      }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        top = fmaxf(top, st[r].x);
        lost = lost || st[r].x != st[r].x;
      }
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        if (st[r].y == 0.f) continue;  // no weight; of a CTA without a block its rows hold anything
        const float f = st[r].x == -INFINITY ? 1.f : ex2_approx(st[r].x - top);
        sum += f * st[r].y;
        o.x += f * z[r].x, o.y += f * z[r].y, o.z += f * z[r].z, o.w += f * z[r].w;
      }
      if (lost) continue;
      const int rl = s.by_g(x), r = place[1] * step + t * nr + rl;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      uint2* dst = reinterpret_cast<uint2*>(
          a.out + ((static_cast<int64_t>(place[0]) * s.rows_max + r) * s.Hq + place[2] * s.g + (x - rl * s.g)) * D + c);
      *dst = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    }
    cluster_arrive_release();  // no CTA leaves while another one reads its rows
    cluster_wait_acquire();
  }
}

template <int D, bool PAIR, bool CLUSTER>
cudaError_t launch(const Args& a, int nr, int groups, int ctas, int cluster, cudaStream_t s) {
  constexpr int kBytes = Layout<D, PAIR>::kBytes;
  if constexpr (CLUSTER)
    return launch_pdl_cluster(tiles_kernel<D, PAIR, CLUSTER>, dim3(a.s.B * a.s.Hkv * groups * cluster), dim3(kThreads), kBytes, cluster, s, a, nr, groups);
  return launch_pdl(tiles_kernel<D, PAIR, CLUSTER>, dim3(ctas), dim3(kThreads), kBytes, s, a, nr, groups);
}

}  // namespace

cudaError_t setup_tiles() {
  cudaError_t e = cudaSuccess;
  auto allow = [&](const void* f, int bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  allow(reinterpret_cast<const void*>(tiles_kernel<64, false, false>), Layout<64, false>::kBytes);
  allow(reinterpret_cast<const void*>(tiles_kernel<64, false, true>), Layout<64, false>::kBytes);
  allow(reinterpret_cast<const void*>(tiles_kernel<64, true, false>), Layout<64, true>::kBytes);
  allow(reinterpret_cast<const void*>(tiles_kernel<64, true, true>), Layout<64, true>::kBytes);
  allow(reinterpret_cast<const void*>(tiles_kernel<128, false, false>), Layout<128, false>::kBytes);
  allow(reinterpret_cast<const void*>(tiles_kernel<128, false, true>), Layout<128, false>::kBytes);
  allow(reinterpret_cast<const void*>(tiles_kernel<128, true, false>), Layout<128, true>::kBytes);
  allow(reinterpret_cast<const void*>(tiles_kernel<128, true, true>), Layout<128, true>::kBytes);
  return e;
}

template <int D>
static cudaError_t launch_any(const Args& a, int nr, int ctas, int cluster, cudaStream_t s) {
  const int groups = ((a.s.rows_max + nr - 1) / nr + 1) / 2;
  if (a.s.rows_max > nr)
    return cluster ? launch<D, true, true>(a, nr, groups, 0, cluster, s) : launch<D, true, false>(a, nr, groups, ctas, 0, s);
  return cluster ? launch<D, false, true>(a, nr, 1, 0, cluster, s) : launch<D, false, false>(a, nr, 1, ctas, 0, s);
}

cudaError_t launch_tiles(const Args& a, int D, int nr, int ctas, int cluster, cudaStream_t s) {
  return D == 64 ? launch_any<64>(a, nr, ctas, cluster, s) : launch_any<128>(a, nr, ctas, cluster, s);
}

}  // namespace paged
}  // namespace ec
