// attention_cached.cu — attention of the recompute rows against caches that the other attention
// kernels do not read: an 8-bit K/V cache (quant_common.cuh), a prefix shared by the whole batch,
// and per-sequence key lengths; on the 5th-generation tensor cores.
//
// EntropyCache, gist.science zh summary §2.2 (the partial forward reads every row outside the
// recompute set from the cache) and pt summary §1 (bidirectional attention, no causal mask). With
// block-by-block decoding (pt §5, zh §5) a prompt's K/V do not depend on what follows it, so a batch
// behind one prompt holds them once. The 8-bit cache has no counterpart in the pages.
//   out[b, r, h] = sum_j softmax_j(scale <q[b, r, h], k_j>) v_j,  r < R[b], over the prefix's Lp
//   keys and the sequence's own kv_len[b] keys, KV head h / g;  zeros when there is no key
//
// Structure (one CTA per SM; the work plan is attention_cached.cuh's):
//   warps 0, 2   make the work plan and are the TMA producers, each for one of two streams (below): halves of
//                64 keys; warp 0 hands out the CTA's items to the others.
//   warps 1, 3   issue tcgen05.mma, each for one stream; warp 1 allocates 512 TMEM columns. (One
//                issuer for both: 102 us for 85 on the long 8-bit case, every wait and every product
//                of a stream in the other's way. Places in a ring worked out between the products:
//                205 us for 189 on the long shared prefix, so every half has a fixed place.)
//   warps 4..7   softmax of an item's even key blocks, warps 8..11 of the odd ones: two independent
//                streams with their own running maximum and sum and O accumulator, joined once per
//                item. A stream takes a block in two halves of 64 keys with an S buffer each: while one
//                half's softmax runs, the tensor cores do the other half's P V and the next block's
//                scores. (One S buffer of 128 keys: 4130 cycles a bf16 block, 2100 of them the
//                softmax, one thing after another. Scores of 128 keys in one product with the softmax in halves:
//                227 us for 184 on the long shared prefix.)
//                One TMEM lane (= one packed query row) per thread; online softmax in base 2 with a
//                lazy rescale of O (only when the running maximum grows by more than 2^8); P in
//                bf16 written back over the first half of the S buffer. Between an item's last softmax and
//                its join they fetch the next item's query tile, row by row (a tile packs rows of any
//                sequences, which no one tensor box covers; TMA gathers of four rows took 6000 cycles a tile).
//   warps 12..27 (8-bit cache) dequantise, four warps the K and four the V tiles of each stream: the
//                producers' TMA brings the codes into raw halves, and these warps write the bf16
//                halves that the products read. The dequantised values are exact in bf16, so the
//                products are those of a bf16 cache with the same values. (Raw tiles of 128 keys and
//                one producer: 93 us for 84 on the long 8-bit case, a tile's refill not under way before all
//                of it was read. Codes loaded from global memory into registers: 180 us for 120, as
//                the shared memory that the kernel takes leaves L1 little room for loads in flight.)
// What bounds an 8-bit call, past the smallest ones: shared memory's 128 bytes a cycle. A block of 128 keys
// moves 256 KB there (D = 128): the scores' operands 96 (a product of 64 keys reads all of Q), P V 32, the codes 32
// in and 32 out, the bf16 halves 64. Counters on the long shared prefix: 50% of those cycles loads and stores,
// 43% products' operands; 196 us, 0.94 PFLOP/s. The long 8-bit case: 82 us, 3.3 TB/s. (Q in tensor
// memory takes 64 KB off, but leaves room for one S buffer a stream beside it: 220 us for 184, 85 for 79.)
// A bf16 cache leaves every unit below half (8 x 32 rows of 32 heads behind 3840 keys: tensor pipe 23%, HBM 40%, L2
// 26%, issue slots 26%; an SM is active for 73% of the launch): the chain scores, softmax, P V of each block, and a
// call of a few blocks a CTA the chain plan, first loads, first scores, join, merge, straight-line code from a cold
// instruction cache.
//
// A waiter on an mbarrier sees a phase's parity only: it cannot tell a phase that is complete from one
// whose predecessor is still open. So whoever waits on a barrier follows every one of its phases, or has seen
// that the one before is complete: a place in shared memory belongs to one half of K or V of one stream.
// Such a place is free again when the product that read it is done (s_full, pv_done).
// Keys past a sequence's length may hold anything: their scores are replaced, and their V rows are
// zeroed in shared memory (0 x NaN is NaN in a matrix product).
// Partial items write fp32 rows, their maximum and their sum to the workspace; the merge kernel
// joins them in a fixed order, so results do not depend on timing.
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "attention_cached.cuh"
#include "ec_common.cuh"
#include "ec_internal.h"
#include "quant_common.cuh"

namespace ec {
namespace cached {
namespace {

constexpr uint32_t kTmemCols = 512;
constexpr int kHalf = 64;         // keys of an S buffer
constexpr uint32_t kTmemO = 256;  // stream s: S of half h at columns [128 s + 64 h, + 64), O at [256 + 128 s, + D)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.f;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per pipeline wait
constexpr int kMaxCtas = 160;                     // bound of the attention grid, for the workspace
constexpr int kMaxUnits = 8;                      // halves of K or V tiles in shared memory
constexpr int kMaxRaw = 8;                        // halves of raw tiles: K and V of each stream
constexpr int kDequantWarps = 4;                  // for K and for V of each stream
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = 32;  // rows of a tile per merge CTA
constexpr int kNarrow = 16;
constexpr int kMergeSteps = kBlockM / kMergeRows;
constexpr int kItems = 4;       // items handed out and not yet finished, see the producer
constexpr int kCum = 32;        // sequences whose row ends are kept in shared memory
constexpr uint32_t kDescHi = sdesc_hi(1024);
constexpr int kAtomBytes = 128 * 128;   // 128 rows x 128 bytes (64 bf16), 128-byte swizzle: the query tile
constexpr int kHalfAtom = kHalf * 128;  // 64 rows x 128 bytes: K and V
__host__ __device__ constexpr uint32_t step_k(int kk, int atom) { return (kk >> 2) * (atom / 16) + (kk & 3) * 2; }
constexpr uint32_t kStepPV = 16 * 128 / 16;

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t unit_full[kMaxUnits];  // a half is free when the product that reads it is done: s_full, pv_done
  uint64_t raw_full[kMaxRaw], raw_empty[kMaxRaw];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // of a stream's halves
  uint64_t join, o_free, v_here[2];  // v_here: a stream's V tile with rows to be zeroed has come
  uint64_t item_full[kItems], item_empty[kItems];
  uint32_t tmem_base;
  int abort;
};

// Shared memory: the query tile, for each stream the bf16 halves of one block's K and V, for
// the 8-bit cache their raw halves (64 rows of codes), the row statistics that the two streams exchange,
// the items, where each sequence's packed rows end, the barriers.
template <int D, bool Q8>
struct Layout {
  static constexpr int kAtoms = D / 64;
  static constexpr int kTileBytes = kAtoms * kAtomBytes;
  static constexpr int kHalfBytes = kAtoms * kHalfAtom;
  static constexpr int kUnits = 8, kPer = 4;  // bf16 half tiles: K's two and V's two of each stream
  static constexpr int kRaw = Q8 ? kMaxRaw : 0;
  static constexpr int kRawBytes = kHalf * D;
  static constexpr int kUnitOff = kTileBytes;
  static constexpr int kRawOff = kUnitOff + kUnits * kHalfBytes;
  static constexpr int kStatOff = kRawOff + kRaw * kRawBytes;
  static constexpr int kItemOff = kStatOff + 2 * kBlockM * static_cast<int>(sizeof(float2));
  static constexpr int kCumOff = kItemOff + kItems * static_cast<int>(sizeof(Item));
  static constexpr int kBarOff = kCumOff + kCum * 4;
  static constexpr int kBytes = kBarOff + static_cast<int>(sizeof(Bars));
  static constexpr int kThreads = Q8 ? 896 : 384;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct Args {
  CUtensorMap tk, tv, tpk, tpv;  // own and prefix caches
  const uint8_t *exps[2], *pexps[2];  // 8-bit: exponents of K and V, own and prefix
  Shape s;
  int32_t Hq, Ls, Lps;
  float scale_log2;
  const uint16_t* q;
  uint16_t* out;
  float4* part_o;     // [slots][D / 4][128]: four columns of a row, neighbouring rows side by side, or
                      // (a tile of kNarrow rows or fewer) [slots][128][D / 4], row by row
  float2* part_stat;  // [slots][128]: running maximum and sum
  Header* header;
  Record* records;    // [max(slots, ctas)]
  int32_t* dev_err;
};

EC_DEV void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
EC_DEV void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// One thread of a converged warp. The descriptors of tcgen05.mma live in uniform registers: behind
// this election, and with operands that a shuffle has made the same in all lanes, they are
// worked out there, while behind a branch on the lane number every one of them is moved over
// (1350 to 1600 cycles for eight products, against 650).
EC_DEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}

template <int N>
EC_DEV void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
EC_DEV void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

EC_DEV void st_shared16(uint32_t dst, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
EC_DEV uint4 ld_shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}
// tcgen05.wait::ld that also names the loaded registers, so that no use of them moves before it
// while other loads are in flight.
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

// Two fp32 lanes in one instruction.
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

// Whole warp: the sequence that packed row x over all sequences belongs to; x becomes the row within
// it. The sequence's number is that of the sequences that end at or before x.
EC_DEV int owner_of(const Shape& s, const int32_t* cum, int& x) {
  int b = 0, before = 0;
  if (s.B <= kCum) {
#pragma unroll 1
    for (int i = 0; i < s.B; ++i) {
      const int e = cum[i];
      if (e <= x) {
        b = i + 1;
        before = e;
      }
    }
  } else {
    const int lane = threadIdx.x & 31;
    int base = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < s.B; b0 += 32) {
      int32_t r, n;
      load_seq(s, b0 + lane, r, n, nullptr, false);
      const int incl = base + warp_inclusive(r * s.g);
#pragma unroll 1
      for (int i = 0; i < min(32, s.B - b0); ++i) {
        const int e = __shfl_sync(0xffffffffu, incl, i);
        if (e <= x) {
          b = b0 + i + 1;
          before = e;
        }
      }
      base = __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  x -= before;
  return b;
}

// Keys of block j of the item that take part.
EC_DEV int valid_keys(const Shape& s, const Item& it, int j) {
  const int left = j < it.np ? s.Lp - j * kBlockN : it.len - (j - it.np) * kBlockN;
  return max(0, min(kBlockN, left));
}

template <int D, bool Q8>
__global__ void __launch_bounds__(Layout<D, Q8>::kThreads, 1) cached_attention_kernel(const __grid_constant__ Args a) {
  using LY = Layout<D, Q8>;
  constexpr int kPer = LY::kPer;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bars = reinterpret_cast<Bars*>(smem + LY::kBarOff);
  const Shape& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0) {  // the lanes share the barriers
    if (lane < LY::kUnits) mbar_init(&bars->unit_full[lane], Q8 ? kDequantWarps : 1);
    if (lane < LY::kRaw) {
      mbar_init(&bars->raw_full[lane], 1);
      mbar_init(&bars->raw_empty[lane], kDequantWarps);
    }
    if (lane < 4) {
      mbar_init(&bars->s_full[lane >> 1][lane & 1], 1);
      mbar_init(&bars->p_full[lane >> 1][lane & 1], 4);
      mbar_init(&bars->pv_done[lane >> 1][lane & 1], 1);
    }
    if (lane < kItems) {
      mbar_init(&bars->item_full[lane], 1);
      mbar_init(&bars->item_empty[lane], Q8 ? 10 + 4 * kDequantWarps : 10);  // all that read the items
    }
    if (lane < 2) mbar_init(&bars->v_here[lane], 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 256);
    mbar_init(&bars->q_empty, 2);
    mbar_init(&bars->join, 8);
    mbar_init(&bars->o_free, 8);
    // the swizzled tiles need the 1024-byte alignment that dynamic shared memory has here
    bars->abort = (smem_u32(smem) & 1023u) != 0u;
    if (bars->abort) report_error(a.dev_err, EC_DEVERR_TIMEOUT);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&a.tk);
    prefetch_tmap(&a.tv);
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort;

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait_bounded(bar, parity, abort_flag, a.dev_err, kWaitLimitNs);
  };
  // The n-th item of this CTA, once the producer has made it; nblk = 0 at the end and after a wait
  // that gave up.
  Item* const items_s = reinterpret_cast<Item*>(smem + LY::kItemOff);
  auto next_item = [&](int n) {
    Item it;
    const bool ok = __all_sync(0xffffffffu, wait(&bars->item_full[n % kItems], (n / kItems) & 1));
    const uint32_t src = smem_u32(items_s + n % kItems);
    uint4* dst = reinterpret_cast<uint4*>(&it);
#pragma unroll
    for (int i = 0; i < 3; ++i) dst[i] = ld_shared16(src + 16 * i);
    if (!ok) it.nblk = 0;
    return it;
  };

  // Block j of the item has rows past the sequence's length (a map zero-fills only past the cache's end).
  auto ragged = [&](const Item& it, int j) { return j >= it.np && valid_keys(s, it, j) < kBlockN; };

  // With 28 warps a thread is launched with 72 registers; the softmax warps take 104, the others go
  // down: 128 x 64 + 256 x 104 + 512 x 56 is below 896 x 72. (With 48 the producers spill.)
  if (warp < 4) {
    if constexpr (Q8) setmaxnreg_dec<64>();
    if (warp == 0 || warp == 2) {
      // ------------------------------------------------------------------ plan, TMA producer of one stream
      // Both warps make the plan and walk the items; warp 0 hands them out.
      const int st = warp >> 1;
      pdl_wait();  // everything above overlaps the previous kernel
      const int cta = static_cast<int>(blockIdx.x);
      const Plan pl = make_plan(s, a.dev_err, cta == 0 && warp == 0);
      pdl_launch_dependents();
      const int u0 = min(pl.units, cta * pl.chunk), uend = *abort_flag ? u0 : min(pl.units, u0 + pl.chunk);
      if (warp == 0 && pl.shared && s.B <= kCum) {
        const int incl = warp_inclusive(pl.rows_l * s.g);
        if (lane < s.B) reinterpret_cast<int32_t*>(smem + LY::kCumOff)[lane] = incl;
        __syncwarp();
      }
      uint32_t c = 0;  // the stream's blocks
      int ok = 1, count = 0;
      Record rec{};
      for (int u = u0;; ++count) {
        Item it;
        it.nblk = 0;
        while (ok && it.nblk == 0 && u < uend) {
          int span;
          it = cta_item(s, pl, u, uend, cta, span);
          u += span;
        }
        if (warp == 0 && lane == 0) {
          if (!wait(&bars->item_empty[count % kItems], ((count / kItems) & 1) ^ 1)) it.nblk = 0;
          items_s[count % kItems] = it;
          mbar_arrive(&bars->item_full[count % kItems]);
        }
        it.nblk = __shfl_sync(0xffffffffu, it.nblk, 0);
        if (it.nblk == 0) break;
        if (tile_record(pl, it, u, cta, rec) && pl.shared && threadIdx.x == 0) a.records[it.tile - pl.ptiles] = rec;
        if (lane == 0) {
#pragma unroll 1
          for (int i = st; ok && i < it.nblk; i += 2, ++c) {
            const int j = it.j0 + i;
            const bool pre = j < it.np;
            const int key0 = (pre ? j : j - it.np) * kBlockN;
            const int b = pre ? 0 : it.b;
#pragma unroll 1
            for (int n = 0; n < 4; ++n) {
              // bf16: K's halves, then V's, as the products want them; 8-bit: the halves of both by turns,
              // as their warps dequantise them
              const int kv = Q8 ? n & 1 : n >> 1, h = Q8 ? n >> 1 : n & 1;
              const CUtensorMap* map = kv == 0 ? (pre ? &a.tpk : &a.tk) : (pre ? &a.tpv : &a.tv);
              if constexpr (Q8) {
                const int raw = 4 * st + 2 * kv + h;
                if (!(ok = wait(&bars->raw_empty[raw], (c & 1u) ^ 1u))) break;
                mbar_arrive_expect_tx(&bars->raw_full[raw], LY::kRawBytes);
                tma_load_4d(smem + LY::kRawOff + raw * LY::kRawBytes, map, &bars->raw_full[raw], 0, it.kvh,
                            key0 + h * kHalf, b);
              } else {
                const int slot = st * kPer + n;
                if (c != 0 && !(ok = wait(kv ? &bars->pv_done[st][h] : &bars->s_full[st][h], (c - 1) & 1u))) break;
                uint8_t* dst = smem + LY::kUnitOff + slot * LY::kHalfBytes;
                mbar_arrive_expect_tx(&bars->unit_full[slot], LY::kHalfBytes);
#pragma unroll
                for (int at = 0; at < LY::kAtoms; ++at)
                  tma_load_4d(dst + at * kHalfAtom, map, &bars->unit_full[slot], at * 64, it.kvh, key0 + h * kHalf, b);
              }
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      if (warp == 0 && pl.shared && __any_sync(0xffffffffu, *abort_flag != 0)) write_records(s, pl, cta, a.records);
      if (threadIdx.x == 0) {
        if (!pl.shared) a.records[cta] = rec;
        if (cta == 0) {
          Header h{};
          h.records = pl.shared ? pl.otiles : pl.whole != 0 ? 0 : s.ctas;
          h.shared = pl.shared;
          h.prefix_units = pl.nbp + kTileCost;
          h.nbp = pl.nbp;
          h.rows = pl.rows;
          h.chunk = pl.chunk;
          h.ptiles_head = s.div_h(pl.ptiles);
          *a.header = h;
        }
      }
    } else if (warp == 1 || warp == 3) {
      // ------------------------------------------------------------------ MMA issuer of one stream
      // The whole warp waits, one thread issues.
      constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kHalf, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 1);
      const uint32_t st = __shfl_sync(0xffffffffu, warp >> 1, 0);
      const uint32_t q_lo = sdesc_lo(smem_u32(smem), 16), unit0 = smem_u32(smem + LY::kUnitOff);
      const uint32_t tmem_u = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t s_col = tmem_u + st * kBlockN, o_col = tmem_u + kTmemO + st * 128;
      uint32_t used = 0;  // blocks of this stream whose P V is under way or done
      bool ok = true;
      auto wait_w = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
      uint64_t* const full = bars->unit_full + st * kPer;
      for (int items = 0; ok; ++items) {
        const Item it = next_item(items);
        if (it.nblk == 0) break;
        const int last = it.nblk - 2;  // block i is the stream's last one if i >= last
        // S of half h of the stream's block c (block i of the item)
        auto issue_qk = [&](int i, uint32_t c, int h) {
          // K is here, and the buffer's last P has been read
          if (!wait_w(full + h, c & 1u) || (c != 0 && !wait_w(&bars->pv_done[st][h], (c - 1) & 1u))) return false;
          tc_fence_after();
          const uint32_t k_lo = sdesc_lo(unit0 + (st * kPer + h) * LY::kHalfBytes, 16);
          const uint32_t col = s_col + h * kHalf;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_ss(col, q_lo + step_k(kk, kAtomBytes), k_lo + step_k(kk, kHalfAtom), kDescHi, idesc_qk, kk > 0 ? 1u : 0u);
            umma_commit(&bars->s_full[st][h]);
            if (h == 1 && i >= last) umma_commit(&bars->q_empty);  // the stream's last S of the item
          }
          __syncwarp();
          return true;
        };
        auto issue_pv = [&](int i, uint32_t c, int h) {
          if (!wait_w(full + 2 + h, c & 1u)) return false;
          if (!Q8 && i >= last && ragged(it, it.j0 + i) && lane == 0) mbar_arrive(&bars->v_here[st]);
          if (!wait_w(&bars->p_full[st][h], c & 1u)) return false;
          tc_fence_after();
          const uint32_t v_lo = sdesc_lo(unit0 + (st * kPer + 2 + h) * LY::kHalfBytes, kHalfAtom);
          const uint32_t col = s_col + h * kHalf;
          // the stream's first half of the item starts O anew
          const uint32_t acc0 = h > 0 ? 1u : __shfl_sync(0xffffffffu, i > 1 ? 1u : 0u, 0);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kHalf / 16; ++kk)
              umma_ts(o_col, col + kk * 8, v_lo + kk * kStepPV, kDescHi, idesc_pv, kk > 0 ? 1u : acc0);
            umma_commit(&bars->pv_done[st][h]);
          }
          __syncwarp();
          return true;
        };
        ok = wait_w(&bars->q_full, items & 1);
        if (static_cast<int>(st) < it.nblk) {
          ok = ok && issue_qk(st, used, 0) && issue_qk(st, used, 1);
          if (items > 0) ok = ok && wait_w(&bars->o_free, (items - 1) & 1);  // O is about to start anew
        } else {
          // Nothing of this item falls to stream 1. It leaves o_free alone: the item ends without this warp, so a
          // wait here could find the barrier a phase ahead. Its next one follows all the same: q_full of an
          // item comes after the join of the one before, and that after o_free of the second last.
          if (ok && lane == 0) mbar_arrive(&bars->q_empty);
        }
#pragma unroll 1
        for (int i = st; ok && i < it.nblk; i += 2, ++used) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && issue_pv(i, used, h);
            if (i < last) ok = ok && issue_qk(i + 2, used + 1, h);
          }
        }
        if (lane == 0) mbar_arrive(&bars->item_empty[items % kItems]);
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ softmax + epilogue
    if constexpr (Q8) setmaxnreg_inc<104>();
    const int st = (warp - 4) >> 2;            // stream
    const int row = 32 * (warp & 3) + lane;    // TMEM lane = packed query row
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    float2* stat = reinterpret_cast<float2*>(smem + LY::kStatOff);
    uint32_t used = 0, n_ragged = 0;    // blocks of this stream, and those with rows past a length
    bool ok = true;
    // An item's query tile, 16 rows a warp: each lane finds one row, and all fetch 16-byte pieces. The rows
    // behind the last one keep what lies there: a row's scores, weights and sums are its own, and no one
    // reads theirs. (With all 128 rows fetched, a one-row
    // tile's from one address: 12.9 us for 12.1 on a single-token call.)
    auto fetch_q = [&](const Item& q) {
      constexpr int kPieces = D / 8, kStep = 32 / kPieces;
      const int base = 16 * (warp - 4), piece = lane % kPieces;
      int x = q.row0 + min(base + (lane & 15), q.nrows - 1), b = q.b;
      if (b < 0) b = owner_of(s, reinterpret_cast<const int32_t*>(smem + LY::kCumOff), x);
      const int r = s.div_g(x);
      const int at = x + (b * s.L + r) * a.Hq + q.kvh * s.g - r * s.g;
#pragma unroll 4
      for (int i = lane / kPieces; i < 16; i += kStep) {
        const int64_t src = __shfl_sync(0xffffffffu, at, i);
        const int q_row = base + i;
        if (q_row < q.nrows)
          cp_async16(smem_u32(smem) + (piece >> 3) * kAtomBytes + q_row * 128 + (((piece & 7) ^ (q_row & 7)) << 4),
                     a.q + src * D + piece * 8);
      }
    };
    auto q_here = [&]() {
      cp_async_wait_all();
      fence_proxy_async_smem();
      mbar_arrive(&bars->q_full);
    };
    Item it = next_item(0);
    if (it.nblk > 0) {
      fetch_q(it);
      q_here();
    }
#pragma unroll 1
    for (int items = 0; it.nblk > 0; ++items) {
      const bool live = 32 * (warp & 3) < it.nrows;  // else the warp's rows are all padding
      float m_used = -INFINITY, l_sum = 0.f;
#pragma unroll 1
      for (int i = st; ok && i < it.nblk; i += 2, ++used) {
        const int j = it.j0 + i;
        // only the prefix's last block and the tile's are cut by a length
        const int keys = j + 1 == it.np || j + 1 == it.blocks ? valid_keys(s, it, j) : kBlockN;
        uint32_t s_addr = tmem + lane_off + st * kBlockN;
        int nv = keys;  // keys of the half that take part: none if 0 or less
#pragma unroll 1
        for (int h = 0; h < 2; ++h, s_addr += kHalf, nv -= kHalf) {
          ok = __all_sync(0xffffffffu, wait(&bars->s_full[st][h], used & 1u));
          if (!ok) break;
          if constexpr (!Q8) {
            if (keys < kBlockN && j >= it.np) {  // their V rows become zeros
              ok = __all_sync(0xffffffffu, wait(&bars->v_here[st], n_ragged++ & 1u));
              if (!ok) break;
              const uint32_t v_half = smem_u32(smem + LY::kUnitOff + (st * kPer + 2 + h) * LY::kHalfBytes);
              for (int e = max(nv, 0) * 8 + row; e < kHalf * 8; e += 128)
#pragma unroll
                for (int at = 0; at < LY::kAtoms; ++at) st_shared16(v_half + at * kHalfAtom + e * 16, make_uint4(0, 0, 0, 0));
              fence_proxy_async_smem();
            }
          }
          if (live) {
            tc_fence_after();
            // maximum (scale > 0 commutes with it), then p = 2^(s scale log2(e) - m)
            uint32_t b0[32], b1[32];
            EC_TMEM_LD32(s_addr, b0);
            EC_TMEM_LD32(s_addr + 32, b1);
            EC_TMEM_WAIT32(b0);
            EC_TMEM_WAIT32(b1);
            if (nv < kHalf) {  // keys that take no part
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                if (e >= nv) b0[e] = __float_as_uint(-INFINITY);
                if (32 + e >= nv) b1[e] = __float_as_uint(-INFINITY);
              }
            }
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              m4[e & 2] = max3(m4[e & 2], __uint_as_float(b0[e]), __uint_as_float(b0[e + 1]));
              m4[(e & 2) + 1] = max3(m4[(e & 2) + 1], __uint_as_float(b1[e]), __uint_as_float(b1[e + 1]));
            }
            const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale_log2;
            bool rescale = false;
            float alpha = 1.f;
            if (i < 2 && h == 0) {
              m_used = mx;
            } else if (mx > m_used + kRescaleLog2) {
              alpha = ex2_approx(m_used - mx);
              m_used = mx;
              l_sum *= alpha;
              rescale = true;
            }
            // without a finite score so far, nothing is subtracted and p = 0
            const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
            const uint64_t scale2 = pack_f32x2(a.scale_log2, a.scale_log2), neg_m2 = pack_f32x2(neg_m, neg_m);
            uint64_t sum2[2] = {0, 0};
            // P over the buffer's first 32 columns, in bf16 as the products take it: each weight is off by 2^-8 of
            // itself at most, as in the attention over a bf16 cache. Their sum is that of the fp32 weights.
            auto weights = [&](const uint32_t (&x)[32], int c) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float p0, p1;
                unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), scale2, neg_m2), p0, p1);
                p0 = ex2_approx(p0);
                p1 = ex2_approx(p1);
                sum2[(e >> 1) & 1] = add_f32x2(sum2[(e >> 1) & 1], pack_f32x2(p0, p1));
                pk[e >> 1] = pack_bf16x2(p0, p1);
              }
              EC_TMEM_ST16(s_addr + c, pk);
            };
            weights(b0, 0);
            weights(b1, 16);
            float sum_lo, sum_hi;
            unpack_f32x2(add_f32x2(sum2[0], sum2[1]), sum_lo, sum_hi);
            l_sum += sum_lo + sum_hi;
            if (__any_sync(0xffffffffu, rescale)) {
              // the half before this one may still be under way into O
              ok = __all_sync(0xffffffffu, wait(&bars->pv_done[st][h ^ 1], (h ? used : used - 1) & 1u));
              if (!ok) break;
              tc_fence_after();
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
            tmem_wait_st();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p_full[st][h]);
        }
      }
      // join the two streams: each warpgroup takes half of the columns of both accumulators
      const Item next = next_item(items + 1);
      if (next.nblk > 0) {
        ok = __all_sync(0xffffffffu, ok && wait(&bars->q_empty, items & 1));
        if (ok) fetch_q(next);
      }
      if (ok && st < it.nblk) ok = wait(&bars->pv_done[st][1], (used - 1) & 1u);
      // every warp is done with the item before, so its statistics may be overwritten
      if (ok && items > 0) ok = wait(&bars->o_free, (items - 1) & 1);
      stat[st * kBlockM + row] = make_float2(m_used, l_sum);
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&bars->join);
      ok = ok && wait(&bars->join, items & 1);
      if (next.nblk > 0) q_here();
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if (live) {
        const float2 s0 = stat[row], s1 = stat[kBlockM + row];
        const float M = fmaxf(s0.x, s1.x);
        // a stream without weight (no block, or no finite score) contributes nothing
        const bool has0 = s0.y != 0.f, has1 = it.nblk > 1 && s1.y != 0.f;
        const float w0 = has0 ? ex2_approx(s0.x - M) : 0.f, w1 = has1 ? ex2_approx(s1.x - M) : 0.f;
        const float L = (has0 ? w0 * s0.y : 0.f) + (has1 ? w1 * s1.y : 0.f);
        const bool complete = it.slot < 0;
        const float norm = complete ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
        const float f0 = w0 * norm, f1 = w1 * norm;
        const bool valid = row < it.nrows;
        uint16_t* orow = nullptr;
        float4* prow = nullptr;
        int pstep = 0;
        if (complete) {
          const int x = it.row0 + row, r = s.div_g(x);
          orow = a.out + static_cast<int64_t>((it.b * s.L + r) * a.Hq + it.kvh * s.g + (x - r * s.g)) * D + st * (D / 2);
        } else {
          const int at = it.slot * kBlockM + row;
          pstep = it.nrows <= kNarrow ? 1 : kBlockM;
          prow = a.part_o + static_cast<int64_t>(it.slot) * (kBlockM * (D / 4)) + st * (D / 8) * pstep +
                 row * (it.nrows <= kNarrow ? D / 4 : 1);
          if (st == 0 && valid) a.part_stat[at] = make_float2(M, L);
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
          if (valid && complete) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(orow + c * 32 + 8 * e) =
                  make_uint4(pack_bf16x2(y[8 * e], y[8 * e + 1]), pack_bf16x2(y[8 * e + 2], y[8 * e + 3]),
                             pack_bf16x2(y[8 * e + 4], y[8 * e + 5]), pack_bf16x2(y[8 * e + 6], y[8 * e + 7]));
          } else if (valid) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              prow[(c * 8 + e) * pstep] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          }
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars->o_free);
        mbar_arrive(&bars->item_empty[items % kItems]);
      }
      it = next;
    }
  } else if constexpr (Q8) {
    // ------------------------------------------------------------------ dequantisation
    setmaxnreg_dec<56>();
    // A thread takes a 16-code piece of a row per step: eight lanes read 128 neighbouring bytes, and the
    // 16-byte pieces of bf16 that they store fall into eight different bank groups: for D = 128
    // lanes 0..3 take the first half of row r and lanes 4..7 the second half of row r ^ 1, whose
    // swizzle differs in the lowest bit. A thread's rows differ by multiples of 8, so its places in
    // the swizzle are the same in all. Each lane loads the exponent byte of one of its warp's 32 rows.
    constexpr int kPieces = D / 16;            // 16-code pieces of a row = steps over the tile's rows
    constexpr int kRowsStep = 128 / kPieces;   // rows of a step
    constexpr int kRowsWarp = 32 / kPieces;    // of a warp
    const int kv = ((warp >> 2) & 1) ^ 1, st = warp >= 20, raw = 4 * st + 2 * kv, w4 = warp & 3, piece = lane % kPieces;
    const int sub = D == 128 ? (lane / kPieces) ^ (piece >> 2) : lane / kPieces;  // row of the warp's
    const int row0 = w4 * kRowsWarp + sub;
    const int exp_row = (lane / kRowsWarp) * kRowsStep + w4 * kRowsWarp + lane % kRowsWarp;
    const uint32_t src0 = smem_u32(smem + LY::kRawOff + raw * LY::kRawBytes) + row0 * D + piece * 16;
    const uint32_t dst_off = (piece >> 2) * kHalfAtom + row0 * 128 + ((((piece & 3) * 2) ^ (row0 & 7)) << 4);
    uint32_t c = 0;  // the stream's blocks
    bool ok = true;
    for (int items = 0; ok; ++items) {
      const Item it = next_item(items);
      if (it.nblk == 0) break;
      // the exponent of this lane's row, one of the stream's blocks ahead (past the cache's end: any)
      const uint8_t* ep = nullptr;
      int left = 0;  // positions from the lane's row to the cache's end
      auto exponent = [&](int j) {
        if (j < it.j0 + 2 || (j >= it.np && j < it.np + 2)) {
          const bool pre = j < it.np;
          const int key = (pre ? j : j - it.np) * kBlockN + exp_row, b = pre ? 0 : it.b;
          left = (pre ? s.Lp : s.L) - key;
          ep = (pre ? a.pexps : a.exps)[kv] + (static_cast<int64_t>(b) * s.Hkv + it.kvh) * (pre ? a.Lps : a.Ls) + key;
        } else {
          left -= 2 * kBlockN;
          ep += 2 * kBlockN;
        }
        return left > 0 ? static_cast<int>(__ldg(ep)) : kExpZeroByte;
      };
      int e_next = st < it.nblk ? exponent(it.j0 + st) : 0;
#pragma unroll 1
      for (int i = st; ok && i < it.nblk; i += 2, ++c) {
        const int nv = kv ? valid_keys(s, it, it.j0 + i) : kBlockN;
        const int e_here = e_next;
        if (i + 2 < it.nblk) e_next = exponent(it.j0 + i + 2);
        const uint32_t f_here = dequant_factor(e_here);
        const bool plain = nv == kBlockN && __all_sync(0xffffffffu, e_here <= kExpOneFactor);
#pragma unroll 1
        for (int h = 0; ok && h < 2; ++h) {
          const int slot = st * kPer + 2 * kv + h;
          ok = __all_sync(0xffffffffu, wait(&bars->raw_full[raw + h], c & 1u) &&
                                             (c == 0 || wait(kv ? &bars->pv_done[st][h] : &bars->s_full[st][h], (c - 1) & 1u)));
          if (!ok) break;
          uint32_t src = src0 + h * kHalf * D;
          uint32_t dst = smem_u32(smem + LY::kUnitOff + slot * LY::kHalfBytes) + dst_off;
          const int q0 = h * (kPieces / 2);
          bool done = false;
          if (plain) {
            uint32_t marks = 0;
            uint4 w = ld_shared16(src);
#pragma unroll
            for (int q = 0; q < kPieces / 2; ++q) {
              const uint4 here = w;
              if (q + 1 < kPieces / 2) w = ld_shared16(src + (q + 1) * kRowsStep * D);
              const uint32_t f = __shfl_sync(0xffffffffu, f_here, q0 * kRowsWarp + sub + q * kRowsWarp);
              uint4 lo, hi;
              dequantise4(here.x, f, lo.x, lo.y);
              dequantise4(here.y, f, lo.z, lo.w);
              dequantise4(here.z, f, hi.x, hi.y);
              dequantise4(here.w, f, hi.z, hi.w);
              st_shared16(dst + q * kRowsStep * 128, lo);
              st_shared16((dst ^ 16u) + q * kRowsStep * 128, hi);
              marks |= nan_marks(here.x) | nan_marks(here.y) | nan_marks(here.z) | nan_marks(here.w);
            }
            done = !__any_sync(0xffffffffu, (marks & kNaNMarks) != 0);
          }
          if (!done) {  // large exponents, NaN, V rows past the length (zeros, whatever lies there)
#pragma unroll 1
            for (int q = 0; q < kPieces / 2; ++q) {
              const uint4 here = ld_shared16(src);
              const DequantScale sc = dequant_scale(__shfl_sync(0xffffffffu, e_here, (q0 + q) * kRowsWarp + sub));
              uint4 lo, hi;
              dequantise4(here.x, sc, lo.x, lo.y);
              dequantise4(here.y, sc, lo.z, lo.w);
              dequantise4(here.z, sc, hi.x, hi.y);
              dequantise4(here.w, sc, hi.z, hi.w);
              if (row0 + (q0 + q) * kRowsStep >= nv) lo = hi = make_uint4(0, 0, 0, 0);
              st_shared16(dst, lo);
              st_shared16(dst ^ 16u, hi);
              src += kRowsStep * D;
              dst += kRowsStep * 128;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bars->raw_empty[raw + h]);
            mbar_arrive(&bars->unit_full[slot]);
          }
        }
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
}

// ---------------------------------------------------------------------------------- merge

// Joins the partial rows of split tiles by their log-sum-exp weights, in a fixed order. A CTA takes 32
// rows of one tile. Up to 8 partials: a lane a row and a warp D / 8 columns of it, as the partials
// lie, four partials in flight. More (few rows over a long cache): a warp takes one row's whole
// width, eight partials in flight; above 32, all eight warps take it, each every eighth partial.
// (A lane a row with 16 partials of 7 rows took 10 us longer, its loads one after another.) Two
// chains of loads (the record; statistics and rows) and the partials' bytes, which the attention
// kernel has just written (L2), are the whole cost.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) cached_merge_kernel(const __grid_constant__ Args a) {
  constexpr int kWarps = kMergeThreads / 32, kQuads = D / 4, kMine = kQuads / kWarps;  // float4 columns; a warp's
  __shared__ float red[kWarps][kQuads][4];
  __shared__ float2 red_stat[kWarps];
  const Shape& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  // the first rows of all tiles first: a tile of few rows has no work for the others, and two CTAs fit an SM
  const int per = gridDim.x / kMergeSteps, row0 = blockIdx.x / per * kMergeRows;  // per <= slots
  int which = blockIdx.x % per;
  const int4* rp = reinterpret_cast<const int4*>(a.records + which);
  int4 t0 = __ldcg(rp), t1 = __ldcg(rp + 1);  // b, kvh, row0, nrows; a1, a2, n2, before (if there is such a record)
  const int4 h = __ldcg(reinterpret_cast<const int4*>(a.header));       // records, shared, prefix units, chunk
  const int4 h2 = __ldcg(reinterpret_cast<const int4*>(a.header) + 1);  // ptiles_head, nbp, rows
  const bool shared = h.y != 0;
  for (bool first = true; which < h.x; which += per, first = false) {
    if (!first) {
      rp = reinterpret_cast<const int4*>(a.records + which);
      t0 = __ldcg(rp);
      t1 = __ldcg(rp + 1);
    }
    const int rows = min(kMergeRows, t0.w - row0);
    if (rows <= 0) continue;
    // the partials of a row: n1 slots from a1 on at `lane1`, then every `step2`-th from a2 on
    const int step2 = shared ? 1 : 2;
    const bool narrow2 = t0.w <= kNarrow;
    auto row_parts = [&](int row, int& a1, int& n1, int& lane1, bool& narrow1) {
      a1 = t1.x, n1 = 1, lane1 = row, narrow1 = narrow2;
      if (shared) {  // the row's prefix tile, and the CTAs that its blocks fell to
        const int gp = t1.w + t0.z + row, pt = t0.y * h2.x + (gp >> 7), pu = pt * h.z;
        const float inv = __fdividef(1.f, static_cast<float>(h.w));
        const int c0 = div_near(pu, h.w, inv);
        a1 = pt + c0;
        n1 = div_near(pu + h2.y - 1, h.w, inv) - c0 + 1;
        lane1 = gp & 127;
        narrow1 = h2.z - (gp & ~127) <= kNarrow;
      }
    };
    auto out_row = [&](int row) {
      const int x = t0.z + row, r = s.div_g(x);
      return a.out + static_cast<int64_t>((t0.x * s.L + r) * a.Hq + t0.y * s.g + (x - r * s.g)) * D;
    };
    int a1, n1, lane1;
    bool narrow1;
    row_parts(row0, a1, n1, lane1, narrow1);
    const int most = n1 + t1.z;
    if (most <= 8 && rows > 8) {
      const int row = row0 + min(lane, rows - 1);
      row_parts(row, a1, n1, lane1, narrow1);
      const int n = n1 + t1.z;
      auto at = [&](int i, int& slot, int& ln) {
        slot = i < n1 ? a1 + i : t1.y + (i - n1) * step2;
        ln = i < n1 ? lane1 : row;
      };
      float M = -INFINITY, Lsum = 0.f;
      float acc[4 * kMine] = {};
#pragma unroll 1
      for (int i0 = 0; i0 < n; i0 += 4) {
        float2 st[4];
        float4 x[4][kMine];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          int slot, ln;
          at(min(i0 + u, n - 1), slot, ln);
          st[u] = __ldcg(a.part_stat + slot * kBlockM + ln);
          const bool nw = min(i0 + u, n - 1) < n1 ? narrow1 : narrow2;
          const int qs = nw ? 1 : kBlockM;
          const float4* src = a.part_o + static_cast<int64_t>(slot) * (kBlockM * kQuads) + warp * kMine * qs + ln * (nw ? kQuads : 1);
#pragma unroll
          for (int q = 0; q < kMine; ++q) x[u][q] = __ldcg(src + q * qs);
          if (i0 + u >= n) st[u].y = 0.f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          // a partial without weight (no finite score) contributes nothing, whatever its row holds
          if (st[u].y == 0.f) continue;
          const float m = fmaxf(M, st[u].x), f = M == -INFINITY ? 0.f : ex2_approx(M - m), w = ex2_approx(st[u].x - m);
          M = m;
          Lsum = fmaf(w, st[u].y, Lsum * f);
#pragma unroll
          for (int q = 0; q < kMine; ++q) {
            acc[4 * q] = fmaf(w, x[u][q].x, acc[4 * q] * f);
            acc[4 * q + 1] = fmaf(w, x[u][q].y, acc[4 * q + 1] * f);
            acc[4 * q + 2] = fmaf(w, x[u][q].z, acc[4 * q + 2] * f);
            acc[4 * q + 3] = fmaf(w, x[u][q].w, acc[4 * q + 3] * f);
          }
        }
      }
      if (lane < rows) {
        const float inv = Lsum == 0.f ? 0.f : 1.f / Lsum;
        uint2* dst = reinterpret_cast<uint2*>(out_row(row) + warp * kMine * 4);
#pragma unroll
        for (int q = 0; q < kMine; ++q)
          dst[q] = make_uint2(pack_bf16x2(acc[4 * q] * inv, acc[4 * q + 1] * inv), pack_bf16x2(acc[4 * q + 2] * inv, acc[4 * q + 3] * inv));
      }
    } else {
      // lane q holds a row's columns [4 q, 4 q + 4) (D = 64: lanes past 15 repeat)
      const int quad = lane % kQuads;
      const bool together = most > 32;  // all warps on one row
#pragma unroll 1
      for (int row = row0 + (together ? 0 : warp); row < row0 + rows; row += together ? 1 : kWarps) {
        row_parts(row, a1, n1, lane1, narrow1);
        const int n = n1 + t1.z, step = together ? kWarps : 1;
        auto place = [&](int i, int& slot, int& ln) {
          slot = i < n1 ? a1 + i : t1.y + (i - n1) * step2;
          ln = i < n1 ? lane1 : row;
        };
        float acc[4] = {}, M = -INFINITY, Lsum = 0.f;
#pragma unroll 1
        for (int i0 = together ? warp : 0; i0 < n; i0 += 8 * step) {
          float2 st[8];
          float4 x[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            int slot, ln;
            place(min(i0 + u * step, n - 1), slot, ln);
            st[u] = __ldcg(a.part_stat + slot * kBlockM + ln);
            const bool nw = min(i0 + u * step, n - 1) < n1 ? narrow1 : narrow2;
            x[u] = __ldcg(a.part_o + static_cast<int64_t>(slot) * (kBlockM * kQuads) +
                          (nw ? ln * kQuads + quad : quad * kBlockM + ln));
            if (i0 + u * step >= n) st[u].y = 0.f;
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            if (st[u].y == 0.f) continue;
            const float m = fmaxf(M, st[u].x), f = M == -INFINITY ? 0.f : ex2_approx(M - m), w = ex2_approx(st[u].x - m);
            M = m;
            Lsum = fmaf(w, st[u].y, Lsum * f);
            acc[0] = fmaf(w, x[u].x, acc[0] * f);
            acc[1] = fmaf(w, x[u].y, acc[1] * f);
            acc[2] = fmaf(w, x[u].z, acc[2] * f);
            acc[3] = fmaf(w, x[u].w, acc[3] * f);
          }
        }
        if (together) {
          if (lane < kQuads) *reinterpret_cast<float4*>(red[warp][quad]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
          if (lane == 0) red_stat[warp] = make_float2(M, Lsum);
          __syncthreads();
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < kWarps; ++k)
            if (red_stat[k].y != 0.f) top = fmaxf(top, red_stat[k].x);
          Lsum = acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
#pragma unroll
          for (int k = 0; k < kWarps; ++k) {
            if (red_stat[k].y == 0.f) continue;
            const float w = ex2_approx(red_stat[k].x - top);
            Lsum = fmaf(w, red_stat[k].y, Lsum);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = fmaf(w, red[k][quad][e], acc[e]);
          }
          __syncthreads();
        }
        if (lane < kQuads && (!together || warp == 0)) {
          const float inv = Lsum == 0.f ? 0.f : 1.f / Lsum;
          reinterpret_cast<uint2*>(out_row(row))[quad] =
              make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------------- host

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// A cache [B, L, Hkv, D] in boxes of one head: bf16 in 64 positions by 64 swizzled elements, codes in 64
// whole unswizzled positions. Rows past L read as zeros.
bool cache_map(EncodeTiledFn enc, CUtensorMap* m, const void* base, bool q8, int D, int Hkv, int L, int B) {
  const cuuint64_t e = q8 ? 1 : 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hkv), static_cast<cuuint64_t>(L),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {e * D, e * D * Hkv, e * D * Hkv * L};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(q8 ? D : 64), 1, static_cast<cuuint32_t>(kHalf), 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
             strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             q8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
             // a head's row of codes is 128 bytes or less; with 256, 80.9 us for 79.3 on the long 8-bit case
             q8 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t part_slots(const ec_params& p, bool prefix) {
  const int64_t separate = 2 * kMaxCtas;
  if (!prefix) return separate;
  // A place of 128 rows for every tile at R = L, but for eight tiles per SM at most (85 MB at D = 128): a
  // workspace does not grow with the batch. With more tiles than places the prefix is not shared, and a
  // large batch of short tiles (36 sequences of 32 KV heads, one row each) pays for it: its tiles run over
  // the prefix one by one.
  const int64_t g = p.Hq / p.Hkv;
  const int64_t tiles = p.Hkv * ((p.B * (static_cast<int64_t>(p.L) * g) + kBlockM - 1) / kBlockM) +
                        static_cast<int64_t>(p.B) * p.Hkv * ((static_cast<int64_t>(p.L) * g + kBlockM - 1) / kBlockM);
  return std::max(separate, std::min<int64_t>(tiles + kMaxCtas, 8 * kMaxCtas));
}

template <int D, bool Q8>
cudaError_t launch_impl(const ec_params& p, Args& a, cudaStream_t s) {
  using LY = Layout<D, Q8>;
  cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(cached_attention_kernel<D, Q8>), LY::kBytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(cached_attention_kernel<D, Q8>, dim3(a.s.ctas), dim3(LY::kThreads), LY::kBytes, s, a);
  if (e != cudaSuccess) return e;
  // A merge CTA for each of as many tiles as there are SMs, or for twice as many where a shared prefix makes a
  // tile of every sequence and head and they are more (8 x 32 of them: 42.8 -> 41.4 us; where there are fewer, the
  // idle CTAs cost up to 0.8 us).
  const int rounds = a.s.Lp > 0 && static_cast<int64_t>(p.B) * p.Hkv > a.s.ctas ? 2 : 1;
  return launch_pdl(cached_merge_kernel<D>, dim3(rounds * kMergeSteps * a.s.ctas), dim3(kMergeThreads), 0, s, a);
}

}  // namespace
}  // namespace cached

size_t cached_attention_workspace_bytes(const ec_params& p, bool prefix) {
  return static_cast<size_t>(cached::part_slots(p, prefix)) *
             (cached::kBlockM * (static_cast<size_t>(p.D) * 4 + sizeof(float2)) + sizeof(cached::Record)) +
         sizeof(cached::Header);
}

cudaError_t launch_cached_attention(const ec_params& p, const void* q, const ec_kv* prefix, const ec_kv& cache,
                                    const int32_t* R, const int32_t* kv_len, float scale, void* out, void* ws,
                                    int32_t* dev_err, cudaStream_t s, ec_status* status) {
  using namespace cached;
  *status = EC_OK;
  EncodeTiledFn enc = get_encode_fn();
  if (enc == nullptr) {
    *status = EC_ERR_CUDA;
    return cudaErrorNotSupported;
  }
  const bool q8 = cache.dtype == EC_E4M3;
  const bool pre = prefix != nullptr && prefix->len > 0;
  int sms = 0;
  cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) {
    *status = EC_ERR_CUDA;
    return e;
  }
  Args a;
  if (!cache_map(enc, &a.tk, cache.k, q8, p.D, p.Hkv, p.L, p.B) || !cache_map(enc, &a.tv, cache.v, q8, p.D, p.Hkv, p.L, p.B) ||
      (pre && (!cache_map(enc, &a.tpk, prefix->k, q8, p.D, p.Hkv, prefix->len, 1) ||
               !cache_map(enc, &a.tpv, prefix->v, q8, p.D, p.Hkv, prefix->len, 1)))) {
    *status = EC_ERR_INVALID_ARG;
    return cudaErrorInvalidValue;
  }
  if (!pre) {  // not used
    a.tpk = a.tk;
    a.tpv = a.tv;
  }
  const ec_kv& pc = pre ? *prefix : cache;
  a.exps[0] = cache.k_exp;
  a.exps[1] = cache.v_exp;
  a.pexps[0] = pc.k_exp;
  a.pexps[1] = pc.v_exp;
  a.s.R = R;
  a.s.kv_len = kv_len;
  a.s.B = p.B;
  a.s.L = p.L;
  a.s.Lk = scope_hi(p);
  a.s.Lp = pre ? prefix->len : 0;
  a.s.Hkv = p.Hkv;
  a.s.g = p.Hq / p.Hkv;
  a.s.div_g.set(a.s.g);
  a.s.div_h.set(p.Hkv);
  a.s.div_ctas.set(std::min(sms, kMaxCtas));
  a.s.ctas = std::min(sms, kMaxCtas);
  a.s.slots = static_cast<int32_t>(part_slots(p, pre));
  a.Hq = p.Hq;
  a.Ls = static_cast<int32_t>(quant_exp_stride(p.L));
  a.Lps = static_cast<int32_t>(quant_exp_stride(pc.len));
  a.scale_log2 = scale * kLog2e;
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.part_o = static_cast<float4*>(ws);
  a.part_stat = reinterpret_cast<float2*>(a.part_o + static_cast<int64_t>(a.s.slots) * kBlockM * (p.D / 4));
  a.records = reinterpret_cast<Record*>(a.part_stat + static_cast<int64_t>(a.s.slots) * kBlockM);
  a.header = reinterpret_cast<Header*>(a.records + a.s.slots);  // slots >= ctas
  a.dev_err = dev_err;
  if (p.D == 128)
    e = q8 ? launch_impl<128, true>(p, a, s) : launch_impl<128, false>(p, a, s);
  else
    e = q8 ? launch_impl<64, true>(p, a, s) : launch_impl<64, false>(p, a, s);
  if (e != cudaSuccess) *status = EC_ERR_CUDA;
  return e;
}

}  // namespace ec
