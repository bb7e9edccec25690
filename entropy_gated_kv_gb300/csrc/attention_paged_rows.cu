// attention_paged_rows.cu — attention over a paged K/V cache for few rows: single tokens and short blocks, at most 16
// packed rows (a sequence's positions times the g query heads of a KV head).
//
//   out[x] = sum_j p_xj v_j / sum_j p_xj, p_xj = 2^(s_xj - m_x), s_xj = scale log2(e) <q_x, k_j>, m_x a running maximum
// A cache byte is used for two products a row, so HBM bounds the call, and for short caches the chain of
// sizes, page numbers, first keys, join. Hence:
//   - Warps work by themselves: a chunk of 16 keys (inside one page, as pages are multiples of 16) is one TMA
//     box for K and one for V in the warp's own ring; scores, softmax and P V of it stay in the warp's
//     registers (mma.sync m16n8k16: with 16 rows a tensor-memory tile would be an eighth full and every block would
//     pass through other warps). No barrier of the CTA until an item ends.
//   - The chunks of all items (sequence, KV head) stand in one line, eight to a unit, and the CTAs, one an SM,
//     take equal shares of it: long and short sequences load the SMs alike. An item cut between CTAs leaves
//     fp32 partial rows, which a second launch joins.
//   - Where the items are few, each goes to a cluster of up to eight CTAs instead, a CTA an equal part of its chunks, joined
//     over distributed shared memory: one launch and no line; paged_choice.h has the rule. (One token, 28/4 heads, 2047
//     keys: 8.9 us in shares of the line, 7.4 in clusters; 16 tokens with a window of 1024: 18.7 and 12.4.)
//   - A window leaves the chunks of its keys and of the sinks, nothing else is read.
#include <algorithm>

#include "paged_common.cuh"

namespace ec {
namespace paged {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 16;  // keys of a warp's step
constexpr int kChunkShift = 4;
static_assert(kChunk * kWarps == kStepKeys);

// A CTA's place in the line: unit u of item (b, kvh), `left` units of the share from there on.
struct Place {
  int b, kvh, u, left;
};

struct Misc {
  int scan[kWarps];
  Place begin;
  int share, abort;
  float2 stat[kFewRows];  // of the CTA's rows, for its cluster
};

template <int D>
struct Layout {
  static constexpr int kKBytes = kChunk * D * 2;  // a K or V chunk: [D / 64][16][64], 128-byte swizzle
  static constexpr int kStage = 2 * kKBytes;
  static constexpr int kStages = D == 64 ? 5 : 3;  // chunks in flight a warp
  static constexpr int kRows = kFewRows;
  static constexpr int kPitch = D + 4;  // floats of a row in the join's buffers: two rows in 8 share a bank
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kJoinOff = kRing;
  static constexpr int kStatOff = kJoinOff + kWarps / 2 * kRows * kPitch * 4;
  static constexpr int kBarOff = kStatOff + kWarps * kRows * 8;
  static constexpr int kMiscOff = kBarOff + kWarps * kStages * 8;
  static constexpr int kBytes = kMiscOff + static_cast<int>(sizeof(Misc));
  static_assert(kBytes <= 227 * 1024 && kRing >= kWarps / 2 * kRows * kPitch * 4, "shared memory");
};

// A sequence in the line: its chunks, and what its rows see.
struct Seq {
  int rows, n, chunks, units;
  Hull h;
  Blocks k;
};

EC_DEV Seq load_seq(const Shape& s, int b, bool tell) {
  Seq q;
  const int64_t first = s.windowed ? raw_position(s.at, b, 0) : 0;
  sizes_of(s, b, tell, q.rows, q.n);
  q.h = q.rows > 0 ? hull_of(s, b, 0, q.rows, q.n, first) : Hull{0, 0, 0};
  q.k = blocks_of(q.h, kChunkShift);
  q.chunks = q.k.count;
  q.units = q.rows > 0 ? max(1, (q.chunks + kWarps - 1) / kWarps) : 0;  // rows without a key are written too
  return q;
}

EC_DEV void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
EC_DEV void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
EC_DEV void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// CLUSTER: an item a cluster; else shares of the line.
template <int D, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1) few_rows_kernel(const __grid_constant__ Args a) {
  using LY = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc& misc = *reinterpret_cast<Misc*>(smem + LY::kMiscOff);
  const Shape& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + LY::kBarOff) + warp * LY::kStages;
  const uint32_t ring = smem_u32(smem) + warp * LY::kStages * LY::kStage;
  if (lane < LY::kStages) {
    mbar_init(&full[lane], 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    misc.abort = (smem_u32(smem) & 1023u) != 0u;  // the swizzled chunks need the alignment that dynamic shared memory has here
    if (misc.abort) report_error(s.dev_err, EC_DEVERR_TIMEOUT);
    misc.begin = {0, 0, 0, 0};
    prefetch_tmap(&a.tk);
    prefetch_tmap(&a.tv);
  }
  prefetch_small(s, kThreads);
  pdl_wait();  // everything may come from the previous kernels in the stream
  pdl_launch_dependents();

  Place at;
  Seq cs;
  int base = 0, lim = 0;  // the item's chunks that fall to this CTA
  if constexpr (CLUSTER) {
    const int S = cluster_size(), rank = cluster_ctarank(), item = blockIdx.x / S;
    at = {item / s.Hkv, item % s.Hkv, 0, 0};
    cs = load_seq(s, at.b, rank == 0 && at.kvh == 0 && warp == 0 && lane == 0);
    if (cs.rows == 0 || (smem_u32(smem) & 1023u) != 0u) return;  // the whole cluster
    base = cs.chunks * rank / S;
    lim = cs.chunks * (rank + 1) / S;
    at.left = (lim - base + kWarps - 1) / kWarps;
    __syncthreads();  // the barriers are up
  } else {
    // The line: each thread adds up the units of its sequences, the CTA their sum, and the thread whose sequences hold the
    // first unit of this CTA's share finds it.
    const int per = (s.B + kThreads - 1) / kThreads, b0 = threadIdx.x * per;
    int mine = 0;
    for (int b = b0; b < min(b0 + per, s.B); ++b) mine += load_seq(s, b, blockIdx.x == 0).units * s.Hkv;
    int incl = warp_inclusive(mine);
    if (lane == 31) misc.scan[warp] = incl;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += misc.scan[w];
      total += misc.scan[w];
    }
    const int share = (total + gridDim.x - 1) / gridDim.x;
    const int begin = blockIdx.x * share;
    if (begin < total && begin >= incl - mine && begin < incl) {
      int off = begin - (incl - mine);
      for (int b = b0;; ++b) {
        const int units = load_seq(s, b, false).units;
        if (off < units * s.Hkv) {
          misc.begin = {b, off / units, off % units, min(share, total - begin)};
          break;
        }
        off -= units * s.Hkv;
      }
    }
    if (threadIdx.x == 0) misc.share = share;
    __syncthreads();
    if (threadIdx.x == 0) a.records[blockIdx.x].parts = 0;
    at = misc.begin;
    if (at.left == 0 || misc.abort) return;
    cs = load_seq(s, at.b, false);
    lim = cs.chunks;
  }

  // ---- loads: the warp's chunks in the line's order, kStages of them ahead
  Place la = at;
  Seq ls = cs;
  int l_u1 = CLUSTER ? la.left : min(ls.units, la.u + la.left);  // end of this item's units in the share
  int l_lim = lim;
  int l_base = -1, l_page = 0;               // lane i: the page of the warp's chunk of unit l_base + i
  int issued = 0;
  auto issue = [&]() {
    for (;;) {
      if (la.left == 0) return;
      if (la.u < l_u1 && base + la.u * kWarps + warp < l_lim) break;
      if (la.u < l_u1) {  // the last unit of an item has no chunk for this warp
        ++la.u;
        --la.left;
        continue;
      }
      if constexpr (CLUSTER) return;
      la.u = 0;
      if (++la.kvh == s.Hkv) {
        la.kvh = 0;
        do ls = load_seq(s, ++la.b, false);
        while (ls.units == 0);
      }
      l_u1 = min(ls.units, la.left);
      l_lim = ls.chunks;
      l_base = -1;
    }
    if (l_base < 0 || la.u >= l_base + 32) {
      l_base = la.u;
      const int v = base + (l_base + lane) * kWarps + warp;
      l_page = l_base + lane < l_u1 && v < l_lim ? page_of(s, la.b, ls.k.block(v) << kChunkShift) : s.n_pages;
    }
    const int page = __shfl_sync(0xffffffffu, l_page, la.u - l_base);
    if (lane == 0) {
      const int st = issued % LY::kStages;
      const int slot = (ls.k.block(base + la.u * kWarps + warp) << kChunkShift) & ((1 << s.page_shift) - 1);
      uint8_t* dst = smem + (warp * LY::kStages + st) * LY::kStage;
      mbar_arrive_expect_tx(&full[st], LY::kStage);
      tma_load_5d(dst, &a.tk, &full[st], 0, slot, 0, la.kvh, page);
      tma_load_5d(dst + LY::kKBytes, &a.tv, &full[st], 0, slot, 0, la.kvh, page);
    }
    ++issued;
    ++la.u;
    --la.left;
  };
  __syncwarp();
#pragma unroll 1
  for (int i = 0; i < LY::kStages; ++i) issue();

  // ---- items of the share
  const int gid = lane >> 2, tid = lane & 3;  // a fragment's row and column pair
  const uint32_t k_lane = ((lane >> 4) * 8 + (lane & 7)) * 128, k_c = (lane >> 3) & 1;
  const uint32_t v_lane = (((lane >> 3) & 1) * 8 + (lane & 7)) * 128, v_c = lane >> 4;
  const uint32_t swz = lane & 7;
  int used = 0;
  bool ok = true;
  for (;;) {
    const int u1 = CLUSTER ? at.left : min(cs.units, at.u + at.left);
    const int packed = cs.rows * s.g;
    // the rows of this thread's fragments: their queries, and the keys that they see
    uint32_t qf[D / 16][4];
    int r_lo[2], r_hi[2];
    bool even = true;  // this thread's rows see the same keys as the hull
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int x = gid + 8 * e;
      const bool live = x < packed;
      const int r = live ? s.by_g(x) : 0;
      const uint16_t* src = a.q + ((static_cast<int64_t>(at.b) * s.rows_max + r) * s.Hq + at.kvh * s.g + (x - r * s.g)) * D + 2 * tid;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][e] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk)) : 0u;
        qf[kk][e + 2] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk + 8)) : 0u;
      }
      r_lo[e] = cs.h.lo, r_hi[e] = cs.h.hi;
      if (s.windowed && live) {
        const int64_t pos = raw_position(s.at, at.b, r);
        const int p = inside(pos, s.L) ? static_cast<int>(pos) : 0;
        r_lo[e] = max(p - s.w.left, 0);
        r_hi[e] = min(p + s.w.right + 1, cs.n);
        even = even && r_lo[e] <= cs.h.lo && r_hi[e] >= cs.h.hi;
      }
    }
    even = __all_sync(0xffffffffu, even);

    float o[D / 8][4] = {};
    float m[2], l[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) m[e] = -INFINITY, l[e] = 0.f;

#pragma unroll 1
    for (int u = at.u; u < u1; ++u) {
      const int v = base + u * kWarps + warp;
      if (v >= lim) break;
      const int st = used % LY::kStages;
      ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(&full[st], (used / LY::kStages) & 1, &misc.abort, s.dev_err, kWaitLimitNs));
      if (!ok) break;
      const int j0 = cs.k.block(v) << kChunkShift;
      const uint32_t kb = ring + st * LY::kStage, vb = kb + LY::kKBytes;
      const bool whole = j0 + kChunk <= cs.h.near || (j0 >= cs.h.lo && j0 + kChunk <= cs.h.hi);
      if (!whole) {  // rows of V outside the hull may hold anything, and a weight of zero times NaN is NaN
        const int j = j0 + (lane >> 1);
        if (!(j < cs.h.near || (j >= cs.h.lo && j < cs.h.hi)))
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int c = (lane & 1) * (D / 16) + i;
            st_shared16(vb + (c >> 3) * (kChunk * 128) + (lane >> 1) * 128 + (c & 7) * 16, make_uint4(0, 0, 0, 0));
          }
        fence_proxy_async_smem();  // before the TMA writes there again
        __syncwarp();
      }
      // scores of 16 keys: two fragments of 8
      float sc[2][4] = {};
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t kf[4];
        ldsm4(kf, kb + (kk >> 2) * (kChunk * 128) + k_lane + ((((kk & 3) * 2 + k_c) ^ swz) << 4));
        mma16816(sc[0], qf[kk], kf[0], kf[1]);
        mma16816(sc[1], qf[kk], kf[2], kf[3]);
      }
      if (!(whole && even)) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int j = j0 + 8 * i + 2 * tid + (c & 1);
            if (!(j < cs.h.near || (j >= r_lo[c >> 1] && j < r_hi[c >> 1]))) sc[i][c] = -INFINITY;
          }
      }
      uint32_t pf[4];
      float mx[2];
      bool grow = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(fmaxf(sc[0][2 * e], sc[0][2 * e + 1]), fmaxf(sc[1][2 * e], sc[1][2 * e + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        mx[e] = x * s.scale_log2;
        grow = grow || mx[e] > m[e] + kRescaleLog2;
      }
      if (__any_sync(0xffffffffu, grow)) {
        float al[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool up = mx[e] > m[e] + kRescaleLog2;
          al[e] = up ? ex2_approx(m[e] - mx[e]) : 1.f;
          if (up) m[e] = mx[e];
          l[e] *= al[e];
        }
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[d][c] *= al[c >> 1];
      }
      float p[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float nm = m[e] == -INFINITY ? 0.f : -m[e];  // no key seen yet: every score is -infinity
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) p[i][2 * e + c] = ex2_approx(fmaf(sc[i][2 * e + c], s.scale_log2, nm));
        l[e] += (p[0][2 * e] + p[0][2 * e + 1]) + (p[1][2 * e] + p[1][2 * e + 1]);
      }
      // the weights are rounded to bf16 for the product (2^-8 of each), the sum is of the unrounded ones
      pf[0] = pack_bf16x2(p[0][0], p[0][1]);
      pf[1] = pack_bf16x2(p[0][2], p[0][3]);
      pf[2] = pack_bf16x2(p[1][0], p[1][1]);
      pf[3] = pack_bf16x2(p[1][2], p[1][3]);
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t vf[4];
        ldsm4t(vf, vb + (d >> 2) * (kChunk * 128) + v_lane + ((((d & 3) * 2 + v_c) ^ swz) << 4));
        mma16816(o[2 * d], pf, vf[0], vf[1]);
        mma16816(o[2 * d + 1], pf, vf[2], vf[3]);
      }
      ++used;
      __syncwarp();
      issue();
    }

    // ---- join of the eight warps
    float2* stat = reinterpret_cast<float2*>(smem + LY::kStatOff);
    float* join = reinterpret_cast<float*>(smem + LY::kJoinOff);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      if (tid == 0) stat[warp * LY::kRows + gid + 8 * e] = make_float2(m[e], l[e]);
    }
    __syncthreads();
    // Buffers of four warps beside the ring; with no loads under way (an item a cluster) the other four's in the ring.
    auto buffer = [&](int w) { return w < kWarps / 2 ? join + w * LY::kRows * LY::kPitch : reinterpret_cast<float*>(smem) + (w - kWarps / 2) * LY::kRows * LY::kPitch; };
    auto put = [&](int w, bool add) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int x = gid + 8 * e;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top = fmaxf(top, stat[i * LY::kRows + x].x);
        const float f = m[e] == -INFINITY ? 0.f : ex2_approx(m[e] - top);
        float2* row = reinterpret_cast<float2*>(buffer(w) + x * LY::kPitch) + tid;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          float2 y = make_float2(o[d][2 * e] * f, o[d][2 * e + 1] * f);
          if (add) y.x += row[4 * d].x, y.y += row[4 * d].y;
          row[4 * d] = y;
        }
      }
    };
    if constexpr (CLUSTER) {
      put(warp, false);
    } else {
      if (warp >= kWarps / 2) put(warp - kWarps / 2, false);
      __syncthreads();
      if (warp < kWarps / 2) put(warp, true);
    }
    __syncthreads();
    const bool cut_here = !CLUSTER && u1 < cs.units;
    const bool part = at.u > 0 || cut_here;
    auto write = [&](int x, int c, const float4 (&y)[2], float sum) {
      const int r = s.by_g(x);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      uint4 z;
      z.x = pack_bf16x2(y[0].x * inv, y[0].y * inv);
      z.y = pack_bf16x2(y[0].z * inv, y[0].w * inv);
      z.z = pack_bf16x2(y[1].x * inv, y[1].y * inv);
      z.w = pack_bf16x2(y[1].z * inv, y[1].w * inv);
      if (sum == 0.f) z = make_uint4(0, 0, 0, 0);  // every score -infinity: y may hold 0 x infinity
      *reinterpret_cast<uint4*>(a.out + ((static_cast<int64_t>(at.b) * s.rows_max + r) * s.Hq + at.kvh * s.g + (x - r * s.g)) * D + c) = z;
    };
    const int slot = blockIdx.x * 2 + (at.u == 0 ? 1 : 0);
#pragma unroll 1
    for (int i = threadIdx.x; i < packed * (D / 8); i += kThreads) {
      const int x = i / (D / 8), c = i % (D / 8) * 8;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[w * LY::kRows + x].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 st = stat[w * LY::kRows + x];
        sum += st.x == -INFINITY ? 0.f * st.y : ex2_approx(st.x - top) * st.y;  // a NaN sum stays one
      }
      const int r = s.by_g(x);
      bool good = true;  // right, or not written: the row's keys are between those of the first and the last row
      if (s.windowed) {
        const int64_t pos = raw_position(s.at, at.b, r);
        const int p = inside(pos, s.L) ? static_cast<int>(pos) : 0;
        good = inside(pos, s.L) && min(max(p - s.w.left, 0), cs.n) >= cs.h.lo && min(p + s.w.right + 1, cs.n) <= cs.h.hi;
        if (!good && c == 0) report_error(s.dev_err, EC_DEVERR_BAD_IDX);
      }
      float4 y[2] = {};
#pragma unroll
      for (int w = 0; w < (CLUSTER ? kWarps : kWarps / 2); ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 z = *reinterpret_cast<const float4*>(buffer(w) + x * LY::kPitch + c + 4 * h);
          y[h].x += z.x, y[h].y += z.y, y[h].z += z.z, y[h].w += z.w;
        }
      if constexpr (CLUSTER) {
        float4* dst = reinterpret_cast<float4*>(join + x * LY::kPitch + c);  // over this thread's own columns
        dst[0] = y[0], dst[1] = y[1];
        if (c == 0) misc.stat[x] = make_float2(good ? top : kNotWritten(), sum);
      } else if (part) {
        float4* dst = reinterpret_cast<float4*>(a.part_o + (static_cast<int64_t>(slot) * kFewRows + x) * D + c);
        dst[0] = y[0], dst[1] = y[1];
        if (c == 0) a.part_stat[slot * kFewRows + x] = make_float2(good ? top : kNotWritten(), sum);
      } else if (good) {
        write(x, c, y, sum);
      }
    }
    if constexpr (CLUSTER) {
      // the cluster's CTAs share out the row's pieces and read all parts of theirs
      const int S = cluster_size(), rank = cluster_ctarank();
      cluster_arrive_release();
      cluster_wait_acquire();
#pragma unroll 1
      for (int i = rank * kThreads + threadIdx.x; i < packed * (D / 8); i += S * kThreads) {
        const int x = i / (D / 8), c = i % (D / 8) * 8;
        float2 st[kMaxCluster];
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          st[r] = r < S ? ld_dsmem8(dsmem_map(smem_u32(&misc.stat[x]), r)) : make_float2(-INFINITY, 0.f);
          top = fmaxf(top, st[r].x);
        }
        const bool lost = st[0].x != st[0].x;
        float4 y[2] = {};
        float4 z[kMaxCluster][2];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)  // all on the way at once
          if (r < S) {
            const uint32_t src = dsmem_map(smem_u32(join + x * LY::kPitch + c), r);
            z[r][0] = ld_dsmem16(src), z[r][1] = ld_dsmem16(src + 16);
          }
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          if (r >= S) break;
          const float4 z0 = z[r][0], z1 = z[r][1];
          const float f = st[r].x == -INFINITY ? 1.f : ex2_approx(st[r].x - top);  // no finite score: zeros, or NaN
          sum += f * st[r].y;
          y[0].x += f * z0.x, y[0].y += f * z0.y, y[0].z += f * z0.z, y[0].w += f * z0.w;
          y[1].x += f * z1.x, y[1].y += f * z1.y, y[1].z += f * z1.z, y[1].w += f * z1.w;
        }
        if (!lost) write(x, c, y, sum);
      }
    }
    if (!ok)  // a wait gave up: the copies in flight land before the CTA ends, as far as they do
      for (; used < issued; ++used)
        for (int i = 0; i < (1 << 16) && !mbar_try_wait(&full[used % LY::kStages], (used / LY::kStages) & 1); ++i) {
        }
    if constexpr (CLUSTER) {
      cluster_arrive_release();  // no CTA leaves while another one reads its rows
      cluster_wait_acquire();
      return;
    }
    at.left -= u1 - at.u;
    if (at.left == 0) {
      if (threadIdx.x == 0 && cut_here && at.u == 0) {  // the item begins here and goes on in the next CTAs
        const int rest = cs.units - u1;
        a.records[blockIdx.x] = {1 + (rest + misc.share - 1) / misc.share, at.b, at.kvh, 0, packed, {0, 0, 0}};
      }
      break;
    }
    __syncthreads();  // the join's buffers are free
    at.u = 0;
    if (++at.kvh == s.Hkv) {
      at.kvh = 0;
      do cs = load_seq(s, ++at.b, false);
      while (cs.units == 0);
      lim = cs.chunks;
    }
  }
}

template <int D>
cudaError_t launch(const Args& a, int ctas, int cluster, cudaStream_t s) {
  if (cluster == 0) return launch_pdl(few_rows_kernel<D, false>, dim3(ctas), dim3(kThreads), Layout<D>::kBytes, s, a);
  return launch_pdl_cluster(few_rows_kernel<D, true>, dim3(a.s.B * a.s.Hkv * cluster), dim3(kThreads), Layout<D>::kBytes, cluster, s, a);
}

}  // namespace

cudaError_t setup_few_rows(Device* d) {
  auto allow = [](const void* f, int bytes) { return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); };
  const void* f = reinterpret_cast<const void*>(few_rows_kernel<128, true>);
  cudaError_t e = allow(f, Layout<128>::kBytes);
  if (e == cudaSuccess) e = allow(reinterpret_cast<const void*>(few_rows_kernel<128, false>), Layout<128>::kBytes);
  if (e == cudaSuccess) e = allow(reinterpret_cast<const void*>(few_rows_kernel<64, true>), Layout<64>::kBytes);
  if (e == cudaSuccess) e = allow(reinterpret_cast<const void*>(few_rows_kernel<64, false>), Layout<64>::kBytes);
  d->clusters[0] = 0;
  d->clusters[1] = d->sms;
  for (int S = 2; e == cudaSuccess && S <= kMaxCluster; ++S) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(S);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(S);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<128>::kBytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&d->clusters[S], f, &cfg);
  }
  return e;
}

cudaError_t launch_few_rows(const Args& a, int D, int ctas, int cluster, cudaStream_t s) {
  return D == 64 ? launch<64>(a, ctas, cluster, s) : launch<128>(a, ctas, cluster, s);
}

}  // namespace paged
}  // namespace ec
