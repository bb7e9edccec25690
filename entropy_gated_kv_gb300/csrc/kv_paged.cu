// kv_paged.cu — fresh K/V rows into a paged cache, rotated on the way, and the rows' rotated queries.
//
// EntropyCache, gist.science zh summary §2.2 (partial forward): the recompute set gets fresh K/V rows; the pages
// of a pool and the rotation beside the write have no counterpart there. For row r < R[b] at position pos:
//   K page row (b, pos) = rotate(k_new[b, r], pos), V page row = v_new[b, r], q_out[b, r] = rotate(q_new[b, r], pos)
//   rotate: (x_i, x_{i + D/2}) -> (x_i c_i - x_{i + D/2} s_i, x_{i + D/2} c_i + x_i s_i), fp32, rounded once.
// HBM-bound: every row is read and written once, 4 (Hq + 2 Hkv) D bytes, beside 4 D bytes of the angles' table; a short
// call by its chain of loads (sizes, rows and positions, page numbers and angles). Loading the rows beside the sizes took
// 0.2 us off that, and registers that cost the long call 30.
#include <algorithm>

#include "ec_common.cuh"
#include "ec_internal.h"
#include "paged_common.cuh"

namespace ec {
namespace paged {
namespace {

// Threads of a CTA, and 32-byte pieces that a thread loads before it stores any. 4 x 4096 rows of 32 heads: 123 us (6.6
// TB/s) so, 139 with 256 x 3, 138 with 256 x 2, 122 with 128 x 3; 8 x 95 rows of 28/4 heads: 4.9 us, 5.8, 5.0, 5.3: smaller
// CTAs mix loads and stores of more rows on an SM, larger ones start fewer for a short call.
constexpr int kThreads = 192;
constexpr int kInFlight = 2;

struct AppendArgs {
  int32_t L, Hq, Hkv, rows_max, page_shift, n_pages;
  RowSplit split;
  int64_t page_stride, table_stride;
  ec_rows k, v, q;
  uint16_t *kp, *vp, *q_out;
  const float *cs, *sn;
  const int32_t *table, *R;
  RowPlaces at;
  int32_t* dev_err;
};

// A piece is 8 features i .. i + 7 and their partners i + D/2 ..: T = D / 16 pieces a head, the heads of a row in
// the order q, k, v.
template <int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int T = D / 16;
  const int b = blockIdx.y, r0 = blockIdx.x * a.split.rows_per_cta;
  pdl_wait();  // the rows, idx and R may come from the previous kernels in the stream
  pdl_launch_dependents();
  const int Rb = __ldg(a.R + b);
  if (Rb < 0 || Rb > a.rows_max) {
    if (r0 == 0 && threadIdx.x == 0) report_error(a.dev_err, EC_DEVERR_BAD_R);
    return;
  }
  const int n = a.split.count(r0, Rb);
  const int nq = a.q_out != nullptr ? a.Hq : 0;
  for (int base = threadIdx.x; base < n; base += kInFlight * kThreads) {
    uint4 lo[kInFlight], hi[kInFlight];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      const int u = base + i * kThreads;
      if (u < n) {
        const int rl = a.split.per_row(u), w = u - rl * a.split.pieces, h = w / T, t = w % T, r = r0 + rl;
        const bool is_q = h < nq;
        const bool is_k = !is_q && h < nq + a.Hkv;
        const ec_rows& x = is_q ? a.q : is_k ? a.k : a.v;
        const int hx = is_q ? h : is_k ? h - nq : h - nq - a.Hkv;
        const uint16_t* src = static_cast<const uint16_t*>(x.x) + b * x.batch_stride + r * x.row_stride + hx * D + t * 8;
        lo[i] = __ldcs(reinterpret_cast<const uint4*>(src));
        hi[i] = __ldcs(reinterpret_cast<const uint4*>(src + D / 2));
      }
    }
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      const int u = base + i * kThreads;
      if (u >= n) break;
      const int rl = a.split.per_row(u), w = u - rl * a.split.pieces, h = w / T, t = w % T, r = r0 + rl;
      const int64_t raw = raw_position(a.at, b, r);
      const int pos = inside(raw, a.L) ? static_cast<int>(raw) : -1;
      // Rows ascend: one that does not lie below its successor is bad, and is left out, as two neighbours at one position
      // would both write it. Rows further apart at one position have such a row between them: the list is reported,
      // but both write.
      const bool falls = a.at.idx != nullptr && r + 1 < Rb && pos >= __ldg(a.at.idx + b * a.at.stride + r + 1);
      if (pos < 0 || falls) {
        if (w == 0) report_error(a.dev_err, EC_DEVERR_BAD_IDX);
        continue;
      }
      const bool is_q = h < nq;
      const bool is_k = !is_q && h < nq + a.Hkv;
      uint4 y0 = lo[i], y1 = hi[i];
      if ((is_q || is_k) && a.cs != nullptr) {
        const float4* cp = reinterpret_cast<const float4*>(a.cs + static_cast<int64_t>(pos) * (D / 2) + t * 8);
        const float4* sp = reinterpret_cast<const float4*>(a.sn + static_cast<int64_t>(pos) * (D / 2) + t * 8);
        const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
        const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
        uint32_t* p0 = &y0.x;
        uint32_t* p1 = &y1.x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a0 = bf16lo_to_f32(p0[e]), a1 = bf16hi_to_f32(p0[e]);
          const float b0 = bf16lo_to_f32(p1[e]), b1 = bf16hi_to_f32(p1[e]);
          p0[e] = pack_bf16x2(a0 * c[2 * e] - b0 * s[2 * e], a1 * c[2 * e + 1] - b1 * s[2 * e + 1]);
          p1[e] = pack_bf16x2(b0 * c[2 * e] + a0 * s[2 * e], b1 * c[2 * e + 1] + a1 * s[2 * e + 1]);
        }
      }
      uint16_t* dst;
      if (is_q) {
        dst = a.q_out + ((static_cast<int64_t>(b) * a.rows_max + r) * a.Hq + h) * D + t * 8;
      } else {
        const int page = __ldg(a.table + b * a.table_stride + (pos >> a.page_shift));
        if (page < 0 || page >= a.n_pages) {
          if (t == 0) report_error(a.dev_err, EC_DEVERR_BAD_PAGE);
          continue;
        }
        const int hx = is_k ? h - nq : h - nq - a.Hkv;
        const int slot = pos & ((1 << a.page_shift) - 1);
        dst = (is_k ? a.kp : a.vp) + page * a.page_stride + (static_cast<int64_t>(slot) * a.Hkv + hx) * D + t * 8;
      }
      *reinterpret_cast<uint4*>(dst) = y0;
      *reinterpret_cast<uint4*>(dst + D / 2) = y1;
    }
  }
}

}  // namespace
}  // namespace paged

cudaError_t launch_kv_append_paged(const ec_params& p, const ec_paged_kv& c, int32_t rows_max, const ec_rows& k,
                                   const ec_rows& v, const ec_rows& q, void* q_out, const float* cs, const float* sn,
                                   const RowPlaces& at, const int32_t* R, int32_t* dev_err, cudaStream_t s) {
  using namespace paged;
  AppendArgs a{};
  a.L = p.L, a.Hq = p.Hq, a.Hkv = p.Hkv, a.rows_max = rows_max;
  while ((1 << a.page_shift) < c.page_size) ++a.page_shift;
  a.n_pages = c.n_pages, a.page_stride = c.page_stride, a.table_stride = c.table_stride;
  a.split.set(rows_max, ((q_out != nullptr ? p.Hq : 0) + 2 * p.Hkv) * (p.D / 16), kInFlight * kThreads);
  a.k = k, a.v = v, a.q = q;
  a.kp = static_cast<uint16_t*>(c.k), a.vp = static_cast<uint16_t*>(c.v), a.q_out = static_cast<uint16_t*>(q_out);
  a.cs = cs, a.sn = sn, a.table = c.table, a.R = R, a.at = at, a.dev_err = dev_err;
  const dim3 grid((rows_max + a.split.rows_per_cta - 1) / a.split.rows_per_cta, p.B);
  return launch_pdl(p.D == 64 ? append_kernel<64> : append_kernel<128>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace ec
