// attention_paged.cu — attention of the recompute rows against a K/V cache in pages, whole or in a window.
//
// EntropyCache, gist.science zh summary §2.2 and pt summary §1: the recompute rows attend to every cached row, with no
// causal mask. Pages and windows have no counterpart there.
//   out[b, r, h] = sum_j softmax_j(scale <q[b, r, h], k_j>) v_j over the keys j that row r sees, KV head h / g
// One warp takes one query row and head: 32 keys at a time, a lane the score of one key, then the weights one
// after the other over the lanes' features, with the running maximum and sum of a softmax in one pass.
#include <algorithm>

#include "ec_common.cuh"
#include "ec_internal.h"
#include "paged_common.cuh"

namespace ec {
namespace paged {
namespace {

constexpr int kWarps = 4;

struct Args {
  int32_t L, Hq, g, Hkv, rows_max, page_shift, n_pages, scope_hi, windowed;
  int64_t page_stride, table_stride, rows;
  float scale_log2;
  const uint16_t *q, *k, *v;
  uint16_t* out;
  const int32_t *table, *R, *kv_len;
  RowPlaces at;
  Window w;
  int32_t* dev_err;
};

template <int D>
__global__ void __launch_bounds__(32 * kWarps) paged_rows_kernel(const __grid_constant__ Args a) {
  __shared__ __align__(16) float qs[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (row >= a.rows) return;
  const int h = static_cast<int>(row % a.Hq), r = static_cast<int>(row / a.Hq % a.rows_max),
            b = static_cast<int>(row / a.Hq / a.rows_max), kvh = h / a.g;
  const int Rb = __ldg(a.R + b), n = key_count(a.kv_len, b, a.L, a.scope_hi);
  if (Rb < 0 || Rb > a.rows_max || n < 0) {
    if (lane == 0) report_error(a.dev_err, n < 0 ? EC_DEVERR_BAD_LEN : EC_DEVERR_BAD_R);
    return;
  }
  if (r >= Rb) return;
  int near = 0, first = 0, end = n;
  if (a.windowed) {
    const int pos = position(a.at, b, r, a.L);
    if (pos < 0) {
      if (lane == 0) report_error(a.dev_err, EC_DEVERR_BAD_IDX);
      return;
    }
    near = min(a.w.sinks, n);
    first = max(0, pos - a.w.left);
    end = min(n, pos + a.w.right + 1);
  }
  for (int d = lane; d < D; d += 32) qs[warp][d] = bf16lo_to_f32(a.q[row * D + d]);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[D / 32] = {};
  for (int j0 = near > 0 ? 0 : first / 32 * 32; j0 < max(near, end); j0 += 32) {
    const int j = j0 + lane;
    const bool see = j < near || (j >= first && j < end);
    if (!__any_sync(0xffffffffu, see)) continue;
    int64_t at = 0;
    int page = 0;
    float sc = -INFINITY;
    if (see) {
      page = __ldg(a.table + b * a.table_stride + (j >> a.page_shift));
      if (page < 0 || page >= a.n_pages) {
        report_error(a.dev_err, EC_DEVERR_BAD_PAGE);
        page = -1;
      }
      at = page * a.page_stride + (static_cast<int64_t>(j & ((1 << a.page_shift) - 1)) * a.Hkv + kvh) * D;
      float dot = 0.f;
      if (page >= 0)
        for (int d = 0; d < D; ++d) dot += qs[warp][d] * bf16lo_to_f32(a.k[at + d]);
      sc = dot * a.scale_log2;
    }
    float mx = sc;
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) continue;
    const float alpha = exp2f(m - mn), pr = exp2f(sc - mn);
    m = mn;
    l *= alpha;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] *= alpha;
    for (int i = 0; i < 32; ++i) {
      const float p = __shfl_sync(0xffffffffu, pr, i);
      const int64_t ai = __shfl_sync(0xffffffffu, at, i);
      const bool si = __shfl_sync(0xffffffffu, see, i), pi = __shfl_sync(0xffffffffu, page, i) >= 0;
      if (!si) continue;
      l += p;
      if (pi)
#pragma unroll
        for (int e = 0; e < D / 32; ++e) o[e] += p * bf16lo_to_f32(a.v[ai + lane + 32 * e]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    a.out[row * D + lane + 32 * e] = static_cast<uint16_t>(pack_bf16x2(l == 0.f ? 0.f : o[e] * inv, 0.f));
}

}  // namespace
}  // namespace paged

size_t paged_attention_workspace_bytes(const ec_params&, int32_t) { return 256; }

cudaError_t launch_paged_attention(const ec_params& p, int32_t rows_max, const void* q, const ec_paged_kv& c,
                                   const RowPlaces& at, const Window* window, const int32_t* R, const int32_t* kv_len,
                                   float scale, void* out, void* ws, int32_t* dev_err, cudaStream_t s, ec_status* status) {
  using namespace paged;
  Args a{};
  a.L = p.L, a.Hq = p.Hq, a.g = p.Hq / p.Hkv, a.Hkv = p.Hkv, a.rows_max = rows_max;
  while ((1 << a.page_shift) < c.page_size) ++a.page_shift;
  a.n_pages = c.n_pages, a.scope_hi = scope_hi(p), a.windowed = window != nullptr;
  a.page_stride = c.page_stride, a.table_stride = c.table_stride, a.rows = static_cast<int64_t>(p.B) * rows_max * p.Hq;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.q = static_cast<const uint16_t*>(q), a.k = static_cast<const uint16_t*>(c.k), a.v = static_cast<const uint16_t*>(c.v);
  a.out = static_cast<uint16_t*>(out), a.table = c.table, a.R = R, a.kv_len = kv_len, a.at = at, a.dev_err = dev_err;
  if (window != nullptr) a.w = *window;
  const unsigned grid = static_cast<unsigned>((a.rows + kWarps - 1) / kWarps);
  const cudaError_t e = launch_pdl(p.D == 64 ? paged_rows_kernel<64> : paged_rows_kernel<128>, dim3(grid), dim3(32 * kWarps), 0, s, a);
  *status = e == cudaSuccess ? EC_OK : EC_ERR_CUDA;
  return e;
}

}  // namespace ec
