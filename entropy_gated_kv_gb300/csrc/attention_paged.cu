// attention_paged.cu — attention of the recompute rows against a K/V cache in pages, whole or in a window: the choice
// of a kernel, and the join of items that were cut between CTAs.
//
// EntropyCache, gist.science zh summary §2.2 and pt summary §1: the recompute rows attend to every cached row, with no
// causal mask. Pages and windows have no counterpart there.
//   out[b, r, h] = sum_j softmax_j(scale <q[b, r, h], k_j>) v_j over the keys j that row r sees, KV head h / g
#include <algorithm>
#include <mutex>

#include "paged_common.cuh"

namespace ec {
namespace paged {
namespace {

// Joins the partial rows of an item that was cut: o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i. One CTA takes a
// CTA's record and one row of it, its warps every kMergeWarps-th part each, in an order that no timing changes.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_kernel(const __grid_constant__ Args a, int slot_rows, int slots) {
  constexpr int E = D / 32;
  __shared__ float acc[kMergeWarps][D];
  const Shape& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, x = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  const Record rec = a.records[blockIdx.x];
  if (rec.parts == 0 || x >= rec.rows) return;
  auto slot = [&](int i) { return i == 0 ? blockIdx.x * slots + 1 : (blockIdx.x + i) * slots; };
  float top = -INFINITY;
  float2 st[(kMaxCtas + 31) / 32];
#pragma unroll
  for (int k = 0; k < (kMaxCtas + 31) / 32; ++k) {
    const int i = lane + 32 * k;
    st[k] = i < rec.parts ? a.part_stat[static_cast<int64_t>(slot(i)) * slot_rows + x] : make_float2(-INFINITY, 0.f);
    top = fmaxf(top, st[k].x);
  }
  for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < (kMaxCtas + 31) / 32; ++k) {
    st[k].x = st[k].x == -INFINITY ? 0.f : ex2_approx(st[k].x - top);
    sum += st[k].x * st[k].y;
  }
  for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
  float o[E] = {};
#pragma unroll
  for (int k = 0; k < (kMaxCtas + 31) / 32; ++k) {
    if (32 * k >= rec.parts) break;
#pragma unroll
    for (int i0 = 0; i0 < 32; i0 += kMergeWarps) {
      const int i = 32 * k + i0 + warp;
      const float f = __shfl_sync(0xffffffffu, st[k].x, i0 + warp);
      if (i < rec.parts) {
        const float* src = a.part_o + (static_cast<int64_t>(slot(i)) * slot_rows + x) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 y = *reinterpret_cast<const float2*>(src + e);
          o[e] += f * y.x, o[e + 1] += f * y.y;
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) acc[warp][lane * E + e] = o[e];
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  const int xr = rec.row0 + x, r = s.by_g(xr);
  if (s.windowed && !inside(raw_position(s.at, rec.b, r), s.L)) {
    report_error(s.dev_err, EC_DEVERR_BAD_IDX);
    return;
  }
  float2 y = make_float2(0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    const float2 z = *reinterpret_cast<const float2*>(&acc[w][2 * threadIdx.x]);
    y.x += z.x, y.y += z.y;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t* dst = reinterpret_cast<uint32_t*>(
      a.out + ((static_cast<int64_t>(rec.b) * s.rows_max + r) * s.Hq + rec.kvh * s.g + (xr - r * s.g)) * D);
  dst[threadIdx.x] = pack_bf16x2(y.x * inv, y.y * inv);
}

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) paged_rows_kernel(const __grid_constant__ Args args, const uint16_t* kpool, const uint16_t* vpool, int64_t page_stride, int64_t rows) {
  const Shape& a = args.s;
  __shared__ __align__(16) float qs[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (row >= rows) return;
  const int h = static_cast<int>(row % a.Hq), r = static_cast<int>(row / a.Hq % a.rows_max),
            b = static_cast<int>(row / a.Hq / a.rows_max), kvh = h / a.g;
  int Rb, n;
  sizes_of(a, b, lane == 0, Rb, n);
  if (r >= Rb) return;
  int near = 0, first = 0, end = n;
  if (a.windowed) {
    const int64_t rp = raw_position(a.at, b, r);
    const int pos = static_cast<int>(rp);
    if (!inside(rp, a.L)) {
      if (lane == 0) report_error(a.dev_err, EC_DEVERR_BAD_IDX);
      return;
    }
    near = min(a.w.sinks, n);
    first = max(0, pos - a.w.left);
    end = min(n, pos + a.w.right + 1);
  }
  for (int d = lane; d < D; d += 32) qs[warp][d] = bf16lo_to_f32(args.q[row * D + d]);
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
      at = page * page_stride + (static_cast<int64_t>(j & ((1 << a.page_shift) - 1)) * a.Hkv + kvh) * D;
      float dot = 0.f;
      if (page >= 0)
        for (int d = 0; d < D; ++d) dot += qs[warp][d] * bf16lo_to_f32(kpool[at + d]);
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
        for (int e = 0; e < D / 32; ++e) o[e] += p * bf16lo_to_f32(vpool[ai + lane + 32 * e]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    args.out[row * D + lane + 32 * e] = static_cast<uint16_t>(pack_bf16x2(l == 0.f ? 0.f : o[e] * inv, 0.f));
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
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

// A pool of pages as [page][head][D / 64][row][64]: a box is `keys` rows of one head of one page in `atoms` pieces of
// 64 features, each with the 128-byte swizzle of the tensor cores' operands.
bool encode_pool(EncodeTiledFn enc, CUtensorMap* m, const void* base, const ec_params& p, const ec_paged_kv& c, int keys,
                 int atoms) {
  const cuuint64_t D = p.D, H = p.Hkv;
  const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(c.page_size), D / 64, H, static_cast<cuuint64_t>(c.n_pages)};
  const cuuint64_t strides[4] = {H * D * 2, 128, D * 2, static_cast<cuuint64_t>(c.page_stride) * 2};
  const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(keys), static_cast<cuuint32_t>(atoms), 1, 1};
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct WsLayout {
  size_t stat, records, total;
};
WsLayout ws_layout(const ec_params& p, int32_t rows_max) {
  const size_t rows = static_cast<size_t>(kMaxCtas) * kFewSlots * kFewRows;
  WsLayout w{};
  w.stat = rows * p.D * sizeof(float);
  w.records = w.stat + rows * sizeof(float2);
  w.total = w.records + kMaxCtas * sizeof(Record);
  return w;
}

bool few_rows(const ec_params& p, int32_t rows_max) { return static_cast<int64_t>(rows_max) * (p.Hq / p.Hkv) <= kFewRows; }

}  // namespace

}  // namespace paged

size_t paged_attention_workspace_bytes(const ec_params& p, int32_t rows_max) { return paged::ws_layout(p, rows_max).total; }

cudaError_t launch_paged_attention(const ec_params& p, int32_t rows_max, const void* q, const ec_paged_kv& c,
                                   const RowPlaces& at, const Window* window, const int32_t* R, const int32_t* kv_len,
                                   float scale, void* out, void* ws, int32_t* dev_err, cudaStream_t s, ec_status* status) {
  using namespace paged;
  *status = EC_ERR_CUDA;
  const EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return cudaErrorNotSupported;
  int sms = 0;
  cudaError_t e = cached_per_device(3000, &sms, [](int* n, void*) { return current_device_sms(n); }, nullptr);
  if (e != cudaSuccess) return e;
  Args a;
  Shape& sh = a.s;
  sh.B = p.B, sh.L = p.L, sh.Hq = p.Hq, sh.Hkv = p.Hkv, sh.g = p.Hq / p.Hkv, sh.rows_max = rows_max;
  sh.scope_hi = scope_hi(p), sh.windowed = window != nullptr, sh.page_shift = 0, sh.n_pages = c.n_pages;
  while ((1 << sh.page_shift) < c.page_size) ++sh.page_shift;
  sh.table_stride = c.table_stride, sh.scale_log2 = scale * kLog2e;
  sh.by_g.set(sh.g);
  sh.w = window != nullptr ? *window : Window{};
  sh.at = at, sh.R = R, sh.kv_len = kv_len, sh.table = c.table, sh.dev_err = dev_err;
  const WsLayout lay = ws_layout(p, rows_max);
  char* w = static_cast<char*>(ws);
  a.q = static_cast<const uint16_t*>(q), a.out = static_cast<uint16_t*>(out);
  a.part_o = reinterpret_cast<float*>(w);
  a.part_stat = reinterpret_cast<float2*>(w + lay.stat);
  a.records = reinterpret_cast<Record*>(w + lay.records);
  const int ctas = std::min(sms, kMaxCtas);
  if (few_rows(p, rows_max)) {
    if (!encode_pool(enc, &a.tk, c.k, p, c, 16, p.D / 64) || !encode_pool(enc, &a.tv, c.v, p, c, 16, p.D / 64)) {
      *status = EC_ERR_INVALID_ARG;
      return cudaErrorInvalidValue;
    }
    e = launch_few_rows(a, p.D, ctas, s);
    if (e == cudaSuccess)
      e = launch_pdl(p.D == 64 ? merge_kernel<64> : merge_kernel<128>, dim3(ctas, rows_max * sh.g), dim3(32 * kMergeWarps), 0, s, a,
                     kFewRows, kFewSlots);
  } else {
    const int64_t rows = static_cast<int64_t>(p.B) * rows_max * p.Hq;
    const unsigned grid = static_cast<unsigned>((rows + kWarps - 1) / kWarps);
    e = launch_pdl(p.D == 64 ? paged_rows_kernel<64> : paged_rows_kernel<128>, dim3(grid), dim3(32 * kWarps), 0, s, a,
                   static_cast<const uint16_t*>(c.k), static_cast<const uint16_t*>(c.v), c.page_stride, rows);
  }
  if (e == cudaSuccess) *status = EC_OK;
  return e;
}

}  // namespace ec
