// attention_paged.cu — attention of the recompute rows against a K/V cache in pages, whole or in a window: the choice
// of a kernel, and the join of items that were cut between CTAs.
//
// EntropyCache, gist.science zh summary §2.2 and pt summary §1: the recompute rows attend to every cached row, with no
// causal mask. Pages and windows have no counterpart there.
//   out[b, r, h] = sum_j softmax_j(scale <q[b, r, h], k_j>) v_j over the keys j that row r sees, KV head h / g
#include <algorithm>
#include <atomic>
#include <mutex>

#include "paged_common.cuh"

namespace ec {
namespace paged {
namespace {

// Joins the partial rows of an item that was cut: o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i. One CTA takes a
// CTA's record and one row of it, its warps every kMergeWarps-th part each, in an order that no timing changes.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_rows_kernel(const __grid_constant__ Args a) {
  constexpr int E = D / 32;
  __shared__ float acc[kMergeWarps][D];
  const Shape& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, x = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  const Record rec = a.records[blockIdx.x];
  if (rec.parts == 0 || x >= rec.rows) return;
  float top = -INFINITY;
  bool lost = false;
  float2 st[(kMaxCtas + 31) / 32];
#pragma unroll
  for (int k = 0; k < (kMaxCtas + 31) / 32; ++k) {
    const int i = lane + 32 * k;
    st[k] = i < rec.parts ? a.part_stat[part_slot(blockIdx.x, i, 1, 0) * kFewRows + x] : make_float2(-INFINITY, 0.f);
    top = fmaxf(top, st[k].x);
    lost = lost || st[k].x != st[k].x;
  }
  if (__any_sync(0xffffffffu, lost)) return;  // a row that is not written, in every warp
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
        const float* src = a.part_o + (part_slot(blockIdx.x, i, 1, 0) * kFewRows + x) * D + lane * E;
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
  float2 y = make_float2(0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    const float2 z = *reinterpret_cast<const float2*>(&acc[w][2 * threadIdx.x]);
    y.x += z.x, y.y += z.y;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t* dst = reinterpret_cast<uint32_t*>(
      a.out + ((static_cast<int64_t>(rec.b) * s.rows_max + r) * s.Hq + rec.kvh * s.g + (xr - r * s.g)) * D);
  dst[threadIdx.x] = sum == 0.f ? 0u : pack_bf16x2(y.x * inv, y.y * inv);  // every score -infinity: y may hold 0 x infinity
}

// The same for tiles: a CTA takes a record and 64 rows of it, a thread a row and every eighth quad of columns, as many
// parts in flight as make eight quads. Where a few items may go over many CTAs each (QUADS 1) a CTA takes eight quads only:
// for all calls that took 7 us more on 8 x 95 rows of 28/4 heads, most of its CTAs without a record. (32 rows a CTA:
// 94.4 us for 93.1 on 95 rows behind 32768 keys, 32 heads, 128 rows 95.0, measured when that call stood in the line; clusters take it now.)
constexpr int kTileMergeThreads = 512;
constexpr int kTileMergeRows = 64;

template <int D, int QUADS>
__global__ void __launch_bounds__(kTileMergeThreads) merge_tiles_kernel(const __grid_constant__ Args a, int tiles) {
  constexpr int kWarps = 8, kBatch = 8 / QUADS;  // of 32 rows
  const Shape& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const Record rec = a.records[blockIdx.x];
  const int row = blockIdx.y * kTileMergeRows + warp / kWarps * 32 + lane, quad0 = blockIdx.z * kWarps * QUADS + warp % kWarps;
  if (rec.parts == 0 || row >= rec.rows || quad0 >= D / 4) return;
  const int cta = blockIdx.x / tiles, tile = blockIdx.x - cta * tiles;
  float m = -INFINITY, l = 0.f;
  float4 o[QUADS] = {};
  bool lost = false;
  for (int i0 = 0; i0 < rec.parts; i0 += kBatch) {
    float2 st[kBatch];
    float4 y[kBatch][QUADS];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = min(i0 + k, rec.parts - 1);
      const int64_t slot = part_slot(cta, i, tiles, tile);
      st[k] = __ldcg(a.part_stat + slot * kTileRows + row);
#pragma unroll
      for (int c = 0; c < QUADS; ++c)
        y[k][c] = __ldcg(reinterpret_cast<const float4*>(a.part_o) + (slot * (D / 4) + quad0 + c * kWarps) * kTileRows + row);
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) top = fmaxf(top, st[k].x);
    const float f0 = m == -INFINITY ? 1.f : ex2_approx(m - top);
    m = top;
    l *= f0;
#pragma unroll
    for (int c = 0; c < QUADS; ++c) o[c].x *= f0, o[c].y *= f0, o[c].z *= f0, o[c].w *= f0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (i0 + k >= rec.parts) break;
      lost = lost || st[k].x != st[k].x;
      const float f = st[k].x == -INFINITY ? 1.f : ex2_approx(st[k].x - top);  // no finite score: zeros, or NaN
      l += f * st[k].y;
#pragma unroll
      for (int c = 0; c < QUADS; ++c) o[c].x += f * y[k][c].x, o[c].y += f * y[k][c].y, o[c].z += f * y[k][c].z, o[c].w += f * y[k][c].w;
    }
  }
  if (lost) return;
  const int xr = rec.row0 + row, r = s.by_g(xr);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2* dst = reinterpret_cast<uint2*>(a.out + ((static_cast<int64_t>(rec.b) * s.rows_max + r) * s.Hq + rec.kvh * s.g + (xr - r * s.g)) * D);
#pragma unroll
  for (int c = 0; c < QUADS; ++c)
    dst[quad0 + c * kWarps] = make_uint2(pack_bf16x2(o[c].x * inv, o[c].y * inv), pack_bf16x2(o[c].z * inv, o[c].w * inv));
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

// Queries as [sequence][row][KV head][head of it][D]: a box is nr rows of the g heads of a KV head, 64 features.
bool encode_queries(EncodeTiledFn enc, CUtensorMap* m, const void* q, const ec_params& p, int rows_max, int nr) {
  const cuuint64_t D = p.D, g = p.Hq / p.Hkv, H = p.Hkv, n = rows_max;
  const cuuint64_t dims[5] = {D, g, H, n, static_cast<cuuint64_t>(p.B)};
  const cuuint64_t strides[4] = {D * 2, g * D * 2, H * g * D * 2, n * H * g * D * 2};
  const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(g), 1, static_cast<cuuint32_t>(nr), 1};
  const cuuint32_t es[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(q), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The current device's; null on an error.
const Device* device_info(cudaError_t* e) {
  constexpr int kDevices = 64;
  static Device info[kDevices];
  static std::atomic<bool> ready[kDevices];
  static std::mutex mutex;
  int dev = 0;
  *e = cudaGetDevice(&dev);
  if (*e != cudaSuccess) return nullptr;
  if (dev < 0 || dev >= kDevices) {
    *e = cudaErrorNotSupported;
    return nullptr;
  }
  if (!ready[dev].load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(mutex);
    if (!ready[dev].load(std::memory_order_relaxed)) {
      *e = current_device_sms(&info[dev].sms);
      if (*e == cudaSuccess) *e = setup_few_rows(&info[dev]);
      if (*e == cudaSuccess) *e = setup_tiles();
      if (*e != cudaSuccess) return nullptr;
      ready[dev].store(true, std::memory_order_release);
    }
  }
  return &info[dev];
}

struct WsLayout {
  size_t stat, records, total;
};
WsLayout ws_layout(const ec_params& p, int32_t rows_max) {
  const int nr = tile_positions(p, rows_max);
  const bool few = few_rows(p, rows_max);
  const size_t tiles = few || rows_max <= nr ? 1 : 2;
  const size_t rows = kMaxCtas * 2 * tiles * (few ? kFewRows : kTileRows);
  WsLayout w{};
  w.stat = rows * p.D * sizeof(float);
  w.records = w.stat + rows * sizeof(float2);
  w.total = w.records + kMaxCtas * tiles * sizeof(Record);
  return w;
}

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
  cudaError_t e = cudaSuccess;
  const Device* const device = device_info(&e);
  if (device == nullptr) return e;
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
  const int ctas = std::min(device->sms, kMaxCtas);
  const bool few = few_rows(p, rows_max);
  // a chunk of 16 keys, or a block of 128 as far as a page holds it
  const int box = few ? 16 : std::min(128, c.page_size), atoms = few || box == 128 ? p.D / 64 : 1;
  const int nr = tile_positions(p, rows_max);
  if (!encode_pool(enc, &a.tk, c.k, p, c, box, atoms) || !encode_pool(enc, &a.tv, c.v, p, c, box, atoms) ||
      (!few && !encode_queries(enc, &a.tq, q, p, rows_max, nr))) {
    *status = EC_ERR_INVALID_ARG;
    return cudaErrorInvalidValue;
  }
  if (few) {
    const int cluster = few_rows_cluster(p, rows_max, window, at, kv_len != nullptr, *device);
    e = launch_few_rows(a, p.D, ctas, cluster, s);
    if (e == cudaSuccess && cluster == 0)
      e = launch_pdl(p.D == 64 ? merge_rows_kernel<64> : merge_rows_kernel<128>, dim3(ctas, rows_max * sh.g), dim3(32 * kMergeWarps), 0, s, a);
  } else {
    const int tiles = rows_max <= nr ? 1 : 2;
    const int cluster = tiles_cluster(p, rows_max, nr, window, at, kv_len != nullptr, *device);
    e = launch_tiles(a, p.D, nr, ctas, cluster, s);
    // eight items or fewer may each go over many CTAs: their parts one column quad a thread
    const bool few_items = static_cast<int64_t>(p.B) * p.Hkv * ((rows_max + nr - 1) / nr) <= 8;
    const int quads = p.D / 32;  // of a thread that takes every eighth one
    const dim3 grid(ctas * tiles, kTileRows / kTileMergeRows, few_items ? quads : 1);
    if (cluster != 0) {
      // joined on the chip
    } else if (e == cudaSuccess && p.D == 64) {
      e = launch_pdl(few_items ? merge_tiles_kernel<64, 1> : merge_tiles_kernel<64, 2>, grid, dim3(kTileMergeThreads), 0, s, a, tiles);
    } else if (e == cudaSuccess) {
      e = launch_pdl(few_items ? merge_tiles_kernel<128, 1> : merge_tiles_kernel<128, 4>, grid, dim3(kTileMergeThreads), 0, s, a, tiles);
    }
  }
  if (e == cudaSuccess) *status = EC_OK;
  return e;
}

}  // namespace ec
