// ec_api.cu — the C ABI of the EntropyCache step library: host-side validation, workspace
// layout and the composition of the stages into one denoising step.
//
// Every entry point validates its arguments on the host before launching anything, returns
// an ec_status and never throws. The library allocates no memory.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>

#include "ec_common.cuh"
#include "ec_internal.h"
#include "entropycache.h"

namespace ec {

static std::mutex g_cfg_mutex;
static std::map<std::pair<int, const void*>, size_t> g_dyn_smem;  // (device, kernel) -> configured bytes
static std::map<std::pair<int, int>, int> g_cached;               // (device, key) -> value

cudaError_t current_device_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

cudaError_t ensure_dyn_smem(const void* func, size_t bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_cfg_mutex);
  size_t& have = g_dyn_smem[{dev, func}];
  if (bytes <= have) return cudaSuccess;
  if (bytes > 48 * 1024) {
    e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e != cudaSuccess) return e;
  }
  have = bytes;
  return cudaSuccess;
}

cudaError_t cached_per_device(int key, int* value, cudaError_t (*make)(int* value, void* ctx), void* ctx) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_cfg_mutex);
  auto it = g_cached.find({dev, key});
  if (it != g_cached.end()) {
    *value = it->second;
    return cudaSuccess;
  }
  int v = 0;
  e = make(&v, ctx);
  if (e != cudaSuccess) return e;
  g_cached[{dev, key}] = v;
  *value = v;
  return cudaSuccess;
}

}  // namespace ec

using namespace ec;

namespace {

constexpr int32_t kMaxB = 4096;
constexpr int32_t kMaxL = 1 << 20;
constexpr int32_t kMaxV = 1 << 30;
constexpr int32_t kMaxCmax = 1024;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The byte ranges [a, a + na) and [b, b + nb) share a byte (addresses compared, never read).
bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
struct Extent {
  const void* p;
  size_t n;
};

// A buffer of `w` shares bytes with another one of `w` or with one of `r`.
template <size_t W, size_t N>
bool any_overlap(const Extent (&w)[W], const Extent (&r)[N]) {
  for (size_t i = 0; i < W; ++i) {
    for (size_t j = i + 1; j < W; ++j)
      if (overlaps(w[i].p, w[i].n, w[j].p, w[j].n)) return true;
    for (size_t j = 0; j < N; ++j)
      if (r[j].p != nullptr && overlaps(w[i].p, w[i].n, r[j].p, r[j].n)) return true;
  }
  return false;
}

size_t q_bytes(const ec_params& p) { return static_cast<size_t>(p.B) * p.L * p.Hq * p.D * 2; }
size_t kv_bytes(const ec_params& p) { return static_cast<size_t>(p.B) * p.L * p.Hkv * p.D * 2; }

// The attention writes out ([B, L, Hq, D]) while it reads q, k_cache and v_cache.
bool attention_io_overlap(const ec_params& p, const void* q, const void* k, const void* v, const void* out) {
  const size_t nq = q_bytes(p), nkv = kv_bytes(p);
  return overlaps(out, nq, q, nq) || overlaps(out, nq, k, nkv) || overlaps(out, nq, v, nkv);
}

// The scatter writes both caches while it reads the fresh rows ([B, L, Hkv, D] each).
bool scatter_io_overlap(const ec_params& p, const void* kc, const void* vc, const void* kn, const void* vn) {
  const size_t n = kv_bytes(p);
  return overlaps(kc, n, vc, n) || overlaps(kc, n, kn, n) || overlaps(kc, n, vn, n) || overlaps(vc, n, kn, n) ||
         overlaps(vc, n, vn, n);
}

ec_status cuda_status(cudaError_t e) { return e == cudaSuccess ? EC_OK : EC_ERR_CUDA; }

// Shape checks common to the stages that need them. `what` selects the groups checked.
enum : int { kCheckDecode = 1, kCheckSelect = 2, kCheckAttn = 4 };

ec_status check_params(const ec_params* p, int what) {
  if (p == nullptr) return EC_ERR_INVALID_ARG;
  if (p->B < 1 || p->B > kMaxB || p->L < 1 || p->L > kMaxL) return EC_ERR_INVALID_ARG;
  if (has_scope(*p) && !(p->scope_lo >= 0 && p->scope_lo < p->scope_hi && p->scope_hi <= p->L))
    return EC_ERR_INVALID_ARG;
  if (what & kCheckDecode) {
    if (p->V < 1 || p->V > kMaxV) return EC_ERR_INVALID_ARG;
    if (p->logits_dtype != EC_F32 && p->logits_dtype != EC_BF16) return EC_ERR_INVALID_ARG;
  }
  if (what & kCheckSelect) {
    if (p->C_max < 1 || p->C_max > std::min(p->L, kMaxCmax)) return EC_ERR_INVALID_ARG;
    if (p->k < 1 || p->k > p->L) return EC_ERR_INVALID_ARG;
    if (p->n_dec < 1 || p->n_dec > p->C_max) return EC_ERR_INVALID_ARG;
    if (p->tau != p->tau) return EC_ERR_INVALID_ARG;  // NaN threshold
    if (!(p->conf_threshold <= 1.f)) return EC_ERR_INVALID_ARG;  // NaN, or above any probability
  }
  if (what & kCheckAttn) {
    if (p->Hq < 1 || p->Hkv < 1 || p->Hq % p->Hkv != 0) return EC_ERR_INVALID_ARG;
    if (p->Hq / p->Hkv > 128) return EC_ERR_UNSUPPORTED;
    if (p->D != 64 && p->D != 128) return EC_ERR_UNSUPPORTED;
    const int64_t g = p->Hq / p->Hkv;
    const int64_t nr = 128 / g;
    const int64_t tiles = static_cast<int64_t>(p->B) * p->Hkv * ((p->L + nr - 1) / nr);
    if (tiles > (1ll << 30)) return EC_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(p->Hq) * p->D * p->L * p->B > (1ll << 40)) return EC_ERR_UNSUPPORTED;
  }
  return EC_OK;
}

ec_status check_state(const ec_state* st) {
  if (st == nullptr) return EC_ERR_INVALID_ARG;
  if (!st->tokens || !st->mask || !st->ring || !st->ring_head || !st->ring_count || !st->dec_pos || !st->E ||
      !st->flag || !st->idx || !st->R)
    return EC_ERR_INVALID_ARG;
  if (!aligned16(st->mask)) return EC_ERR_INVALID_ARG;  // the mask row is read with 16-byte loads
  return EC_OK;
}

// ---- ec_step workspace layout --------------------------------------------------------
struct StepLayout {
  size_t k1, ids, ent, conf, qbuf, attn, total;
};

StepLayout step_layout(const ec_params& p) {
  StepLayout s{};
  const size_t rows = static_cast<size_t>(p.B) * p.C_max;
  size_t off = 0;
  s.k1 = off;
  off += align_up(entropy_workspace_bytes(static_cast<int32_t>(rows), p.V, p.logits_dtype), 256);
  s.ids = off;
  off += align_up(rows * 4, 256);
  s.ent = off;
  off += align_up(rows * 4, 256);
  s.conf = off;
  off += align_up(rows * 4, 256);
  s.qbuf = off;
  off += align_up(static_cast<size_t>(p.B) * p.L * p.Hq * p.D * 2, 256);
  s.attn = off;
  off += align_up(attention_workspace_bytes(p), 256);
  s.total = off;
  return s;
}

// One CTA: thread 0 waits for a phase of a barrier on which nothing ever arrives.
__global__ void selftest_wait_kernel(int32_t* dev_err, uint64_t limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort;
  if (threadIdx.x == 0) {
    abort = 0;
    ec::mbar_init(&bar, 1);
    ec::fence_mbar_init();
    ec::mbar_wait_bounded(&bar, 0, &abort, dev_err, limit_ns);
  }
}

}  // namespace

extern "C" {

const char* ec_status_string(ec_status st) {
  switch (st) {
    case EC_OK: return "EC_OK";
    case EC_ERR_INVALID_ARG: return "EC_ERR_INVALID_ARG";
    case EC_ERR_UNSUPPORTED: return "EC_ERR_UNSUPPORTED";
    case EC_ERR_CUDA: return "EC_ERR_CUDA";
    case EC_ERR_DEVICE_CHECK: return "EC_ERR_DEVICE_CHECK";
    case EC_ERR_TIMEOUT: return "EC_ERR_TIMEOUT";
    default: return "EC_ERR_UNKNOWN";
  }
}

int32_t ec_version(void) { return 100; }

ec_status ec_read_device_error(const int32_t* dev_err, int32_t* host_word, ec_stream_t stream) {
  if (dev_err == nullptr) return EC_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t w = 0;
  cudaError_t e = cudaMemcpyAsync(&w, dev_err, sizeof(w), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return EC_ERR_CUDA;
  if (host_word != nullptr) *host_word = w;
  if (w == 0) return EC_OK;
  return (w & EC_DEVERR_TIMEOUT) ? EC_ERR_TIMEOUT : EC_ERR_DEVICE_CHECK;
}

ec_status ec_selftest_bounded_wait(int32_t* dev_err, uint64_t limit_ns, ec_stream_t stream) {
  if (dev_err == nullptr || limit_ns < 1 || limit_ns > 10000000000ull) return EC_ERR_INVALID_ARG;
  selftest_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(dev_err, limit_ns);
  return cuda_status(cudaGetLastError());
}

// ---- (a) ----------------------------------------------------------------------------------
size_t ec_entropy_decode_workspace_size(int32_t n_rows, int32_t V, int32_t dtype) {
  if (n_rows < 0 || V < 1 || V > kMaxV || (dtype != EC_F32 && dtype != EC_BF16)) return 0;
  return entropy_workspace_bytes(n_rows, V, dtype);
}

ec_status ec_entropy_decode(const void* logits, int64_t row_stride, int32_t n_rows, int32_t V, int32_t dtype,
                            int32_t* ids, float* entropy, float* log_conf, void* ws, size_t ws_bytes,
                            ec_stream_t stream) {
  if (dtype != EC_F32 && dtype != EC_BF16) return EC_ERR_INVALID_ARG;
  if (V < 1 || V > kMaxV || n_rows < 0 || row_stride < V) return EC_ERR_INVALID_ARG;
  if (n_rows == 0) return EC_OK;
  const int64_t esize = dtype == EC_F32 ? 4 : 2;
  if ((row_stride * esize) % 16 != 0) return EC_ERR_INVALID_ARG;
  if (!logits || !ids || !entropy || !log_conf || !aligned16(logits)) return EC_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n_rows) * entropy_num_chunks(V, dtype) > INT32_MAX) return EC_ERR_UNSUPPORTED;
  const size_t need = entropy_workspace_bytes(n_rows, V, dtype);
  if (ws == nullptr || ws_bytes < need || !aligned16(ws)) return EC_ERR_INVALID_ARG;
  return cuda_status(launch_entropy_decode(logits, row_stride, n_rows, V, dtype, ids, entropy, log_conf, ws,
                                           nullptr, 1, true, false, static_cast<cudaStream_t>(stream)));
}

// ---- (a) from the hidden states ----------------------------------------------------------------
size_t ec_lm_head_entropy_workspace_size(int32_t n_rows) {
  if (n_rows < 1 || n_rows > lm_head_max_rows()) return 0;
  return lm_head_workspace_bytes(n_rows);
}

ec_status ec_lm_head_entropy(const void* hidden, const void* weight, int32_t n_rows, int32_t d_model, int32_t V,
                             int32_t* ids, float* entropy, float* log_conf, void* ws, size_t ws_bytes,
                             ec_stream_t stream) {
  if (n_rows < 1 || n_rows > lm_head_max_rows()) return EC_ERR_INVALID_ARG;
  if (d_model < 64 || d_model > 65536 || d_model % 64 != 0 || V < 1 || V > kMaxV) return EC_ERR_INVALID_ARG;
  if (!hidden || !weight || !ids || !entropy || !log_conf || !ws) return EC_ERR_INVALID_ARG;
  if (!aligned16(hidden) || !aligned16(weight) || !aligned16(ws)) return EC_ERR_INVALID_ARG;
  if (ws_bytes < lm_head_workspace_bytes(n_rows)) return EC_ERR_INVALID_ARG;
  return cuda_status(launch_lm_head_entropy(hidden, weight, n_rows, d_model, V, ids, entropy, log_conf, ws, nullptr,
                                            static_cast<cudaStream_t>(stream)));
}

// ---- (b)+(c) --------------------------------------------------------------------------------
ec_status ec_select_recompute(const ec_params* p, const ec_state* st, const int32_t* cand_pos,
                              const int32_t* cand_count, const int32_t* ids, const float* entropy,
                              const float* log_conf, ec_stream_t stream) {
  ec_status r = check_params(p, kCheckSelect);
  if (r != EC_OK) return r;
  if ((r = check_state(st)) != EC_OK) return r;
  if (!cand_pos || !cand_count || !ids || !entropy || !log_conf) return EC_ERR_INVALID_ARG;
  return cuda_status(launch_select_recompute(*p, *st, cand_pos, cand_count, ids, entropy, log_conf, false, nullptr,
                                             0, static_cast<cudaStream_t>(stream)));
}

// ---- candidates for block-wise / sliding-window decoding -----------------------------------------
ec_status ec_candidates(const ec_params* p, const ec_state* st, int32_t mode, int32_t start, int32_t width,
                        int32_t* cand_pos, int32_t* cand_count, ec_stream_t stream) {
  ec_status r = check_params(p, kCheckSelect);
  if (r != EC_OK) return r;
  if (st == nullptr || st->mask == nullptr || !cand_pos || !cand_count) return EC_ERR_INVALID_ARG;
  if (mode != EC_CAND_BLOCK && mode != EC_CAND_SLIDING) return EC_ERR_INVALID_ARG;
  if (start < 0 || start >= p->L || width < 1 || width > p->C_max) return EC_ERR_INVALID_ARG;
  return cuda_status(launch_candidates(*p, st->mask, mode, start, width, cand_pos, cand_count,
                                       static_cast<cudaStream_t>(stream)));
}

// ---- (c) scatter ------------------------------------------------------------------------------
ec_status ec_kv_scatter(const ec_params* p, void* k_cache, void* v_cache, const void* k_new, const void* v_new,
                        int32_t src_by_position, const int32_t* idx, const int32_t* R, int32_t* dev_err,
                        ec_stream_t stream) {
  if (p == nullptr) return EC_ERR_INVALID_ARG;
  if (p->B < 1 || p->B > kMaxB || p->L < 1 || p->L > kMaxL || p->Hkv < 1) return EC_ERR_INVALID_ARG;
  if (p->D != 64 && p->D != 128) return EC_ERR_UNSUPPORTED;
  if (src_by_position != 0 && src_by_position != 1) return EC_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !k_new || !v_new || !idx || !R) return EC_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_new) || !aligned16(v_new))
    return EC_ERR_INVALID_ARG;
  if (scatter_io_overlap(*p, k_cache, v_cache, k_new, v_new)) return EC_ERR_INVALID_ARG;
  return cuda_status(launch_kv_scatter(*p, k_cache, v_cache, k_new, v_new, src_by_position, idx, R, nullptr,
                                       nullptr, dev_err, static_cast<cudaStream_t>(stream)));
}

// ---- (d) ----------------------------------------------------------------------------------------
size_t ec_partial_attention_workspace_size(const ec_params* p) {
  if (check_params(p, kCheckAttn) != EC_OK) return 0;
  return attention_workspace_bytes(*p);
}

ec_status ec_dense_attention(const ec_params* p, const void* q, const void* k_cache, const void* v_cache,
                             float scale, void* out, int32_t* dev_err, ec_stream_t stream) {
  ec_status r = check_params(p, kCheckAttn);
  if (r != EC_OK) return r;
  if (!q || !k_cache || !v_cache || !out) return EC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return EC_ERR_INVALID_ARG;
  if (!(scale == scale)) return EC_ERR_INVALID_ARG;
  if (p->D != 128) return EC_ERR_UNSUPPORTED;
  if (attention_io_overlap(*p, q, k_cache, v_cache, out)) return EC_ERR_INVALID_ARG;
  ec_status st = EC_OK;
  launch_dense_attention_tiles(*p, q, k_cache, v_cache, scale, out, dev_err, static_cast<cudaStream_t>(stream), &st);
  return st;
}

ec_status ec_partial_attention(const ec_params* p, const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* R, float scale, void* out, void* ws, size_t ws_bytes,
                               int32_t* dev_err, ec_stream_t stream) {
  ec_status r = check_params(p, kCheckAttn);
  if (r != EC_OK) return r;
  if (!q || !k_cache || !v_cache || !R || !out || !ws) return EC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(ws))
    return EC_ERR_INVALID_ARG;
  if (ws_bytes < attention_workspace_bytes(*p)) return EC_ERR_INVALID_ARG;
  if (!(scale == scale)) return EC_ERR_INVALID_ARG;
  if (attention_io_overlap(*p, q, k_cache, v_cache, out)) return EC_ERR_INVALID_ARG;
  ec_status st = EC_OK;
  launch_partial_attention(*p, q, k_cache, v_cache, R, scale, out, ws, dev_err, false, static_cast<cudaStream_t>(stream),
                           &st);
  return st;
}

// ---- 8-bit cache, shared prefix ------------------------------------------------------------------
namespace {

size_t int_bytes(size_t n) { return n * sizeof(int32_t); }
// Sizes and indices are read, and the error word is written, as whole 32-bit words.
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t kv_extent(const ec_params& p, const ec_kv& c, int32_t B) {
  return static_cast<size_t>(B) * c.len * p.Hkv * p.D * (c.dtype == EC_BF16 ? 2 : 1);
}
size_t exp_extent(const ec_params& p, const ec_kv& c, int32_t B) {
  return c.dtype == EC_BF16 ? 0 : static_cast<size_t>(B) * p.Hkv * quant_exp_stride(c.len);
}

// The cache `c` of len positions has a type, pointers and alignment that the kernels take.
ec_status check_kv(const ec_kv* c, int32_t len) {
  if (c == nullptr || c->len != len) return EC_ERR_INVALID_ARG;
  if (c->dtype != EC_BF16 && c->dtype != EC_E4M3) return EC_ERR_INVALID_ARG;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return EC_ERR_INVALID_ARG;
  if (c->dtype == EC_E4M3 && (!c->k_exp || !c->v_exp || !aligned16(c->k_exp) || !aligned16(c->v_exp)))
    return EC_ERR_INVALID_ARG;
  return EC_OK;
}

ec_status check_quant_rows(const ec_params* p, const ec_kv* c) {
  if (p == nullptr) return EC_ERR_INVALID_ARG;
  if (p->B < 1 || p->B > kMaxB || p->L < 1 || p->L > kMaxL || p->Hkv < 1 || p->Hkv > 65536) return EC_ERR_INVALID_ARG;
  if (p->D != 64 && p->D != 128) return EC_ERR_UNSUPPORTED;
  // a sequence's rows are counted in 32 bits (more would not fit the device)
  if (2ll * p->L * p->Hkv > INT32_MAX) return EC_ERR_UNSUPPORTED;
  const ec_status r = check_kv(c, p->L);
  if (r != EC_OK) return r;
  return c->dtype == EC_E4M3 ? EC_OK : EC_ERR_UNSUPPORTED;
}

ec_status cached_attention(const ec_params* p, const void* q, const ec_kv* prefix, const ec_kv* cache,
                           const int32_t* R, const int32_t* kv_len, float scale, void* out, void* ws,
                           size_t ws_bytes, size_t ws_need, int32_t* dev_err, ec_stream_t stream) {
  ec_status r = check_kv(cache, p->L);
  if (r != EC_OK) return r;
  // rows of q are counted in 32 bits (more would not fit the device beside their output)
  if (static_cast<int64_t>(p->B) * p->L * p->Hq > INT32_MAX) return EC_ERR_UNSUPPORTED;
  if (!q || !R || !out || !ws || !aligned16(q) || !aligned16(out) || !aligned16(ws)) return EC_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale > 2e38f || ws_bytes < ws_need) return EC_ERR_INVALID_ARG;
  if (!aligned4(R) || !aligned4(kv_len) || !aligned4(dev_err)) return EC_ERR_INVALID_ARG;
  static const ec_kv none{};
  const ec_kv* pre = prefix != nullptr && prefix->len != 0 ? prefix : &none;
  if (pre->len != 0) {
    if (pre->len < 0 || pre->len > kMaxL) return EC_ERR_INVALID_ARG;
    if ((r = check_kv(pre, pre->len)) != EC_OK) return r;
    if (pre->dtype != cache->dtype) return EC_ERR_UNSUPPORTED;
  }
  const size_t n = kv_extent(*p, *cache, p->B), ne = exp_extent(*p, *cache, p->B);
  const size_t np = kv_extent(*p, *pre, 1), npe = exp_extent(*p, *pre, 1);
  const Extent written[] = {{out, q_bytes(*p)}, {ws, ws_need}};
  const Extent read[] = {{q, q_bytes(*p)},    {cache->k, n},      {cache->v, n},      {ne ? cache->k_exp : nullptr, ne},
                         {ne ? cache->v_exp : nullptr, ne},       {pre->k, np},       {pre->v, np},
                         {npe ? pre->k_exp : nullptr, npe},       {npe ? pre->v_exp : nullptr, npe},
                         {R, int_bytes(p->B)}, {kv_len, int_bytes(p->B)}};
  if (any_overlap(written, read)) return EC_ERR_INVALID_ARG;
  ec_status st = EC_OK;
  launch_cached_attention(*p, q, pre->len != 0 ? pre : nullptr, *cache, R, kv_len, scale, out, ws, dev_err,
                          static_cast<cudaStream_t>(stream), &st);
  return st;
}

}  // namespace

ec_status ec_kv_scatter_quant(const ec_params* p, const ec_kv* cache, const void* k_new, const void* v_new,
                              int32_t src_by_position, const int32_t* idx, const int32_t* R, int32_t* dev_err,
                              ec_stream_t stream) {
  const ec_status r = check_quant_rows(p, cache);
  if (r != EC_OK) return r;
  if (src_by_position != 0 && src_by_position != 1) return EC_ERR_INVALID_ARG;
  if (!k_new || !v_new || !idx || !R || !aligned16(k_new) || !aligned16(v_new)) return EC_ERR_INVALID_ARG;
  if (!aligned4(idx) || !aligned4(R) || !aligned4(dev_err)) return EC_ERR_INVALID_ARG;
  const size_t n = kv_extent(*p, *cache, p->B), ne = exp_extent(*p, *cache, p->B);
  const Extent written[] = {{cache->k, n}, {cache->v, n}, {cache->k_exp, ne}, {cache->v_exp, ne}};
  const Extent read[] = {{k_new, kv_bytes(*p)}, {v_new, kv_bytes(*p)}, {R, int_bytes(p->B)},
                         {idx, int_bytes(static_cast<size_t>(p->B) * p->L)}};
  if (any_overlap(written, read)) return EC_ERR_INVALID_ARG;
  return cuda_status(launch_kv_scatter_quant(*p, *cache, k_new, v_new, src_by_position, idx, R, dev_err,
                                             static_cast<cudaStream_t>(stream)));
}

ec_status ec_kv_gather_quant(const ec_params* p, const ec_kv* cache, const int32_t* idx, const int32_t* R,
                             void* k_out, void* v_out, int32_t* dev_err, ec_stream_t stream) {
  const ec_status r = check_quant_rows(p, cache);
  if (r != EC_OK) return r;
  if (!R || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return EC_ERR_INVALID_ARG;
  if (!aligned4(idx) || !aligned4(R) || !aligned4(dev_err)) return EC_ERR_INVALID_ARG;
  const size_t n = kv_extent(*p, *cache, p->B), ne = exp_extent(*p, *cache, p->B);
  const Extent written[] = {{k_out, kv_bytes(*p)}, {v_out, kv_bytes(*p)}};
  const Extent read[] = {{cache->k, n}, {cache->v, n}, {cache->k_exp, ne}, {cache->v_exp, ne}, {R, int_bytes(p->B)},
                         {idx, int_bytes(static_cast<size_t>(p->B) * p->L)}};
  if (any_overlap(written, read)) return EC_ERR_INVALID_ARG;
  return cuda_status(launch_kv_gather_quant(*p, *cache, idx, R, k_out, v_out, dev_err, static_cast<cudaStream_t>(stream)));
}

size_t ec_partial_attention_quant_workspace_size(const ec_params* p) {
  return check_params(p, kCheckAttn) != EC_OK ? 0 : cached_attention_workspace_bytes(*p, false);
}

ec_status ec_partial_attention_quant(const ec_params* p, const void* q, const ec_kv* cache, const int32_t* R,
                                     const int32_t* kv_len, float scale, void* out, void* ws, size_t ws_bytes,
                                     int32_t* dev_err, ec_stream_t stream) {
  const ec_status r = check_params(p, kCheckAttn);
  if (r != EC_OK) return r;
  if (cache != nullptr && cache->dtype == EC_BF16) return EC_ERR_UNSUPPORTED;
  return cached_attention(p, q, nullptr, cache, R, kv_len, scale, out, ws, ws_bytes,
                          cached_attention_workspace_bytes(*p, false), dev_err, stream);
}

size_t ec_prefix_attention_workspace_size(const ec_params* p) {
  return check_params(p, kCheckAttn) != EC_OK ? 0 : cached_attention_workspace_bytes(*p, true);
}

ec_status ec_prefix_attention(const ec_params* p, const void* q, const ec_kv* prefix, const ec_kv* cache,
                              const int32_t* R, const int32_t* kv_len, float scale, void* out, void* ws,
                              size_t ws_bytes, int32_t* dev_err, ec_stream_t stream) {
  const ec_status r = check_params(p, kCheckAttn);
  if (r != EC_OK) return r;
  return cached_attention(p, q, prefix, cache, R, kv_len, scale, out, ws, ws_bytes,
                          cached_attention_workspace_bytes(*p, true), dev_err, stream);
}

// ---- caches in pages -------------------------------------------------------------------------------
namespace {

size_t page_bytes(const ec_params& p, const ec_paged_kv& c) { return static_cast<size_t>(c.page_size) * p.Hkv * p.D * 2; }
size_t pool_extent(const ec_params& p, const ec_paged_kv& c) {
  return static_cast<size_t>(c.n_pages - 1) * c.page_stride * 2 + page_bytes(p, c);
}
size_t table_extent(const ec_params& p, const ec_paged_kv& c) {
  const size_t row = (static_cast<size_t>(p.L) + c.page_size - 1) / c.page_size;
  return (static_cast<size_t>(p.B - 1) * c.table_stride + row) * sizeof(int32_t);
}
// The pages of K and of V share no byte: apart, or page by page in one pool.
bool pools_apart(const ec_params& p, const ec_paged_kv& c) {
  const size_t n = pool_extent(p, c);
  if (!overlaps(c.k, n, c.v, n)) return true;
  const uintptr_t a = reinterpret_cast<uintptr_t>(c.k), b = reinterpret_cast<uintptr_t>(c.v);
  const size_t off = (a < b ? b - a : a - b) % (static_cast<size_t>(c.page_stride) * 2), page = page_bytes(p, c);
  return off >= page && off + page <= static_cast<size_t>(c.page_stride) * 2;
}

ec_status check_pages(const ec_params& p, const ec_paged_kv* c, int32_t rows_max) {
  if (c == nullptr || rows_max < 1 || rows_max > p.L) return EC_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0) return EC_ERR_UNSUPPORTED;
  if (c->n_pages < 1 || !c->k || !c->v || !c->table) return EC_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->table)) return EC_ERR_INVALID_ARG;
  if (c->page_stride % 8 != 0 || c->page_stride < static_cast<int64_t>(c->page_size) * p.Hkv * p.D) return EC_ERR_INVALID_ARG;
  // bytes to any page in 40 bits, as tensor maps count them
  if (c->page_stride >= (1ll << 36) || c->page_stride * 2 > (1ll << 40) / c->n_pages) return EC_ERR_UNSUPPORTED;
  if (c->table_stride < 1 || c->table_stride > (1ll << 31) || c->table_stride * c->page_size < p.L) return EC_ERR_INVALID_ARG;
  return pools_apart(p, *c) ? EC_OK : EC_ERR_INVALID_ARG;
}

// Strides of rows of `width` elements, and the bytes that they span.
bool check_rows(const ec_params& p, const ec_rows& x, int32_t rows_max, int64_t width, size_t* bytes) {
  if (!x.x || !aligned16(x.x) || x.batch_stride < 0 || x.row_stride < 0) return false;
  if (x.batch_stride % 8 != 0 || x.row_stride % 8 != 0 || x.batch_stride > (1ll << 40) || x.row_stride > (1ll << 36)) return false;
  if (rows_max > 1 && x.row_stride < width) return false;
  *bytes = (static_cast<size_t>(p.B - 1) * x.batch_stride + static_cast<size_t>(rows_max - 1) * x.row_stride + width) * 2;
  return true;
}

size_t idx_extent(const ec_params& p, int64_t stride, int32_t rows_max) {
  return (static_cast<size_t>(p.B - 1) * stride + rows_max) * sizeof(int32_t);
}
bool check_places(const ec_params& p, const int32_t* idx, int64_t stride, const int32_t* start, int32_t rows_max) {
  if (idx != nullptr && (start != nullptr || stride < rows_max || stride > (1ll << 31))) return false;
  return aligned4(idx) && aligned4(start);
}

ec_status paged_attention(const ec_params* p, int32_t rows_max, const void* q, const ec_paged_kv* c, const RowPlaces& at,
                          const Window* window, const int32_t* R, const int32_t* kv_len, float scale, void* out, void* ws,
                          size_t ws_bytes, int32_t* dev_err, ec_stream_t stream) {
  ec_status r = check_params(p, kCheckAttn);
  if (r != EC_OK) return r;
  if ((r = check_pages(*p, c, rows_max)) != EC_OK) return r;
  const int64_t heads = static_cast<int64_t>(p->B) * rows_max * p->Hq;  // rows of q, counted in 32 bits
  if (heads > INT32_MAX) return EC_ERR_UNSUPPORTED;
  const int64_t tiles = (static_cast<int64_t>(rows_max) * (p->Hq / p->Hkv) + 127) / 128, blocks = p->L / 128 + 2;
  if (p->B * static_cast<int64_t>(p->Hkv) * tiles > (1ll << 30) / blocks) return EC_ERR_UNSUPPORTED;  // steps, in 32 bits
  if (!q || !R || !out || !ws || !aligned16(q) || !aligned16(out) || !aligned16(ws)) return EC_ERR_INVALID_ARG;
  const size_t ws_need = paged_attention_workspace_bytes(*p, rows_max);
  if (!(scale > 0.f) || scale > 2e38f || ws_bytes < ws_need) return EC_ERR_INVALID_ARG;
  if (!aligned4(R) || !aligned4(kv_len) || !aligned4(dev_err)) return EC_ERR_INVALID_ARG;
  if (!check_places(*p, at.idx, at.stride, at.start, rows_max)) return EC_ERR_INVALID_ARG;
  const size_t n = static_cast<size_t>(heads) * p->D * 2, pool = pool_extent(*p, *c);
  const Extent written[] = {{out, n}, {ws, ws_need}};
  const Extent read[] = {{q, n},          {c->k, pool},
                         {c->v, pool},    {c->table, table_extent(*p, *c)},
                         {R, int_bytes(p->B)}, {kv_len, int_bytes(p->B)},
                         {at.idx, at.idx ? idx_extent(*p, at.stride, rows_max) : 0}, {at.start, int_bytes(p->B)}};
  if (any_overlap(written, read)) return EC_ERR_INVALID_ARG;
  ec_status st = EC_OK;
  launch_paged_attention(*p, rows_max, q, *c, at, window, R, kv_len, scale, out, ws, dev_err,
                         static_cast<cudaStream_t>(stream), &st);
  return st;
}

}  // namespace

ec_status ec_kv_append_paged(const ec_params* p, const ec_paged_kv* cache, int32_t rows_max, const ec_rows* k_new,
                             const ec_rows* v_new, const ec_rows* q_new, void* q_out, const float* rope_cos,
                             const float* rope_sin, const int32_t* idx, int64_t idx_stride, const int32_t* start,
                             const int32_t* R, int32_t* dev_err, ec_stream_t stream) {
  ec_status r = check_params(p, kCheckAttn);
  if (r != EC_OK) return r;
  if ((r = check_pages(*p, cache, rows_max)) != EC_OK) return r;
  if (!k_new || !v_new || !R || (q_new != nullptr) != (q_out != nullptr) || (rope_cos != nullptr) != (rope_sin != nullptr))
    return EC_ERR_INVALID_ARG;
  const int64_t kv_width = static_cast<int64_t>(p->Hkv) * p->D, q_width = static_cast<int64_t>(p->Hq) * p->D;
  if (kv_width > (1 << 26) || q_width > (1 << 26)) return EC_ERR_UNSUPPORTED;  // a row's pieces are counted in 32 bits
  size_t nk = 0, nv = 0, nq = 0;
  if (!check_rows(*p, *k_new, rows_max, kv_width, &nk) || !check_rows(*p, *v_new, rows_max, kv_width, &nv)) return EC_ERR_INVALID_ARG;
  if (q_new && (!check_rows(*p, *q_new, rows_max, q_width, &nq) || !aligned16(q_out))) return EC_ERR_INVALID_ARG;
  if (!aligned16(rope_cos) || !aligned16(rope_sin) || !aligned4(R) || !aligned4(dev_err)) return EC_ERR_INVALID_ARG;
  if (!check_places(*p, idx, idx_stride, start, rows_max)) return EC_ERR_INVALID_ARG;
  const size_t pool = pool_extent(*p, *cache), table = static_cast<size_t>(p->L) * p->D / 2 * sizeof(float);
  const size_t no = q_out ? static_cast<size_t>(p->B) * rows_max * q_width * 2 : 0;
  const Extent read[] = {{k_new->x, nk},  {v_new->x, nv}, {q_new ? q_new->x : nullptr, nq}, {rope_cos, table}, {rope_sin, table},
                         {idx, idx ? idx_extent(*p, idx_stride, rows_max) : 0}, {start, int_bytes(p->B)}, {R, int_bytes(p->B)},
                         {cache->table, table_extent(*p, *cache)}};
  const Extent pools[] = {{cache->k, pool}}, pools_v[] = {{cache->v, pool}}, rotated[] = {{q_out, no}};
  const Extent caches[] = {{cache->k, pool}, {cache->v, pool}};
  if (any_overlap(pools, read) || any_overlap(pools_v, read)) return EC_ERR_INVALID_ARG;
  if (no != 0 && (any_overlap(rotated, read) || any_overlap(rotated, caches))) return EC_ERR_INVALID_ARG;
  return cuda_status(launch_kv_append_paged(*p, *cache, rows_max, *k_new, *v_new, q_new ? *q_new : ec_rows{}, q_out, rope_cos,
                                            rope_sin, {idx, idx_stride, start}, R, dev_err, static_cast<cudaStream_t>(stream)));
}

size_t ec_paged_attention_workspace_size(const ec_params* p, int32_t rows_max) {
  if (check_params(p, kCheckAttn) != EC_OK || rows_max < 1 || rows_max > p->L) return 0;
  return paged_attention_workspace_bytes(*p, rows_max);
}

ec_status ec_paged_attention(const ec_params* p, int32_t rows_max, const void* q, const ec_paged_kv* cache, const int32_t* R,
                             const int32_t* kv_len, float scale, void* out, void* ws, size_t ws_bytes, int32_t* dev_err,
                             ec_stream_t stream) {
  return paged_attention(p, rows_max, q, cache, {}, nullptr, R, kv_len, scale, out, ws, ws_bytes, dev_err, stream);
}

ec_status ec_paged_window_attention(const ec_params* p, int32_t rows_max, const void* q, const ec_paged_kv* cache,
                                    const int32_t* idx, int64_t idx_stride, const int32_t* start, const int32_t* R,
                                    const int32_t* kv_len, int32_t left, int32_t right, int32_t sinks, float scale, void* out,
                                    void* ws, size_t ws_bytes, int32_t* dev_err, ec_stream_t stream) {
  if (left < -1 || right < -1 || sinks < 0) return EC_ERR_INVALID_ARG;
  const Window w{left < 0 ? kMaxL : std::min(left, kMaxL), right < 0 ? kMaxL : std::min(right, kMaxL), std::min(sinks, kMaxL)};
  return paged_attention(p, rows_max, q, cache, {idx, idx_stride, start}, &w, R, kv_len, scale, out, ws, ws_bytes, dev_err, stream);
}

// ---- the partial forward of one layer --------------------------------------------------------------
namespace {
ec_status check_layer(const ec_params* p, const ec_layer* w) {
  ec_status r = check_params(p, kCheckAttn);
  if (r != EC_OK) return r;
  if (w == nullptr) return EC_ERR_INVALID_ARG;
  const int64_t d = static_cast<int64_t>(p->Hq) * p->D, kvf = static_cast<int64_t>(p->Hkv) * p->D;
  if (d % 128 != 0 || d > 8192 || kvf % 128 != 0) return EC_ERR_UNSUPPORTED;
  if (w->d_ff < 64 || w->d_ff % 64 != 0 || w->d_ff > 65536) return EC_ERR_INVALID_ARG;
  if (!(w->eps > 0.f)) return EC_ERR_INVALID_ARG;
  const void* ptrs[] = {w->wq, w->wk, w->wv, w->wo, w->wg, w->wu, w->wd, w->gamma1, w->gamma2, w->rope_cos, w->rope_sin};
  for (const void* q : ptrs)
    if (q == nullptr || !aligned16(q)) return EC_ERR_INVALID_ARG;
  return EC_OK;
}
}  // namespace

size_t ec_layer_forward_workspace_size(const ec_params* p, int32_t d_ff) {
  if (check_params(p, kCheckAttn) != EC_OK || d_ff < 64 || d_ff % 64 != 0) return 0;
  return layer_forward_workspace_bytes(*p, d_ff);
}

ec_status ec_layer_forward(const ec_params* p, const ec_layer* w, const int32_t* idx, const int32_t* R,
                           const void* x_src, void* k_cache, void* v_cache, void* y, void* ws, size_t ws_bytes,
                           int32_t* dev_err, ec_stream_t stream) {
  ec_status r = check_layer(p, w);
  if (r != EC_OK) return r;
  if (!idx || !R || !x_src || !k_cache || !v_cache || !y || !ws) return EC_ERR_INVALID_ARG;
  if (!aligned16(x_src) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(y) || !aligned16(ws))
    return EC_ERR_INVALID_ARG;
  if (ws_bytes < layer_forward_workspace_bytes(*p, w->d_ff)) return EC_ERR_INVALID_ARG;
  ec_status st = EC_OK;
  launch_layer_forward(*p, *w, idx, R, x_src, k_cache, v_cache, y, ws, dev_err, static_cast<cudaStream_t>(stream), &st);
  return st;
}

ec_status ec_rope_table(int32_t L, int32_t D, float theta, float* rope_cos, float* rope_sin, ec_stream_t stream) {
  if (L < 1 || L > kMaxL || D < 2 || D > 256 || D % 2 != 0 || !(theta > 0.f)) return EC_ERR_INVALID_ARG;
  if (!rope_cos || !rope_sin) return EC_ERR_INVALID_ARG;
  return cuda_status(launch_rope_table(L, D, theta, rope_cos, rope_sin, static_cast<cudaStream_t>(stream)));
}

// ---- measurement aid -----------------------------------------------------------------------------
ec_status ec_read_floor(const void* buf, size_t bytes, uint32_t* sink, ec_stream_t stream) {
  if (buf == nullptr || sink == nullptr || !aligned16(buf) || bytes % 16 != 0 || bytes > (size_t(1) << 40))
    return EC_ERR_INVALID_ARG;
  return cuda_status(launch_read_floor(buf, bytes, sink, static_cast<cudaStream_t>(stream)));
}

// ---- whole step ---------------------------------------------------------------------------------
size_t ec_step_workspace_size(const ec_params* p) {
  if (check_params(p, kCheckDecode | kCheckSelect | kCheckAttn) != EC_OK) return 0;
  return step_layout(*p).total;
}

ec_status ec_step(const ec_params* p, const ec_state* st, const void* logits, const int32_t* cand_pos,
                  const int32_t* cand_count, int32_t n_layers, void* const* k_cache, void* const* v_cache,
                  const void* const* k_src, const void* const* v_src, const void* const* q_src, void* const* out,
                  float scale, void* ws, size_t ws_bytes, ec_stream_t stream) {
  ec_status r = check_params(p, kCheckDecode | kCheckSelect | kCheckAttn);
  if (r != EC_OK) return r;
  if ((r = check_state(st)) != EC_OK) return r;
  const int64_t esize = p->logits_dtype == EC_F32 ? 4 : 2;
  if ((static_cast<int64_t>(p->V) * esize) % 16 != 0) return EC_ERR_INVALID_ARG;
  if (!logits || !aligned16(logits) || !cand_pos || !cand_count || !ws || !aligned16(ws)) return EC_ERR_INVALID_ARG;
  if (n_layers < 0 || (n_layers > 0 && (!k_cache || !v_cache || !k_src || !v_src || !q_src || !out)))
    return EC_ERR_INVALID_ARG;
  if (!(scale == scale)) return EC_ERR_INVALID_ARG;
  for (int32_t l = 0; l < n_layers; ++l) {
    if (!k_cache[l] || !v_cache[l] || !k_src[l] || !v_src[l] || !q_src[l] || !out[l]) return EC_ERR_INVALID_ARG;
    if (!aligned16(k_cache[l]) || !aligned16(v_cache[l]) || !aligned16(k_src[l]) || !aligned16(v_src[l]) ||
        !aligned16(q_src[l]) || !aligned16(out[l]))
      return EC_ERR_INVALID_ARG;
    if (scatter_io_overlap(*p, k_cache[l], v_cache[l], k_src[l], v_src[l]) ||
        attention_io_overlap(*p, q_src[l], k_cache[l], v_cache[l], out[l]))
      return EC_ERR_INVALID_ARG;
  }
  const StepLayout lay = step_layout(*p);
  if (ws_bytes < lay.total) return EC_ERR_INVALID_ARG;
  char* w = static_cast<char*>(ws);
  auto* ids = reinterpret_cast<int32_t*>(w + lay.ids);
  auto* ent = reinterpret_cast<float*>(w + lay.ent);
  auto* conf = reinterpret_cast<float*>(w + lay.conf);
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  // stages (a)-(c): decode + entropy of the candidate rows, then the select stage
  cudaError_t e = launch_entropy_decode(logits, p->V, p->B * p->C_max, p->V, p->logits_dtype, ids, ent, conf,
                                        w + lay.k1, cand_count, p->C_max, false, true, s);
  // the decode kernel waits for every earlier kernel before it releases this one, so the select
  // kernel may stage the state before its own wait
  if (e == cudaSuccess)
    e = launch_select_recompute(*p, *st, cand_pos, cand_count, ids, ent, conf, true,
                                reinterpret_cast<const ChunkPartial*>(w + lay.k1), entropy_num_chunks(p->V, p->logits_dtype),
                                s);
  if (e != cudaSuccess) return EC_ERR_CUDA;
  // Entropies are non-negative (an empty decode set counts 0, a NaN counts as full), so with
  // tau < 0 the gate fires on every step. Without a scope every step then recomputes every
  // position in order (idx is the identity), and the attention is the dense one for every
  // sequence: the two-tile kernel reads the position-indexed queries where they are, and the
  // scatter kernel refreshes the cache only (no query gather).
  const bool always_full = p->tau < 0.f && !has_scope(*p) && p->D == 128;
  for (int32_t l = 0; l < n_layers; ++l) {
    e = launch_kv_scatter(*p, k_cache[l], v_cache[l], k_src[l], v_src[l], 1, st->idx, st->R,
                          always_full ? nullptr : q_src[l], always_full ? nullptr : w + lay.qbuf, st->dev_err, s);
    if (e != cudaSuccess) return EC_ERR_CUDA;
    ec_status as = EC_OK;
    if (always_full)
      launch_dense_attention_tiles(*p, q_src[l], k_cache[l], v_cache[l], scale, out[l], st->dev_err, s, &as);
    else
      launch_partial_attention(*p, w + lay.qbuf, k_cache[l], v_cache[l], st->R, scale, out[l], w + lay.attn,
                               st->dev_err, true, s, &as);
    if (as != EC_OK) return as;
  }
  return EC_OK;
}

}  // extern "C"
