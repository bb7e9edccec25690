// kv_quant.cu — the 8-bit K/V cache: quantising the fresh rows of the recompute set as they are
// written, and reading rows back as bf16. The counterparts of the bf16 refresh (kv_scatter.cu,
// EntropyCache, gist.science zh summary §2.2, partial forward); the row format is
// quant_common.cuh's. The pages keep the cache in the model's precision: the 8-bit cache has no
// counterpart there.
//
//   write: a = max_d |x_d|, e from a, code_d = e4m3(x_d 2^-e)       for K and V of each row
//   read:  x_d = bf16(code_d 2^e)                                    (exact)
//
// Both are bound by HBM (3 D + 1 bytes a row) or, for a partial step's few rows, by launch and
// one chain of dependent loads. The rows (recompute row, K or V, KV head) of a sequence stand in one
// line. A row's D values lie in D / 8 neighbouring lanes, 16 bytes of bf16 each, so both sides of the
// copy are full sectors; a thread loads its part of kRows rows before it works on any. The maxima
// of two rows share a register's halves, so a reduction step is one shuffle for both.
#include <algorithm>

#include "ec_common.cuh"
#include "ec_internal.h"
#include "quant_common.cuh"

namespace ec {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;  // rows in flight per thread

struct QuantArgs {
  int32_t L, Ls, Hkv;   // Ls: positions of an exponent row
  FastDiv div_2h;       // by 2 Hkv
  uint2 *k, *v;
  uint8_t *ke, *ve;
  const int32_t *idx, *R;
  int32_t* dev_err;
};

EC_DEV uint4 ld_stream(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// Rows of sequence b, 0 when R[b] is bad (reported once).
EC_DEV int checked_rows(const QuantArgs& a, int b) {
  const int r = __ldg(a.R + b);
  if (r >= 0 && r <= a.L) return r;
  if (blockIdx.x == 0 && threadIdx.x == 0) report_error(a.dev_err, EC_DEVERR_BAD_R);
  return 0;
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_scatter_quant_kernel(const __grid_constant__ QuantArgs a,
                                                                    const uint4* __restrict__ k_new,
                                                                    const uint4* __restrict__ v_new,
                                                                    int32_t src_by_position) {
  constexpr int kLanes = D / 8, kStep = kThreads / kLanes;  // lanes of a row; rows of a CTA per step
  const int b = blockIdx.y, lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  pdl_wait();
  pdl_launch_dependents();
  const int Rb = checked_rows(a, b);
  const int64_t rowL = static_cast<int64_t>(b) * a.L;
  const int n = Rb * 2 * a.Hkv;  // below 2^31
  for (int base = blockIdx.x * (kStep * kRows); base < n; base += gridDim.x * (kStep * kRows)) {
    uint4 x[kRows];
    int pos[kRows], head[kRows];  // head: of 2 Hkv, the K heads first
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int i = base + u * kStep + sub;
      x[u] = make_uint4(0, 0, 0, 0);
      pos[u] = -1;
      head[u] = 0;
      if (i >= n) continue;
      const int r = a.div_2h(i);
      head[u] = i - r * 2 * a.Hkv;
      const int p = __ldg(a.idx + rowL + r);
      // rows in recompute order ascend: a position that is not below its successor is a bad
      // (possibly repeated) one, whose codes and exponent two rows could write at once
      const bool bad = p < 0 || p >= a.L || (!src_by_position && r + 1 < Rb && p >= __ldg(a.idx + rowL + r + 1));
      if (bad && head[u] == 0) report_error(a.dev_err, EC_DEVERR_BAD_IDX);
      if (!src_by_position || !bad) {
        const int h = head[u] < a.Hkv ? head[u] : head[u] - a.Hkv;
        x[u] = ld_stream((head[u] < a.Hkv ? k_new : v_new) +
                         ((rowL + (src_by_position ? p : r)) * a.Hkv + h) * kLanes + lane);
      }
      pos[u] = bad ? -1 : p;
    }
    // largest magnitudes as bf16 bits (ordered like the values, NaN and infinity on top), of rows u
    // and u + 1 in the halves of a word
    uint32_t top[kRows / 2];
#pragma unroll
    for (int u = 0; u < kRows; u += 2) {
      uint32_t m[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        m[e] = __vmaxu2(__vmaxu2(x[u + e].x & 0x7FFF7FFFu, x[u + e].y & 0x7FFF7FFFu),
                        __vmaxu2(x[u + e].z & 0x7FFF7FFFu, x[u + e].w & 0x7FFF7FFFu));
      top[u / 2] = __vmaxu2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
    }
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1)
#pragma unroll
      for (int u = 0; u < kRows / 2; ++u) top[u] = __vmaxu2(top[u], __shfl_xor_sync(0xffffffffu, top[u], off));
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (pos[u] < 0) continue;
      const int byte = row_exp_byte(u & 1 ? top[u / 2] >> 16 : top[u / 2] & 0xFFFFu);
      uint2 code;
      if (byte < kExpTopByte) {
        const float f = quant_factor(byte);
        code = make_uint2(quantise4(x[u].x, x[u].y, f), quantise4(x[u].z, x[u].w, f));
      } else if (byte == kExpNaNByte) {
        code = make_uint2(kCodeNaN4, kCodeNaN4);
      } else {
        const float f = quant_factor(byte);
        code = make_uint2(cap_top_codes(quantise4(x[u].x, x[u].y, f)), cap_top_codes(quantise4(x[u].z, x[u].w, f)));
      }
      const bool is_k = head[u] < a.Hkv;
      const int h = is_k ? head[u] : head[u] - a.Hkv;
      (is_k ? a.k : a.v)[((rowL + pos[u]) * a.Hkv + h) * kLanes + lane] = code;
      if (lane == 0) (is_k ? a.ke : a.ve)[(static_cast<int64_t>(b) * a.Hkv + h) * a.Ls + pos[u]] = static_cast<uint8_t>(byte);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_gather_quant_kernel(const __grid_constant__ QuantArgs a,
                                                                   uint4* __restrict__ k_out,
                                                                   uint4* __restrict__ v_out) {
  constexpr int kLanes = D / 8, kStep = kThreads / kLanes;
  const int b = blockIdx.y, lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  pdl_wait();
  pdl_launch_dependents();
  const int Rb = checked_rows(a, b);
  const int64_t rowL = static_cast<int64_t>(b) * a.L;
  const int n = Rb * 2 * a.Hkv;
  for (int base = blockIdx.x * (kStep * kRows); base < n; base += gridDim.x * (kStep * kRows)) {
    uint2 code[kRows];
    int byte[kRows];
    int64_t to[kRows];  // the output row, complemented for V; kNone: none
    constexpr int64_t kNone = INT64_MIN;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int i = base + u * kStep + sub;
      to[u] = kNone;
      if (i >= n) continue;
      const int r = a.div_2h(i), head = i - r * 2 * a.Hkv;
      const int p = a.idx != nullptr ? __ldg(a.idx + rowL + r) : r;
      if (p < 0 || p >= a.L) {
        if (head == 0) report_error(a.dev_err, EC_DEVERR_BAD_IDX);
        continue;
      }
      const bool is_k = head < a.Hkv;
      const int h = is_k ? head : head - a.Hkv;
      code[u] = __ldg((is_k ? a.k : a.v) + ((rowL + p) * a.Hkv + h) * kLanes + lane);
      byte[u] = __ldg((is_k ? a.ke : a.ve) + (static_cast<int64_t>(b) * a.Hkv + h) * a.Ls + p);
      const int64_t row = (rowL + r) * a.Hkv + h;
      to[u] = is_k ? row : ~row;
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (to[u] == kNone) continue;
      uint4 y;
      if (byte[u] <= kExpOneFactor) {
        const uint32_t f = dequant_factor(byte[u]);
        dequantise4(code[u].x, f, y.x, y.y);
        dequantise4(code[u].y, f, y.z, y.w);
      } else {
        const DequantScale s = dequant_scale(byte[u]);
        dequantise4(code[u].x, s, y.x, y.y);
        dequantise4(code[u].y, s, y.z, y.w);
      }
      if (to[u] >= 0)
        k_out[to[u] * kLanes + lane] = y;
      else
        v_out[~to[u] * kLanes + lane] = y;
    }
  }
}

QuantArgs make_args(const ec_params& p, const ec_kv& c, const int32_t* idx, const int32_t* R, int32_t* dev_err) {
  QuantArgs a;
  a.L = p.L;
  a.Ls = static_cast<int32_t>(quant_exp_stride(p.L));
  a.Hkv = p.Hkv;
  a.div_2h.set(2 * p.Hkv);
  a.k = static_cast<uint2*>(c.k);
  a.v = static_cast<uint2*>(c.v);
  a.ke = c.k_exp;
  a.ve = c.v_exp;
  a.idx = idx;
  a.R = R;
  a.dev_err = dev_err;
  return a;
}

// CTAs over the rows of each sequence: eight per SM at most (R is known on the device only), striding.
cudaError_t quant_grid(const ec_params& p, dim3* grid) {
  int sms = 0;
  const cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  const int64_t cap = std::max<int64_t>(1, 8 * static_cast<int64_t>(sms) / p.B);
  const int64_t rows = static_cast<int64_t>(p.L) * 2 * p.Hkv, step = kThreads / (p.D / 8) * kRows;
  *grid = dim3(static_cast<unsigned>(std::min<int64_t>((rows + step - 1) / step, cap)), p.B);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv_scatter_quant(const ec_params& p, const ec_kv& c, const void* k_new, const void* v_new,
                                    int32_t src_by_position, const int32_t* idx, const int32_t* R, int32_t* dev_err,
                                    cudaStream_t s) {
  const QuantArgs a = make_args(p, c, idx, R, dev_err);
  dim3 grid;
  const cudaError_t e = quant_grid(p, &grid);
  if (e != cudaSuccess) return e;
  return launch_pdl(p.D == 128 ? kv_scatter_quant_kernel<128> : kv_scatter_quant_kernel<64>, grid, dim3(kThreads), 0, s,
                    a, static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), src_by_position);
}

cudaError_t launch_kv_gather_quant(const ec_params& p, const ec_kv& c, const int32_t* idx, const int32_t* R,
                                   void* k_out, void* v_out, int32_t* dev_err, cudaStream_t s) {
  const QuantArgs a = make_args(p, c, idx, R, dev_err);
  dim3 grid;
  const cudaError_t e = quant_grid(p, &grid);
  if (e != cudaSuccess) return e;
  return launch_pdl(p.D == 128 ? kv_gather_quant_kernel<128> : kv_gather_quant_kernel<64>, grid, dim3(kThreads), 0, s,
                    a, static_cast<uint4*>(k_out), static_cast<uint4*>(v_out));
}

}  // namespace ec
