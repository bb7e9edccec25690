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
// one chain of dependent loads. A row's D values lie in D / 8 neighbouring lanes, 16 bytes of bf16
// each, so the maximum is three or four shuffles and both sides of the copy are full sectors. A CTA
// takes the K and V rows of one or more positions (about 1024 vectors), and a thread loads
// kVec of them before it reduces any.
#include <algorithm>

#include "ec_common.cuh"
#include "ec_internal.h"
#include "quant_common.cuh"

namespace ec {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 4;  // 16-byte vectors of bf16 in flight per thread

struct QuantArgs {
  int32_t L, Ls, Hkv, row_vecs;  // Ls: positions of an exponent row; row_vecs: bf16 vectors of a position's K (= of its V)
  int32_t rows_per_pass;
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
  constexpr int kLanes = D / 8;
  const int b = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  const int Rb = checked_rows(a, b);
  const int64_t rowL = static_cast<int64_t>(b) * a.L;
  const int per_pos = 2 * a.row_vecs;
  for (int r0 = blockIdx.x * a.rows_per_pass; r0 < Rb; r0 += gridDim.x * a.rows_per_pass) {
    const int n = min(a.rows_per_pass, Rb - r0) * per_pos;
    for (int base = 0; base < n; base += kThreads * kVec) {
      uint4 x[kVec];
      int pos[kVec], vec[kVec];
#pragma unroll
      for (int u = 0; u < kVec; ++u) {
        const int i = base + u * kThreads + static_cast<int>(threadIdx.x);
        x[u] = make_uint4(0, 0, 0, 0);
        pos[u] = -1;
        vec[u] = 0;
        if (i >= n) continue;
        const int rl = i / per_pos;
        vec[u] = i - rl * per_pos;
        const int r = r0 + rl;
        const int p = __ldg(a.idx + rowL + r);
        // rows in recompute order ascend: a position that is not below its successor is a bad
        // (possibly repeated) one, whose codes and exponent two rows could write at once
        const bool bad = p < 0 || p >= a.L || (!src_by_position && r + 1 < Rb && p >= __ldg(a.idx + rowL + r + 1));
        if (bad && vec[u] == 0) report_error(a.dev_err, EC_DEVERR_BAD_IDX);
        if (!src_by_position || !bad) {
          const int64_t src = (rowL + (src_by_position ? p : r)) * a.row_vecs;
          x[u] = ld_stream(vec[u] < a.row_vecs ? k_new + src + vec[u] : v_new + src + (vec[u] - a.row_vecs));
        }
        pos[u] = bad ? -1 : p;
      }
#pragma unroll
      for (int u = 0; u < kVec; ++u) {
        // the largest magnitude as bf16 bits (ordered like the values; NaN and infinity on top)
        uint32_t m = __vmaxu2(__vmaxu2(x[u].x & 0x7FFF7FFFu, x[u].y & 0x7FFF7FFFu),
                              __vmaxu2(x[u].z & 0x7FFF7FFFu, x[u].w & 0x7FFF7FFFu));
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
        const int byte = row_exp_byte(max(m & 0xFFFFu, m >> 16));
        if (pos[u] < 0) continue;
        uint2 code;
        if (byte == kExpNaNByte) {
          code = make_uint2(kCodeNaN4, kCodeNaN4);
        } else {
          const float f = quant_factor(byte);
          code = make_uint2(quantise4(x[u].x, x[u].y, f), quantise4(x[u].z, x[u].w, f));
          if (byte == kExpTopByte) code = make_uint2(cap_top_codes(code.x), cap_top_codes(code.y));
        }
        const bool is_k = vec[u] < a.row_vecs;
        const int w = is_k ? vec[u] : vec[u] - a.row_vecs;
        (is_k ? a.k : a.v)[(rowL + pos[u]) * a.row_vecs + w] = code;
        if (w % kLanes == 0)
          (is_k ? a.ke : a.ve)[(static_cast<int64_t>(b) * a.Hkv + w / kLanes) * a.Ls + pos[u]] = static_cast<uint8_t>(byte);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_gather_quant_kernel(const __grid_constant__ QuantArgs a,
                                                                   uint4* __restrict__ k_out,
                                                                   uint4* __restrict__ v_out) {
  constexpr int kLanes = D / 8;
  const int b = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  const int Rb = checked_rows(a, b);
  const int64_t rowL = static_cast<int64_t>(b) * a.L;
  const int per_pos = 2 * a.row_vecs;
  for (int r0 = blockIdx.x * a.rows_per_pass; r0 < Rb; r0 += gridDim.x * a.rows_per_pass) {
    const int n = min(a.rows_per_pass, Rb - r0) * per_pos;
    for (int base = 0; base < n; base += kThreads * kVec) {
      uint2 code[kVec];
      int byte[kVec], vec[kVec];
      int64_t row[kVec];
#pragma unroll
      for (int u = 0; u < kVec; ++u) {
        const int i = base + u * kThreads + static_cast<int>(threadIdx.x);
        row[u] = -1;
        if (i >= n) continue;
        const int rl = i / per_pos;
        vec[u] = i - rl * per_pos;
        const int r = r0 + rl;
        const int p = a.idx != nullptr ? __ldg(a.idx + rowL + r) : r;
        if (p < 0 || p >= a.L) {
          if (vec[u] == 0) report_error(a.dev_err, EC_DEVERR_BAD_IDX);
          continue;
        }
        const bool is_k = vec[u] < a.row_vecs;
        const int w = is_k ? vec[u] : vec[u] - a.row_vecs;
        code[u] = __ldg((is_k ? a.k : a.v) + (rowL + p) * a.row_vecs + w);
        byte[u] = __ldg((is_k ? a.ke : a.ve) + (static_cast<int64_t>(b) * a.Hkv + w / kLanes) * a.Ls + p);
        row[u] = (rowL + r) * a.row_vecs + w;
      }
#pragma unroll
      for (int u = 0; u < kVec; ++u) {
        if (row[u] < 0) continue;
        const DequantScale s = dequant_scale(byte[u]);
        uint4 y;
        dequantise4(code[u].x, s, y.x, y.y);
        dequantise4(code[u].y, s, y.z, y.w);
        (vec[u] < a.row_vecs ? k_out : v_out)[row[u]] = y;
      }
    }
  }
}

QuantArgs make_args(const ec_params& p, const ec_kv& c, const int32_t* idx, const int32_t* R, int32_t* dev_err) {
  QuantArgs a;
  a.L = p.L;
  a.Ls = static_cast<int32_t>(quant_exp_stride(p.L));
  a.Hkv = p.Hkv;
  a.row_vecs = p.Hkv * (p.D / 8);
  a.rows_per_pass = std::max(1, kThreads * kVec / (2 * a.row_vecs));
  a.k = static_cast<uint2*>(c.k);
  a.v = static_cast<uint2*>(c.v);
  a.ke = c.k_exp;
  a.ve = c.v_exp;
  a.idx = idx;
  a.R = R;
  a.dev_err = dev_err;
  return a;
}

// CTAs over positions and sequences: eight per SM at most (R is known on the device only), striding.
cudaError_t quant_grid(const ec_params& p, const QuantArgs& a, dim3* grid) {
  int sms = 0;
  const cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  const int64_t cap = std::max<int64_t>(1, 8 * static_cast<int64_t>(sms) / p.B);
  *grid = dim3(static_cast<unsigned>(std::min<int64_t>((p.L + a.rows_per_pass - 1) / a.rows_per_pass, cap)), p.B);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv_scatter_quant(const ec_params& p, const ec_kv& c, const void* k_new, const void* v_new,
                                    int32_t src_by_position, const int32_t* idx, const int32_t* R, int32_t* dev_err,
                                    cudaStream_t s) {
  const QuantArgs a = make_args(p, c, idx, R, dev_err);
  dim3 grid;
  const cudaError_t e = quant_grid(p, a, &grid);
  if (e != cudaSuccess) return e;
  return launch_pdl(p.D == 128 ? kv_scatter_quant_kernel<128> : kv_scatter_quant_kernel<64>, grid, dim3(kThreads), 0, s,
                    a, static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), src_by_position);
}

cudaError_t launch_kv_gather_quant(const ec_params& p, const ec_kv& c, const int32_t* idx, const int32_t* R,
                                   void* k_out, void* v_out, int32_t* dev_err, cudaStream_t s) {
  const QuantArgs a = make_args(p, c, idx, R, dev_err);
  dim3 grid;
  const cudaError_t e = quant_grid(p, a, &grid);
  if (e != cudaSuccess) return e;
  return launch_pdl(p.D == 128 ? kv_gather_quant_kernel<128> : kv_gather_quant_kernel<64>, grid, dim3(kThreads), 0, s,
                    a, static_cast<uint4*>(k_out), static_cast<uint4*>(v_out));
}

}  // namespace ec
