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
// line. A row's D values lie in D / 16 neighbouring lanes, 32 bytes of bf16 (one 256-bit access where
// the buffers are aligned to it) and 16 of codes each; a thread loads its part of kRows rows before
// it works on any. The maxima of two rows share a register's halves, so a reduction step is one
// shuffle for both. (With 16 bytes a lane the write was bound by its instructions, most of them
// addresses: 190 us for 807 MB; with 32, 133 us, 6.1 TB/s. The read of 332 MB takes 59 us, 5.6 TB/s; a call
// of a few hundred rows 3.7 us.)
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
  int32_t wide;         // the bf16 buffers are 32-byte aligned
  uint4 *k, *v;
  uint8_t *ke, *ve;
  const int32_t *idx, *R;
  int32_t* dev_err;
};

// 32 bytes of a row; `wide`: the address is a multiple of 32.
struct Oct {
  uint32_t w[8];
};

EC_DEV Oct ld_oct(const uint4* p, bool wide) {
  Oct v;
  if (wide)
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                   "=r"(v.w[7])
                 : "l"(p));
  else
    asm volatile(
        "ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%8];\n\tld.global.nc.v4.b32 {%4,%5,%6,%7}, [%8+16];"
        : "=&r"(v.w[0]), "=&r"(v.w[1]), "=&r"(v.w[2]), "=&r"(v.w[3]), "=&r"(v.w[4]), "=&r"(v.w[5]), "=&r"(v.w[6]),
          "=&r"(v.w[7])
        : "l"(p));
  return v;
}

EC_DEV void st_oct(uint4* p, const Oct& v, bool wide) {
  if (wide)
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]), "r"(v.w[2]),
                 "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7])
                 : "memory");
  else {
    p[0] = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    p[1] = make_uint4(v.w[4], v.w[5], v.w[6], v.w[7]);
  }
}

EC_DEV uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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
  constexpr int kLanes = D / 16, kStep = kThreads / kLanes;  // lanes of a row; rows of a CTA per step
  const int b = blockIdx.y, lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  pdl_wait();
  pdl_launch_dependents();
  const int Rb = checked_rows(a, b);
  const int64_t rowL = static_cast<int64_t>(b) * a.L;
  const int n = Rb * 2 * a.Hkv;  // below 2^31
  for (Pieces line(n, kStep * kRows, blockIdx.x, gridDim.x); line.more(); line.next()) {
    Oct x[kRows];
    int pos[kRows], head[kRows];  // head: of 2 Hkv, the K heads first
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const uint32_t i = line.at + u * kStep + sub;
      pos[u] = -1;
      head[u] = 0;
      if (i >= line.n) continue;
      const int r = a.div_2h(static_cast<int>(i));
      head[u] = static_cast<int>(i) - r * 2 * a.Hkv;
      const int p = __ldg(a.idx + rowL + r);
      // rows in recompute order ascend: a position that is not below its successor is a bad
      // (possibly repeated) one, whose codes and exponent two rows could write at once
      const bool bad = p < 0 || p >= a.L || (!src_by_position && r + 1 < Rb && p >= __ldg(a.idx + rowL + r + 1));
      if (bad && head[u] == 0) report_error(a.dev_err, EC_DEVERR_BAD_IDX);
      if (!src_by_position || !bad) {
        const int h = head[u] < a.Hkv ? head[u] : head[u] - a.Hkv;
        x[u] = ld_oct((head[u] < a.Hkv ? k_new : v_new) +
                          (((rowL + (src_by_position ? p : r)) * a.Hkv + h) * kLanes + lane) * 2, a.wide);
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
      for (int e = 0; e < 2; ++e) {
        m[e] = 0;
        if (pos[u + e] >= 0)
#pragma unroll
          for (int q = 0; q < 8; ++q) m[e] = max_u16x2(m[e], x[u + e].w[q] & 0x7FFF7FFFu);
      }
      top[u / 2] = max_u16x2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
    }
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1)
#pragma unroll
      for (int u = 0; u < kRows / 2; ++u) top[u] = max_u16x2(top[u], __shfl_xor_sync(0xffffffffu, top[u], off));
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (pos[u] < 0) continue;
      const int byte = row_exp_byte(u & 1 ? top[u / 2] >> 16 : top[u / 2] & 0xFFFFu);
      uint32_t code[4];
      if (byte != kExpNaNByte) {
        const float f = quant_factor(byte);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          code[q] = quantise4(x[u].w[2 * q], x[u].w[2 * q + 1], f);
          if (byte == kExpTopByte) code[q] = cap_top_codes(code[q]);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) code[q] = kCodeNaN4;
      }
      const bool is_k = head[u] < a.Hkv;
      const int h = is_k ? head[u] : head[u] - a.Hkv;
      (is_k ? a.k : a.v)[((rowL + pos[u]) * a.Hkv + h) * kLanes + lane] = make_uint4(code[0], code[1], code[2], code[3]);
      if (lane == 0) (is_k ? a.ke : a.ve)[(static_cast<int64_t>(b) * a.Hkv + h) * a.Ls + pos[u]] = static_cast<uint8_t>(byte);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_gather_quant_kernel(const __grid_constant__ QuantArgs a,
                                                                   uint4* __restrict__ k_out,
                                                                   uint4* __restrict__ v_out) {
  constexpr int kLanes = D / 16, kStep = kThreads / kLanes;
  const int b = blockIdx.y, lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  pdl_wait();
  pdl_launch_dependents();
  const int Rb = checked_rows(a, b);
  const int64_t rowL = static_cast<int64_t>(b) * a.L;
  const int n = Rb * 2 * a.Hkv;
  for (Pieces line(n, kStep * kRows, blockIdx.x, gridDim.x); line.more(); line.next()) {
    uint4 code[kRows];
    int byte[kRows];
    int64_t to[kRows];  // the output row, complemented for V; kNone: none
    constexpr int64_t kNone = INT64_MIN;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const uint32_t i = line.at + u * kStep + sub;
      to[u] = kNone;
      if (i >= line.n) continue;
      const int r = a.div_2h(static_cast<int>(i)), head = static_cast<int>(i) - r * 2 * a.Hkv;
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
      const uint32_t c[4] = {code[u].x, code[u].y, code[u].z, code[u].w};
      Oct y;
      if (byte[u] <= kExpOneFactor) {
        const uint32_t f = dequant_factor(byte[u]);
#pragma unroll
        for (int q = 0; q < 4; ++q) dequantise4(c[q], f, y.w[2 * q], y.w[2 * q + 1]);
        if ((nan_marks(c[0]) | nan_marks(c[1]) | nan_marks(c[2]) | nan_marks(c[3])) & kNaNMarks)
#pragma unroll
          for (int q = 0; q < 4; ++q) keep_nan(c[q], y.w[2 * q], y.w[2 * q + 1]);
      } else {
        const DequantScale s = dequant_scale(byte[u]);
#pragma unroll
        for (int q = 0; q < 4; ++q) dequantise4(c[q], s, y.w[2 * q], y.w[2 * q + 1]);
      }
      st_oct(to[u] >= 0 ? k_out + (to[u] * kLanes + lane) * 2 : v_out + (~to[u] * kLanes + lane) * 2, y, a.wide);
    }
  }
}

QuantArgs make_args(const ec_params& p, const ec_kv& c, const void* k, const void* v, const int32_t* idx,
                    const int32_t* R, int32_t* dev_err) {
  QuantArgs a;
  a.L = p.L;
  a.Ls = static_cast<int32_t>(quant_exp_stride(p.L));
  a.Hkv = p.Hkv;
  a.div_2h.set(2 * p.Hkv);
  a.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0;
  a.k = static_cast<uint4*>(c.k);
  a.v = static_cast<uint4*>(c.v);
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
  const int64_t rows = static_cast<int64_t>(p.L) * 2 * p.Hkv, step = kThreads / (p.D / 16) * kRows;
  *grid = dim3(static_cast<unsigned>(std::min<int64_t>((rows + step - 1) / step, cap)), p.B);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_kv_scatter_quant(const ec_params& p, const ec_kv& c, const void* k_new, const void* v_new,
                                    int32_t src_by_position, const int32_t* idx, const int32_t* R, int32_t* dev_err,
                                    cudaStream_t s) {
  const QuantArgs a = make_args(p, c, k_new, v_new, idx, R, dev_err);
  dim3 grid;
  const cudaError_t e = quant_grid(p, &grid);
  if (e != cudaSuccess) return e;
  return launch_pdl(p.D == 128 ? kv_scatter_quant_kernel<128> : kv_scatter_quant_kernel<64>, grid, dim3(kThreads), 0, s,
                    a, static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), src_by_position);
}

cudaError_t launch_kv_gather_quant(const ec_params& p, const ec_kv& c, const int32_t* idx, const int32_t* R,
                                   void* k_out, void* v_out, int32_t* dev_err, cudaStream_t s) {
  const QuantArgs a = make_args(p, c, k_out, v_out, idx, R, dev_err);
  dim3 grid;
  const cudaError_t e = quant_grid(p, &grid);
  if (e != cudaSuccess) return e;
  return launch_pdl(p.D == 128 ? kv_gather_quant_kernel<128> : kv_gather_quant_kernel<64>, grid, dim3(kThreads), 0, s,
                    a, static_cast<uint4*>(k_out), static_cast<uint4*>(v_out));
}

}  // namespace ec
