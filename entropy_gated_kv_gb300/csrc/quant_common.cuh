// quant_common.cuh — the 8-bit row format of the K/V cache, shared by the kernels that write and
// read it.
//
// A row is the D values of one (position, KV head) of K or of V. It is held as D e4m3 codes and one
// exponent byte: value = code * 2^(byte - 127). The exponent is the smallest integer e >= -110
// with max|x| <= 448 * 2^e, so the row's largest code lies in (224, 448] and nothing saturates.
// A power of two costs e4m3 no precision (its relative step does not depend on the exponent), makes
// the scaling exact, so a value is rounded once, and lets the integer fields of the bf16 maximum
// give the exponent: no logarithm, no division, one answer on every device. The floor of -110
// keeps the smallest step (2^-9 * 2^-110) a normal bf16; at the top, exponent 120, codes stop at 240,
// since 256 * 2^120 is no bf16 number. So every stored value is one. A row that holds an infinity or a NaN
// has no such exponent: it is stored as byte 255 with NaN codes and reads back as NaN. A NaN code in a row of
// another exponent is not written here, but a cache may come from elsewhere: it reads as NaN too.
#pragma once

#include <cstdint>

#include "ec_common.cuh"

namespace ec {

constexpr int kExpZeroByte = 17;   // exponent -110, the smallest one
constexpr int kExpTopByte = 247;   // exponent 120, that of the largest bf16 values
constexpr int kExpNaNByte = 255;
constexpr uint32_t kCodeNaN4 = 0x7F7F7F7Fu;

// The exponent byte of a row whose largest magnitude has the bf16 bits a (sign cleared).
EC_DEV int row_exp_byte(uint32_t a) {
  if (a >= 0x7F80u) return kExpNaNByte;
  // a = (1 + m/128) 2^(E - 127): 1.75 = 448 / 256 is m = 0x60, so the exponent is E - 127 - 8, one
  // more above it (for subnormal a, E = 0, the floor decides)
  return max(kExpZeroByte, static_cast<int>(a >> 7) - 8 + ((a & 0x7Fu) > 0x60u ? 1 : 0));
}

// 2^(127 - byte) as fp32: the exact factor that brings a row into code range (byte 17 .. 247).
EC_DEV float quant_factor(int byte) { return __uint_as_float(static_cast<uint32_t>(254 - byte) << 23); }

// Four codes of lo.x, lo.y, hi.x, hi.y (each the two bf16 of a word) times `f`; nearest even.
EC_DEV uint32_t quantise4(uint32_t lo, uint32_t hi, float f) {
  uint16_t a, b;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(bf16hi_to_f32(lo) * f), "f"(bf16lo_to_f32(lo) * f));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(bf16hi_to_f32(hi) * f), "f"(bf16lo_to_f32(hi) * f));
  return static_cast<uint32_t>(a) | (static_cast<uint32_t>(b) << 16);
}

// Codes of a row of exponent 120: magnitudes above 240 (0x77) become 240.
EC_DEV uint32_t cap_top_codes(uint32_t w) { return __vminu4(w & 0x7F7F7F7Fu, 0x77777777u) | (w & 0x80808080u); }

// The rows [0, n) of a sequence's line in pieces of `piece`, dealt to the CTAs in turn. Counted without
// a sign: n is below 2^31 and a step (piece times CTAs) below 2^22, so the sum that ends the loop, and
// a row of the last piece past n, stay below 2^32. (With a sign the last step of a line close to 2^31
// rows wraps, and the loop goes on at negative rows.)
struct Pieces {
  uint32_t at, n, step;
  EC_DEV Pieces(int32_t rows, uint32_t piece, uint32_t cta, uint32_t ctas)
      : at(cta * piece), n(static_cast<uint32_t>(rows)), step(ctas * piece) {}
  EC_DEV bool more() const { return at < n; }
  EC_DEV void next() { at += step; }
};

EC_DEV uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Dequantisation to bf16 without a conversion instruction: an e4m3 code (s eeee mmm) put at bits
// 15, 10..7 and 6..4 of a bf16 is the code's value times 2^(7 - 127), subnormals included, so one
// exact product with 2^(120 + e) gives code * 2^e. Above e = 7 that factor leaves bf16's range and
// a second one follows (byte > 134: rows with a magnitude above 57344).
struct DequantScale {
  uint32_t f1, f2;  // bf16x2 factors; f2 is used when two
  bool two;
};

EC_DEV DequantScale dequant_scale(int byte) {
  DequantScale s;
  const int e1 = min(byte + 120, 254);
  const int e2 = 127 + byte + 120 - e1;
  s.f1 = byte == kExpNaNByte ? 0x7FC07FC0u : static_cast<uint32_t>(e1) * 0x00800080u;
  s.f2 = static_cast<uint32_t>(e2) * 0x00800080u;
  s.two = byte > 134 && byte != kExpNaNByte;
  return s;
}

// The one factor of bytes up to kExpOneFactor.
constexpr int kExpOneFactor = 134;
EC_DEV uint32_t dequant_factor(int byte) { return static_cast<uint32_t>(byte + 120) * 0x00800080u; }

// Four codes, none of them NaN -> two words of two bf16.
EC_DEV void dequantise4(uint32_t w, uint32_t f, uint32_t& lo, uint32_t& hi) {
  // each byte sign-extended to 16 bits, shifted left by 4, then the copies of the sign over the
  // exponent's upper bits cleared
  uint32_t a, b;
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(a) : "r"(w));
  asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(b) : "r"(w));
  lo = mul_bf16x2((a << 4) & 0x87F087F0u, f);
  hi = mul_bf16x2((b << 4) & 0x87F087F0u, f);
}

// e4m3 has two codes without a value, 0x7F and 0xFF. By its bits alone such a code would read as 480, so
// the dequantisation above is for words without one. Adding 1 to every byte carries into bit 7 from a
// NaN only; a carry out of a byte 0xFF may mark its neighbour too, but then there is a NaN. The marks of
// several words may be joined with "or". (Two instructions a word: 191 -> 196 us on the long shared prefix, 79.8 ->
// 81.7 on the long 8-bit case. Masking the signs off first: 202 and 83.9. A comparison that puts the NaN
// into the product by an fma: 211 and 84.9.)
constexpr uint32_t kNaNMarks = 0x80808080u;
EC_DEV uint32_t nan_marks(uint32_t w) { return (w + 0x01010101u) ^ w; }

// NaN in lo and hi where a code of w is one (and only there).
EC_DEV void keep_nan(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t m = (w & 0x7F7F7F7Fu) + 0x01010101u;
  uint32_t a, b;
  asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(a) : "r"(m));  // bit 7 of bytes 0 and 1, over their halves
  asm("prmt.b32 %0, %1, 0, 0xBBAA;" : "=r"(b) : "r"(m));
  lo |= a;
  hi |= b;
}

// Any row, any code.
EC_DEV void dequantise4(uint32_t w, const DequantScale& s, uint32_t& lo, uint32_t& hi) {
  dequantise4(w, s.f1, lo, hi);
  if (s.two) {
    lo = mul_bf16x2(lo, s.f2);
    hi = mul_bf16x2(hi, s.f2);
  }
  keep_nan(w, lo, hi);
}

}  // namespace ec
