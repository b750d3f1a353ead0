// Number formats of a key/value cache row: bf16, or 8-bit numbers (e4m3 or
// int8) with one power-of-two scale per row.
//
// A row x of d bf16 numbers is stored as rne(x 2^-e) with the smallest e
// that keeps max|x| 2^-e within the type's largest number (448 or 127), at
// least -100, and at most 119 (e4m3) or 121 (int8), where the largest number
// is still finite in bf16: beyond (|x| > 2.97e38) it saturates.  The scale
// byte is e + 127.  A power of two scales
// without rounding, so there is one rounding per element, the same in any
// precision, and what reads back is exact in bf16 (e4m3 has 4 significant
// bits, int8 at most 7).  e >= -100 keeps numbers, scales and the products
// of a score's factors far from the ends of fp32's range; it costs rows whose
// largest number is below 2^-91 (e4m3) or 2^-93 (int8) bits, and all of them
// from 2^-110 (2^-101) on.  Storing what was read back gives the same numbers
// again.  A row with a NaN or an infinity gets the scale byte 255 and reads
// back as NaN whole.
#pragma once

#include <stdint.h>

#include "fa_ptx.cuh"

namespace fa {

enum CacheFormat : int { kCacheBf16 = 0, kCacheE4m3 = 1, kCacheInt8 = 2 };

constexpr uint32_t kScaleNan = 255;

// Scale byte of a row whose largest |x| has the bf16 bits `amax`.  448 is
// 1.75 x 2^8 and 127 is 1.984375 x 2^6: the exponent of amax decides, and
// its fraction (7 bits) whether one more is needed.
template <int FMT>
FA_DEV uint32_t row_scale(uint32_t amax) {
  if (amax >= 0x7F80u) return kScaleNan;
  const int ex = static_cast<int>(amax >> 7) - 127, frac = static_cast<int>(amax & 0x7Fu);
  const int e = FMT == kCacheE4m3 ? ex - 8 + (frac > 0x60) : ex - 6 + (frac > 0x7E);
  return static_cast<uint32_t>(min(max(e, -100), FMT == kCacheE4m3 ? 119 : 121) + 127);
}

// 2^-e for the scale byte e + 127 of row_scale (27 .. 248)
FA_DEV float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// four numbers times f = 2^-e (exact), as four stored bytes (x0 lowest);
// int8: at most 127 then
template <int FMT>
FA_DEV uint32_t quantise4(float x0, float x1, float x2, float x3, float f) {
  if (FMT == kCacheE4m3) {
    uint32_t w;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(w)
        : "f"(x0 * f), "f"(x1 * f), "f"(x2 * f), "f"(x3 * f));
    return w;
  }
  // Added to 1.5 x 2^23, whose last place is 1, a number is rounded to an
  // integer (ties to even) whose two's complement is the sum's low byte.
  const auto q = [f](float x) { return __float_as_uint(fmaf(x, f, 12582912.f)); };
  return __byte_perm(__byte_perm(q(x0), q(x1), 0x0040), __byte_perm(q(x2), q(x3), 0x0040), 0x5410);
}

// The scale of a row, prepared for widening its numbers.
// e4m3: a number's exponent and fraction moved to their bf16 places read as
// value x 2^-120, so the factor is 2^(e + 120), in two steps where that
// passes bf16's range (e > 7).
struct RowScale {
  uint32_t f1, f2;  // bf16 pairs
  bool two;
};
template <int FMT>
FA_DEV RowScale widen_scale(uint32_t byte) {
  RowScale s;
  if (FMT == kCacheE4m3) {
    const uint32_t lo = min(byte, 134u);  // 2^(byte - 127), at most 2^7
    s.f1 = ((lo + 120u) << 7) * 0x00010001u;
    s.f2 = ((byte - lo + 127u) << 7) * 0x00010001u;
    s.two = byte > 134u;
  } else {
    s.f1 = (byte << 7) * 0x00010001u;
    s.f2 = 0;
    s.two = false;
  }
  if (byte == kScaleNan) s.f1 = 0x7FFF7FFFu;
  return s;
}

// four stored bytes -> four bf16 values (two words)
template <int FMT>
FA_DEV void widen4(uint32_t w, const RowScale& s, uint32_t& lo, uint32_t& hi) {
  if (FMT == kCacheE4m3) {
    const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);  // b0, b1 | b2, b3
    lo = mul_bf16x2((a & 0x80008000u) | ((a >> 4) & 0x07F007F0u), s.f1);
    hi = mul_bf16x2((b & 0x80008000u) | ((b >> 4) & 0x07F007F0u), s.f1);
    if (s.two) {
      lo = mul_bf16x2(lo, s.f2);
      hi = mul_bf16x2(hi, s.f2);
    }
  } else {
    // a byte x = low7 - 128 [sign]: 0x4300 | low7 is 128 + low7 and
    // 0x4300 | sign bit is 128 or 256 in bf16; their difference is exact
    const uint32_t a = __byte_perm(w, 0, 0x4140), b = __byte_perm(w, 0, 0x4342);
    lo = mul_bf16x2(sub_bf16x2((a & 0x007F007Fu) | 0x43004300u, (a & 0x00800080u) | 0x43004300u),
                    s.f1);
    hi = mul_bf16x2(sub_bf16x2((b & 0x007F007Fu) | 0x43004300u, (b & 0x00800080u) | 0x43004300u),
                    s.f1);
  }
}

// four stored bytes as f16 pairs (bytes 0, 1) and (2, 3), exact
template <int FMT>
FA_DEV void stored_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == kCacheE4m3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    // x + 128 under the exponent of 1024, less 1152
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
  }
}

// 2^(byte - 127); NaN for the scale of a bad row
FA_DEV float scale_value(uint32_t byte) {
  return byte == kScaleNan ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(byte << 23);
}
// byte - 127: the byte as the last bits of 2^23, less 2^23 + 127
FA_DEV float scale_exponent(uint32_t byte) {
  return byte == kScaleNan ? __uint_as_float(0x7FFFFFFFu)
                           : __uint_as_float(0x4B000000u | byte) - 8388735.f;
}

}  // namespace fa
