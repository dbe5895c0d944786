// The 4-bit cache page: encoding and expansion shared by the prologue, the
// page operators and the FP4 decode.
//
// A page of 32 rows is 10,752 bytes in three planes, so that each plane of a
// row is contiguous and 16-byte aligned:
//   [0, 8192)      latent codes: 32 rows x 256 bytes, two E2M1 values a byte
//   [8192, 8704)   scale codes: 16 blocks x 32 rows, one byte each
//   [8704, 10752)  rope part: 32 rows x 64 E4M3 codes
// A block is 32 consecutive latent values of a row.  With scale code e in
// 0..14 its values are kv_scale * 2^(e - 8) * v, v one of +-{0, .5, 1, 1.5, 2,
// 3, 4, 6}.  Scale code 15 (and no other) marks a block with a NaN: every
// value of it reads as NaN.  Only the low 4 bits of a scale byte count.
//
// 2^(e - 8) * v is an E4M3 number for every e in 0..14 (the smallest step,
// 2^-9, is E4M3's, and 6 * 2^6 = 384 <= 448), so a block expands to E4M3 codes
// without any rounding: the decode's operands, scores and weights over an FP4
// cache are those over the E4M3 cache that it expands to (up to 16 rows the
// row sums are added in another order, and differ by rounding).
//
// Bit layout of a 32-bit word (8 consecutive values, little endian): the low
// three bits of nibble j are value j's magnitude code; the top bits of nibbles
// 1, 3, 5, 7 are the signs of values 0 to 3 and those of nibbles 0, 2, 4, 6
// the signs of values 4 to 7.  The magnitudes are then byte-permute selectors
// into the scale's eight E4M3 codes, and the signs of values 0-3 already sit
// at the four bytes' sign bits: 7 instructions expand 8 values, where signs
// kept in their own nibbles need 9.
#pragma once
#include <cstdint>

#include "mla_internal.h"

namespace mla {

constexpr int kFp4RowCodes = MLA_LATENT_DIM / 2;                                // 256 bytes
constexpr int kFp4Blocks = MLA_LATENT_DIM / MLA_FP4_BLOCK;                      // 16
constexpr int kFp4ScaleOffset = MLA_PAGE_SIZE * kFp4RowCodes;                   // 8192
constexpr int kFp4RopeOffset = kFp4ScaleOffset + kFp4Blocks * MLA_PAGE_SIZE;    // 8704
static_assert(kFp4RopeOffset + MLA_PAGE_SIZE * MLA_ROPE_DIM == MLA_FP4_PAGE_BYTES, "FP4 page");
constexpr int kFp4NanScale = 15;

#ifdef __CUDACC__
// Scale code of a block from its largest magnitude (as float bits without the
// sign; a NaN's bits are above infinity's): the smallest e in 0..14 with
// amax <= 7 * 2^(e - 8), 14 where none is.  7 is half a step above the largest
// code, 6, so under that scale no value is more than half a step from its code;
// larger values saturate at 384.  7 * 2^(k - 8) has the bits ((121 + k) << 23)
// + 0x600000, and positive floats order like their bits.
__device__ __forceinline__ int fp4_scale_code(uint32_t amax_bits) {
  if (amax_bits > 0x7F800000u) return kFp4NanScale;
  const int k = ((static_cast<int>(amax_bits) - 0x600001) >> 23) - 120;
  return min(max(k, 0), 14);
}

// 2^(8 - e), exactly.
__device__ __forceinline__ float fp4_inv_scale(int e) { return __int_as_float((135 - e) << 23); }

// Signs of a word of plain E2M1 nibbles (bits 4j + 3) to the format's places.
__device__ __forceinline__ uint32_t fp4_place_signs(uint32_t w) {
  const uint32_t up = w << 4;  // even nibbles' signs at their bytes' top bits
  const uint32_t lo = __byte_perm(up, w, 0x5140) & 0x80808080u;         // values 0-3
  const uint32_t hi = (__byte_perm(up, w, 0x7362) & 0x80808080u) >> 4;  // values 4-7
  return (w & 0x77777777u) | lo | hi;
}

// Eight values times 2^(8 - e) as one word of the format: nearest E2M1, ties
// to even, saturating at 6.
__device__ __forceinline__ uint32_t fp4_encode8(const float (&x)[8], float inv) {
  uint32_t w;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(w)
      : "f"(x[0] * inv), "f"(x[1] * inv), "f"(x[2] * inv), "f"(x[3] * inv), "f"(x[4] * inv),
        "f"(x[5] * inv), "f"(x[6] * inv), "f"(x[7] * inv));
  return fp4_place_signs(w);
}

// The same from four pairs of halves already multiplied by 2^(8 - e) (low half:
// the earlier value).
__device__ __forceinline__ uint32_t fp4_encode8_halves(uint32_t x01, uint32_t x23, uint32_t x45,
                                                       uint32_t x67) {
  uint32_t w;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f16x2 b0, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f16x2 b1, %2;\n"
      " cvt.rn.satfinite.e2m1x2.f16x2 b2, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f16x2 b3, %4;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(w)
      : "r"(x01), "r"(x23), "r"(x45), "r"(x67));
  return fp4_place_signs(w);
}

// The E4M3 codes of scale code e's eight magnitudes, as two words: from e = 3 to
// 14 all are normal numbers, e - 2 exponents above e = 2's pattern, so each word
// is one multiply-add.
__device__ __forceinline__ uint2 fp4_scale_table_normal(uint32_t e) {
  return make_uint2(0x0C080000u - 2u * 0x08080800u + e * 0x08080800u,
                    0x1C181410u - 2u * 0x08080808u + e * 0x08080808u);
}

// For every e: the smaller scales and NaN blocks take their constants.
__device__ __forceinline__ uint2 fp4_scale_table(uint32_t e) {
  uint2 t = fp4_scale_table_normal(e);
  if (e - 3u >= 12u) {
    t = e == 0 ? make_uint2(0x03020100u, 0x0C080604u)
        : e == 1 ? make_uint2(0x06040200u, 0x14100C08u)
        : e == 2 ? make_uint2(0x0C080400u, 0x1C181410u)
                 : make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  }
  return t;
}

// Expands a word of the format to the E4M3 codes of its eight values.
__device__ __forceinline__ uint2 fp4_expand8(uint32_t w, uint2 table) {
  const uint32_t sel = w & 0x77777777u;
  const uint32_t lo = __byte_perm(table.x, table.y, sel);
  const uint32_t hi = __byte_perm(table.x, table.y, sel >> 16);
  return make_uint2(lo | (w & 0x80808080u), hi | ((w << 4) & 0x80808080u));
}
#endif

}  // namespace mla
