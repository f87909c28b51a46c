// 4-bit floating point with block scales (e2m1 elements; a power-of-two byte
// per 32 or an e4m3 byte per 16): conversions and the scale array's layout,
// shared by the quantiser and the product.
#pragma once
#include <cstdint>

namespace cbmoe {

constexpr int kFp4Mx = 0;
constexpr int kFp4Nv = 1;
constexpr int kScaleTileRows = 128;
constexpr int kScaleTileBytes = 512;  // 128 rows x 4 blocks

template <int FMT>
constexpr int kFp4Block = FMT == kFp4Mx ? 32 : 16;

// Byte of (row r of the tile, block j of its 4) within a 512-byte scale tile.
__host__ __device__ constexpr int scale_tile_byte(int r, int j) { return (r % 32) * 16 + (r / 32) * 4 + j; }

// Two floats -> two e2m1 codes (nearest, ties to the even code, saturating),
// lo in the low nibble; eight of them packed in order into a word.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The float that is v(c) for the 4-bit code c: e2m1's exponent and mantissa
// bits under fp32's, times 2^126 to move the bias from 1 to 127.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const float m = __uint_as_float((c & 7u) << 22) * __uint_as_float(253u << 23);
  return __uint_as_float(__float_as_uint(m) | ((c & 8u) << 28));
}

// The value of an e4m3 byte with sign 0 (0x7F: NaN), from its bits: as above,
// with 2^120 between the biases 7 and 127.
__device__ __forceinline__ float e4m3_value(uint32_t s) {
  return s == 0x7Fu ? __uint_as_float(0x7FC00000u)
                    : __uint_as_float(s << 20) * __uint_as_float((120u + 127u) << 23);
}

// 2^(b - 127), a subnormal for b = 0; NaN for b = 255.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7FC00000u : b == 0u ? 0x00400000u : b << 23);
}

template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t b) {
  return FMT == kFp4Mx ? e8m0_value(b) : e4m3_value(b);
}

}  // namespace cbmoe
