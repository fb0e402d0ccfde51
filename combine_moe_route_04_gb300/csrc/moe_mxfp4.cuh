// moe_mxfp4.cuh -- device helpers of the MXFP4 format (blocks of 32 along a
// row, elements e2m1, one e8m0 scale byte s per block standing for 2^(s-127)).
#pragma once

#include <cstdint>

#include "moe_device.cuh"

namespace moe {

constexpr uint32_t kScaleNan = 255u;  // e8m0's only NaN

// Offset of the scale bytes of row r, columns [128 c, 128 c + 128) (four
// blocks, one 32-bit word): 512-byte tiles of 128 rows x 4 blocks, tiles of a
// row block in column order, rows r, r + 32, r + 64, r + 96 of a tile adjacent.
// kb128 = columns / 128.
__host__ __device__ __forceinline__ int64_t scale_word_offset(int64_t r, int64_t c, int64_t kb128) {
  return ((r >> 7) * kb128 + c) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// The scale byte of a block whose largest magnitude has the bf16 bits `amax`
// (sign clear): floor(log2(amax)) - 2 as a biased exponent, so that the
// block's largest element lands in [4, 8) and saturates at 6 when above it.
// bf16's exponent field is floor(log2) + 127 for normal numbers; below them
// (and for 0) the scale is clamped to the smallest, 2^-127.  A block with a
// NaN or an infinity has no scale: its byte is NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax >= 0x7F80u) return kScaleNan;
  const uint32_t e = amax >> 7;
  return e > 2u ? e - 2u : 0u;
}

// 2^(127 - s): elements are divided by their scale exactly (s <= 252 here).
__device__ __forceinline__ float scale_inverse(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// 2^(s - 127) for any scale byte (s = 0 is a subnormal float, 255 is NaN).
__device__ __forceinline__ float scale_value(uint32_t s) {
  if (s == kScaleNan) return __uint_as_float(0x7FC00000u);
  return s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23);
}

// Eight floats to eight e2m1 codes (v[0] in the low nibble), round to nearest
// even, saturating at +-6.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&v)[8]) {
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

// Largest magnitude (bf16 bits, sign clear) of the two bf16 in w and m.
__device__ __forceinline__ uint32_t amax_bf16x2(uint32_t m, uint32_t w) {
  return max(m, max(w & 0x7FFFu, (w >> 16) & 0x7FFFu));
}

// The eight bf16 in v to e2m1 codes under scale byte s (codes 0 under a NaN
// scale).
__device__ __forceinline__ uint32_t quantize_bf16x8(const uint4& v, uint32_t s) {
  if (s == kScaleNan) return 0u;
  const float inv = scale_inverse(s);
  const float f[8] = {bf16lo_to_f32(v.x) * inv, bf16hi_to_f32(v.x) * inv, bf16lo_to_f32(v.y) * inv,
                      bf16hi_to_f32(v.y) * inv, bf16lo_to_f32(v.z) * inv, bf16hi_to_f32(v.z) * inv,
                      bf16lo_to_f32(v.w) * inv, bf16hi_to_f32(v.w) * inv};
  return pack_e2m1x8(f);
}

// Eight consecutive bf16 per lane, four lanes per block: the block's scale
// byte, known to its four lanes.  All 32 lanes call it.
__device__ __forceinline__ uint32_t block_scale_of_quad(const uint4& v) {
  uint32_t m = amax_bf16x2(0u, v.x);
  m = amax_bf16x2(m, v.y);
  m = amax_bf16x2(m, v.z);
  m = amax_bf16x2(m, v.w);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return scale_byte(m);
}

// The scale word of the 16 lanes' four blocks (block 0 in the low byte), known
// to all 16.  All 32 lanes call it.
__device__ __forceinline__ uint32_t scale_word_of_half(uint32_t s, int lane) {
  uint32_t w = s << (8 * ((lane >> 2) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, 4);
  w |= __shfl_xor_sync(0xffffffffu, w, 8);
  return w;
}

}  // namespace moe
