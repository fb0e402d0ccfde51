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

// 2^(s - 127) as bf16 bits for any scale byte (0 is a subnormal, 255 is NaN).
__device__ __forceinline__ uint32_t scale_bf16(uint32_t s) {
  return s == 0u ? 0x0040u : s == kScaleNan ? 0x7FC0u : s << 7;
}

// Both halves times m (bf16x2; powers of two here, so exact; subnormals are
// kept).
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t m) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(m));
  return r;
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

// The eight bf16 in v to e2m1 codes under scale byte s (codes 0 under a NaN
// scale).
__device__ __forceinline__ uint32_t quantize_bf16x8(const uint4& v, uint32_t s) {
  if (s == kScaleNan) return 0u;
  const uint32_t inv = ((254u - s) << 7) * 0x10001u;  // 2^(127 - s) in both halves
  const uint32_t w[4] = {mul_bf16x2(v.x, inv), mul_bf16x2(v.y, inv), mul_bf16x2(v.z, inv), mul_bf16x2(v.w, inv)};
  const float f[8] = {bf16lo_to_f32(w[0]), bf16hi_to_f32(w[0]), bf16lo_to_f32(w[1]), bf16hi_to_f32(w[1]),
                      bf16lo_to_f32(w[2]), bf16hi_to_f32(w[2]), bf16lo_to_f32(w[3]), bf16hi_to_f32(w[3])};
  return pack_e2m1x8(f);
}

// Byte i of the result is the byte of (b:a) that nibble i of `sel` names; a
// nibble with its top bit set gives that byte's sign bit eight times.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Four codes (the low 16 bits of q) to four bf16 times the scale (bf16x2 sc):
// the e2m1 magnitudes are bf16 whose two bytes come from eight-entry tables.
__device__ __forceinline__ void dequantize_bf16x4(uint32_t q, uint32_t sc, uint32_t& w0, uint32_t& w1) {
  const uint32_t sel = q & 0x7777u;
  // the sign bit of a code is its selector's top bit: 0xFF below zero, else 0x80
  const uint32_t neg = (prmt(0x80808080u, 0x80808080u, q) & 0x01010101u) << 7;
  const uint32_t hi = prmt(0x3F3F3F00u, 0x40404040u, sel) | neg;
  const uint32_t lo = prmt(0xC0800000u, 0xC0804000u, sel);
  w0 = mul_bf16x2(prmt(lo, hi, 0x5140u), sc);
  w1 = mul_bf16x2(prmt(lo, hi, 0x7362u), sc);
}

// Eight consecutive bf16 per lane, four lanes per block: the block's scale
// byte, known to its four lanes.  All 32 lanes call it.  The maxima are of the
// magnitudes' bits, two bf16 at a time.
__device__ __forceinline__ uint32_t block_scale_of_quad(const uint4& v) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  uint32_t m = __vimax3_u16x2(v.x & kAbs, v.y & kAbs, v.z & kAbs);
  m = __vmaxu2(m, v.w & kAbs);
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return scale_byte(max(m & 0xFFFFu, m >> 16));
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
