// moe_epilogue.cuh -- what the products' epilogues share: pieces of 32 rows x 128
// columns between TMEM, registers and shared memory where accumulators hold the
// output transposed (TMEM lane = output column, TMEM column = output row), and the
// activation.
#pragma once

#include <cstdint>

#include "moe_device.cuh"

namespace moe {

// Staging of 32 rows x 128 bf16 columns, written by the four warps of a turn:
// two halves of 64 columns, rows of 128 bytes, in the 128-byte swizzle of the
// stores' tensor map (which also puts eight rows on different banks).
constexpr int kPieceBytes = kPieceRows * 128 * 2;
static_assert(kPieceRows == 32, "a warp's piece of TMEM");
// byte offset of row t, 16-byte chunk c (of 16) in the staging (of `rows` rows)
__device__ __forceinline__ int staged_at(int t, int c, int rows = 32) {
  return (c >> 3) * (rows * 128) + t * 128 + (((c & 7) ^ (t & 7)) << 4);
}

// 16 TMEM lanes x 32 columns: thread i gets, for each group j of eight columns,
// lane i / 4, columns 8 j + 2 (i % 4) and the next (v[4 j], v[4 j + 1]) and the
// same of lane i / 4 + 8 (v[4 j + 2], v[4 j + 3]).
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

// A 32-lane x 32-column piece of an accumulator: lanes 0-15 in v[0..15], lanes
// 16-31 in v[16..31].
__device__ __forceinline__ void load_piece(uint32_t taddr, uint32_t (&v)[32]) {
  tmem_ld_16x256b_x4(taddr, v);
  tmem_ld_16x256b_x4(taddr + (16u << 16), v + 16);
}

// A piece to bf16 pairs: entry 4 j + x holds the columns 8 j + 2 (i % 4) and the
// next of TMEM lane 8 x + i / 4.
__device__ __forceinline__ constexpr int piece_entry(int k) { return (k & 2) * 8 + (k >> 2) * 4 + (k & 1) * 2; }
__device__ __forceinline__ void round_piece(const uint32_t (&v)[32], uint32_t (&out)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int i = piece_entry(k);
    out[k] = pack_bf16x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
  }
}

// Four 8 x 8 bf16 matrices to shared memory, transposed: thread i's pairs lie
// along a matrix row's neighbours 2 (i % 4), row i / 4; the address of row r of
// matrix m comes from thread 8 m + r.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// Writes a piece as bf16 to the staging at `out`, columns 32 q..: packed[4 j + x]
// holds the rows 8 j + 2 (i % 4) and the next of column x * 8 + i / 4, so matrix
// (j, x) lands at rows 8 j.., columns 32 q + 8 x...
__device__ __forceinline__ void stage_piece(uint32_t out, int q, const uint32_t (&packed)[16], int lane,
                                            int rows = 32) {
  const uint32_t at = out + staged_at(lane & 7, 4 * q + (lane >> 3), rows);  // thread 8 x + r: row r, columns 8 x
#pragma unroll
  for (int j = 0; j < 4; ++j)
    stmatrix_x4_trans(at + 8 * j * 128, packed[4 * j], packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
}

// Four 8 x 8 bf16 matrices from shared memory, transposed: the inverse of
// stmatrix_x4_trans, so that a piece in the staging reaches the threads in the
// layout of round_piece's result.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}

// silu(g) * u with the sigmoid on the SFU.  The exponent g log2 e is rounded
// before ex2, so below zero the relative error grows with |g|, to about
// |g| 2^-24 and a few ulps (2^-17 at g = -88, below which the result is the
// limit 0, as in the bf16 GEMM): far under h's rounding to bf16, 2^-9.
__device__ __forceinline__ float silu_mul(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return g * r * u;
}

}  // namespace moe
