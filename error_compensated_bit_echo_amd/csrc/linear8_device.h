// linear8_device.h -- gfx950 kernels' common parts of the matrix product in 8-bit
// floating point, out[i][j] = sum over blocks b of sx[i][b] sw[j / 128][b] times the
// sum over c in b of x[i][c] w[j][c].
//
// A step of the contraction is one block of 128, one v_mfma_f32_16x16x128_f8f6f4 a
// pair of fragments: lane 16 g + rho holds, for row rho of a fragment's 16, the
// sixteen bytes of chunk g and those of chunk g + 4 of the row's 128.  (The order of
// the contraction within a block is free as long as both operands have the same.)
// w is the instruction's first operand, so a lane's four sums are neighbours along j
// and belong to one row of x: one scale of x and one of w for each fragment pair.
//
// What the instruction rounds (measured with products of single powers of two): the
// products of eight neighbours of the contraction are cut towards zero at 2^(E - 13),
// E the largest sum of two codes' exponents among them (a subnormal code's counts as
// the smallest normal one's); the sum of the eight, those of the other eights and the
// accumulator are added as binary32, to nearest.  Root-mean-square error of a sum of
// products of normal values 1.3e-5 of its own, against 2.1e-4 of one rounding to
// half.  The 16-bit instructions on the converted codes would cut nothing, at twice
// the time of the matrix cores and of LDS.
#pragma once

#include "fp8_device.h"
#include "linear8_plan.h"
#include "linear_tile.h"

namespace echo {

struct Tile8Args : TileArgs {
  const float *sx, *sw;
  int32_t wide;  // rows of scales are whole and aligned groups of four
};

// X: 0 if x is e4m3, 1 if e5m2 (the instruction's own numbers)
template <int X>
__device__ __forceinline__ f32x4 mfma8(i32x8 w, i32x8 x, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, X, 0, 0, 0, 0);
}
// the same with the operands' scales 2^(ew - 127) and 2^(ex - 127) applied
template <int X>
__device__ __forceinline__ f32x4 mfma8(i32x8 w, i32x8 x, f32x4 c, int ew, int ex) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, X, 0, ew, 0, ex);
}

// whether a scale is a power of two that the instruction's exponent holds
__device__ __forceinline__ bool is_power(uint32_t bits) {
  return (bits & 0x807FFFFFu) == 0 && bits - 0x00800000u < 0x7F000000u;
}

__device__ __forceinline__ i32x8 join16(u32x4 a, u32x4 b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// ones in the bytes of a word that lie before `n`
__device__ __forceinline__ uint32_t bytes_before(int n) {
  return n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
}
__device__ __forceinline__ u32x4 chunk_before(u32x4 w, int n) {
#pragma unroll
  for (int d = 0; d < 4; ++d) w[d] &= bytes_before(n - 4 * d);
  return w;
}

// a decode step's: at most kFewRows rows of x
int rows8_forward(const Tile8Args& a, int32_t dtype, int32_t format, bool gated, hipStream_t s);

}  // namespace echo
