// linear_device.h -- gfx950 kernels of the matrix products with an epilogue.
//
// One kernel template covers the three products of a layer, each of the form
// C[i][j] = sum over c of A(i, c) B(j, c):
//   forward   out = x w^T     A = x  [m][k]    B = w [n][k]    c along the rows
//   dx        dx  = dp w      A = dp [m][n]    B = w [n][k]^T  c across B's rows
//   dw        dw  = dp^T x    A = dp [m][n]^T  B = x [m][k]^T  c across both
// A workgroup computes a BI x BJ tile of C in steps of kC = 64 along c.  Both
// operands' tiles are staged in LDS, two to four stages deep, and feed
// v_mfma_f32_16x16x32: lane l of a wavefront holds, for row (or column) l % 16
// of an operand's 16, the eight elements c = 8 (l / 16) .. + 7 of the 32.
// B's fragment goes into the instruction's first operand, so a lane's four sums
// are neighbours along j.
//
// LDS.  An operand whose rows run along c is stored row by row, 64 elements =
// eight 16-byte chunks each, and a lane reads its eight elements with one
// ds_read_b128.  An operand that c runs across is stored as it lies in memory,
// 64 rows of c, and read with ds_read_b64_tr_b16: sixteen lanes read four rows
// of sixteen elements and get them transposed.  Either way the chunks of a row
// are permuted by an exclusive-or with bits of the row's number, so the lanes
// of one read spread over the banks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <type_traits>

#include "echo_layer.h"
#include "layer_device.h"
#include "linear_plan.h"

namespace echo {

// addresses in LDS, as such: through a generic pointer the compiler loses track
// of which buffer a transposed read is from and waits for every load in flight
typedef __attribute__((address_space(3))) short lds_short;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

struct TileArgs {
  const void *a, *b;
  int64_t lda, ldb;
  int64_t I, J, C;  // J counts outputs: gated, B has 2J rows
  int64_t chunk;    // contraction length of one split, a multiple of kC
  float* part;      // splits > 1: binary32 sums, [splits][I][columns of B]
  void *out, *p;
  const void *bias, *residual;
  int64_t ldo, ldr;
  uint32_t tiles_i, tiles_j, splits, workgroups;  // workgroups: tiles of all splits
  int32_t act;
  int32_t padded;   // rows along c are followed by zeros up to a whole chunk
};

// ---- activations ---------------------------------------------------------------
// exp through v_exp_f32 (2^x): the rounded product p log2(e) costs |p| 2^-24
// relative, below 2^-17 wherever the result is not already 0 or infinite, far
// under the half unit of a 16-bit output; so does v_rcp_f32 (one ulp).
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp_fast(-x));
}
// Normal distribution function, erfc(-x / sqrt 2) / 2.  With z = |x| / sqrt 2 and t =
// 1 / (1 + 0.4 z), erfc(z) = exp(-z^2) t P(t) for a smooth P on (0, 1]; P / 2
// below is a polynomial of degree 8 fitted to erfc(z) exp(z^2) / t in binary64
// (least squares of the relative error, reweighted towards its largest), good to
// 1e-7 for all z, so the far negative tail keeps its digits.
__device__ __forceinline__ float normal_cdf(float x) {
  constexpr float c[9] = {0.112831444f, 0.11296837f, 0.102805234f, 0.0892399177f, 0.0577344857f, 0.0177173372f, 0.0652485639f, -0.0815293491f, 0.022984039f};
  const float t = __builtin_amdgcn_rcpf(fmaf(0.28284271f, fabsf(x), 1.0f));
  float p = c[8];
#pragma unroll
  for (int i = 7; i >= 0; --i) p = fmaf(p, t, c[i]);
  p *= t * exp_fast(-0.5f * x * x);
  return x < 0.f ? p : 1.0f - p;
}
// (1 + tanh a) / 2 = sigmoid(2 a), a = sqrt(2/pi) (x + 0.044715 x^3)
__device__ __forceinline__ float gelu_tanh_gate(float x) {
  return sigmoid(1.59576912f * fmaf(0.044715f * x * x, x, x));
}

// value and slope of each activation
template <int ACT>
__device__ __forceinline__ void act_slope(float p, float& v, float& d) {
  if constexpr (ACT == ECHO_ACT_RELU) {
    v = p <= 0.f ? 0.f : p;
    d = p > 0.f ? 1.f : 0.f;
  } else if constexpr (ACT == ECHO_ACT_GELU) {
    const float c = normal_cdf(p);
    v = p * c;
    d = fmaf(p * 0.39894228f, exp_fast(-0.5f * p * p), c);
  } else if constexpr (ACT == ECHO_ACT_GELU_TANH) {
    const float s = gelu_tanh_gate(p);
    v = p * s;
    // p^2 capped where 1 - s or v is 0 long before it, so that it is never infinite
    d = fmaf(v * (1.f - s), 1.59576912f * fmaf(0.134145f, fminf(p * p, 1e30f), 1.f), s);
  } else if constexpr (ACT == ECHO_ACT_SILU) {
    const float s = sigmoid(p);
    v = p * s;
    d = fmaf(v, 1.f - s, s);
  } else {
    v = p;
    d = 1.f;
  }
}

// f<ACT>() for the activation a call names: one branch for a whole vector
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case ECHO_ACT_RELU: return f(std::integral_constant<int, ECHO_ACT_RELU>{});
    case ECHO_ACT_GELU: return f(std::integral_constant<int, ECHO_ACT_GELU>{});
    case ECHO_ACT_GELU_TANH: return f(std::integral_constant<int, ECHO_ACT_GELU_TANH>{});
    case ECHO_ACT_SILU: return f(std::integral_constant<int, ECHO_ACT_SILU>{});
    default: return f(std::integral_constant<int, ECHO_ACT_NONE>{});
  }
}

// ---- epilogue --------------------------------------------------------------------
// g: W neighbouring sums of row i from column j (gated: the gate's, and u the
// up rows'), of which the first n exist.
template <typename T, int W, bool GATED>
__device__ __forceinline__ void finish(const TileArgs& a, int64_t i, int64_t j, int n, float (&g)[W],
                                       float (&u)[W]) {
  const int64_t cols = GATED ? 2 * a.J : a.J;
  float f[W];
  if (a.bias) {
    load_w<T, W>((const T*)a.bias + j, n, f);
#pragma unroll
    for (int e = 0; e < W; ++e) g[e] += f[e];
    if constexpr (GATED) {
      load_w<T, W>((const T*)a.bias + a.J + j, n, f);
#pragma unroll
      for (int e = 0; e < W; ++e) u[e] += f[e];
    }
  }
  if (a.p) {
    T* p = (T*)a.p + i * cols + j;
    store_w<T, W>(p, n, g);
    if constexpr (GATED) store_w<T, W>(p + a.J, n, u);
  }
  with_act(a.act, [&](auto act) {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      float slope;
      act_slope<decltype(act)::value>(g[e], g[e], slope);
    }
  });
  if constexpr (GATED) {
#pragma unroll
    for (int e = 0; e < W; ++e) g[e] *= u[e];
  }
  if (a.residual) {
    load_w<T, W>((const T*)a.residual + i * a.ldr + j, n, f);
#pragma unroll
    for (int e = 0; e < W; ++e) g[e] += f[e];
  }
  store_w<T, W>((T*)a.out + i * a.ldo + j, n, g);
}

// ---- operand tiles ---------------------------------------------------------------
__device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c, bf16_t) {
  typedef __bf16 v8 __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b),
                                                 c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c, f16_t) {
  typedef _Float16 v8 __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b),
                                                c, 0, 0, 0);
}

// R rows of an operand by kC of the contraction, NT threads staging it.
template <bool ACROSS, int R, int NT>
struct OperandTile {
  static constexpr int kChunks = R * kC / 8;  // 16-byte chunks
  static constexpr int kPer = kChunks / NT;   // of a thread
  static constexpr int kRow = ACROSS ? R / 8 : kC / 8;  // chunks of a stored row
  static_assert(kChunks % NT == 0, "chunks per thread");

  static __device__ __forceinline__ int spread(int row) {
    if (ACROSS) return ((row & 3) | (row >> 1 & 4)) & (R / 16 - 1);
    return row & 7;
  }
  // chunk of its row that is stored at place pc of row `row`, and back
  static __device__ __forceinline__ int place(int row, int pc) {
    return ACROSS ? pc ^ (spread(row) << 1) : pc ^ spread(row);
  }
  // eight elements c = kk*32 + 8 g .. of row rho of the 16 of fragment t (lane = 16 g + rho)
  static __device__ __forceinline__ s16x8 fragment(const lds_short* lds, int t, int kk, int lane, int base) {
    const int g = lane >> 4, rho = lane & 15;
    if constexpr (!ACROSS) {
      const int row = base + t * 16 + rho;
      typedef __attribute__((address_space(3))) const s16x8 lds8;
      return *(lds8*)(lds + row * kC + place(row, kk * 4 + g) * 8);
    } else {
      typedef __attribute__((address_space(3))) s16x4 lds4;
      s16x4 h[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int c = kk * 32 + g * 8 + q * 4 + (rho >> 2);
        const int chunk = (base + t * 16) / 8 + (rho >> 1 & 1);
        const lds_short* p = lds + c * R + place(c, chunk) * 8 + (rho & 1) * 4;
        h[q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
      }
      return __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// Gated, B's tile alternates runs of 32 gate rows and the 32 up rows of the same
// outputs, so one lane holds both sums of an output: row r of the tile belongs
// to output (r / 64) 32 + r % 32, and bit 5 of r says up.

// Workgroups are dealt to the 8 XCDs in turn; renumbered, an XCD takes one run
// of tiles, and runs go over a band of tile rows before the next tile column, so
// that the 32 tiles in flight on an XCD share operands in its L2: 8 rows by 4
// columns, or, where there are fewer columns, all of them by as many rows
// (131072 x 1792 x 4096, seven columns: bands of 4 rows 1541 us, of 8 1580).  A
// split's tiles follow each other, so that its part of both operands is read by
// one XCD or two.
__device__ __forceinline__ void tile_of(uint32_t b, uint32_t nb, uint32_t tiles_i, uint32_t tiles_j,
                                        uint32_t& ti, uint32_t& tj, uint32_t& split) {
  const uint32_t xcd = b % 8, k = b / 8, per = nb / 8, extra = nb % 8, tiles = tiles_i * tiles_j;
  uint32_t t = xcd * per + (xcd < extra ? xcd : extra) + k;
  split = tiles == nb ? 0 : t / tiles;
  t -= split * tiles;
  const uint32_t rows_of = tiles_j >= 8 ? 8 : 32 / tiles_j;
  const uint32_t band = t / (rows_of * tiles_j), first = band * rows_of;
  const uint32_t rows = min(rows_of, tiles_i - first), r = t - first * tiles_j;
  ti = first + r % rows;
  tj = r / rows;
}

}  // namespace echo
