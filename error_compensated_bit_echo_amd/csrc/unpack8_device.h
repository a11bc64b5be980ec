// unpack8_device.h -- codes times scales to a 16- or 32-bit matrix: a kernel of its own,
// and a part of the backward call's first.
#pragma once

#include "fp8_device.h"
#include "launch_shape.h"

namespace echo {

// A division of numbers below 2^31 by a launch's constant d > 1: with L = ceil(log2 d) and m
// = floor(2^(31 + L) / d) + 1, which 32 bits hold, t m is above t 2^(31 + L) / d by at most t,
// less than 2^(31 + L) / d, so its part past 2^(31 + L) is t / d.
struct Divisor {
  uint32_t d, m, shift;  // shift: L - 1; m 0: numbers are not below 2^31, or d is 1
  static Divisor of(uint32_t d, int64_t items) {
    Divisor v = {d, 0, 0};
    if (d < 2 || items > INT64_C(0x7FFFFFFF)) return v;
    uint32_t L = 1;
    while ((UINT64_C(1) << L) < d) ++L;
    v.m = (uint32_t)((UINT64_C(1) << (31 + L)) / d + 1);
    v.shift = L - 1;
    return v;
  }
  __device__ __forceinline__ int64_t quotient(int64_t t) const {
    if (m) return (int64_t)(__umulhi((uint32_t)t, m) >> shift);
    return d < 2 ? t : t / d;
  }
};

struct Unpack8Args {
  const void* codes;
  const float* scales;
  void* x;
  int64_t rows, cols, fill;  // of a part; zeros are written from cols to fill
  int64_t ld_x, ld_c, x_part, c_part, s_part, ld_s;
  int64_t items;  // vectors of eight of all parts
  uint32_t parts, vectors;  // vectors of a row of a part
  Divisor per_row;          // of a row
  int32_t blocks;
  // a row (of a part) is a multiple of a wavefront's 512 elements
  bool runs() const { return cols % 512 == 0 && fill == cols; }
};

inline uint32_t unpack_blocks(const Unpack8Args& a) { return blocks_for_items(((uint64_t)a.items + 1) / 2); }

// m rows of k codes in blocks of 1 x 128 to rows of pitch ld, filled up with zeros
inline Unpack8Args unpack_args(const void* codes, int64_t ld_c, const float* scales, int64_t m, int64_t k, void* x, int64_t ld) {
  Unpack8Args a = {};
  a.codes = codes;
  a.scales = scales;
  a.x = x;
  a.rows = m;
  a.cols = k;
  a.fill = a.ld_x = ld;
  a.ld_c = ld_c;
  a.ld_s = (k + ECHO_FP8_BLOCK - 1) / ECHO_FP8_BLOCK;
  a.parts = 1;
  a.vectors = (uint32_t)((ld + 7) / 8);
  a.items = m * a.vectors;
  a.per_row = Divisor::of(a.vectors, a.items);
  return a;
}

// Where item t, or the wavefront's lane, stands: RUN says that a wavefront's items follow
// each other in one row, whose place scalar registers then have.
template <bool RUN>
__device__ __forceinline__ int64_t lead(int64_t t) {
  if constexpr (!RUN) return t;
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)t) |
                   (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(t >> 32)) << 32);
}

// Twice eight elements to a thread.  RUN: a row (of a part) is a multiple of 512 elements,
// a wavefront's.
template <typename T, int FORMAT, bool RUN>
__device__ __forceinline__ void unpack8(const Unpack8Args& a, uint32_t block, uint32_t blocks) {
  constexpr int U = 2;
  for (int64_t t0 = (int64_t)block * U * kBlock + threadIdx.x; t0 < a.items; t0 += (int64_t)blocks * U * kBlock) {
    u32x2 w[U];
    float s[U];
    T* x[U];
    int n[U], room[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {  // past the end the last vector once more
      const int64_t t = RUN ? min(lead<RUN>(t0 + u * kBlock), a.items - 64) : min(t0 + u * kBlock, a.items - 1);
      const int64_t line = a.per_row.quotient(t);
      uint32_t v = (uint32_t)(t - line * a.per_row.d), q = 0;
      if (a.parts == 2 && v >= a.vectors) {
        v -= a.vectors;
        q = 1;
      }
      // (where zeros fill the row up, a vector may begin past its last element)
      const int64_t col = (int64_t)v * 8 + (RUN ? (int)(threadIdx.x & 63) * 8 : 0);
      const int64_t at = RUN ? col : min(col, (a.cols - 1) / 8 * 8);
      n[u] = (int)min(a.cols - col, (int64_t)8);
      room[u] = (int)min(a.fill - col, (int64_t)8);
      x[u] = (T*)a.x + line * a.ld_x + q * a.x_part + col;
      // a row's last eight bytes lie within the sixteen that its pitch rounds up to
      w[u] = *(const u32x2_a1*)((const uint8_t*)a.codes + line * a.ld_c + q * a.c_part + at);
      s[u] = a.scales[q * a.s_part + (a.blocks ? line / ECHO_FP8_BLOCK : line) * a.ld_s + at / ECHO_FP8_BLOCK];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t0 + u * kBlock >= a.items) break;
      float f[8];
      values_of<T, FORMAT>(w[u], s[u], f);
      if (n[u] < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < n[u] ? f[i] : 0.f;
      }
      store_n<true>(x[u], room[u], f);
    }
  }
}

}  // namespace echo
