// fp8_device.h -- gfx950 device helpers of the operators in 8-bit floating point:
// codes to and from binary32, and a block's scale.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <type_traits>

#include "echo_fp8.h"
#include "layer_device.h"

namespace echo {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

// eight codes, in the order of their bytes (v_cvt_pk_fp8_f32, v_cvt_pk_bf8_f32:
// nearest even; nothing past the largest code comes here but inf and NaN)
template <int FORMAT>
__device__ __forceinline__ u32x2 codes_of(const float (&f)[8]) {
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int c = 0;
    if constexpr (FORMAT == ECHO_E4M3) {
      c = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], c, false);
      c = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], c, true);
    } else {
      c = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * i], f[4 * i + 1], c, false);
      c = __builtin_amdgcn_cvt_pk_bf8_f32(f[4 * i + 2], f[4 * i + 3], c, true);
    }
    w[i] = (uint32_t)c;
  }
  return w;
}

template <int FORMAT>
__device__ __forceinline__ void values_of(u32x2 w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f32x2 lo, hi;
    if constexpr (FORMAT == ECHO_E4M3) {
      lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
      hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
    } else {
      lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)w[i], false);
      hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)w[i], true);
    }
    f[4 * i] = lo[0];
    f[4 * i + 1] = lo[1];
    f[4 * i + 2] = hi[0];
    f[4 * i + 3] = hi[1];
  }
}

// |v|'s bits, which order as the magnitudes do; 0 for inf and NaN
__device__ __forceinline__ uint32_t magnitude(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}

// A block's scale exponent, biased by 127, for the bits of its largest magnitude.
// The largest code of both formats is 1.75 times a power of two, 2^8 or 2^15: the
// magnitude's own exponent, and one more where its fraction is past .75, less that.
template <int FORMAT>
__device__ __forceinline__ int scale_exponent(uint32_t largest) {
  if (largest == 0) return 127;
  const int e = (int)((largest + 0x1FFFFFu) >> 23) - (FORMAT == ECHO_E4M3 ? 8 : 15);
  return e > 1 ? e : 1;
}
__device__ __forceinline__ float power_of_two(int biased) { return __uint_as_float((uint32_t)biased << 23); }

// largest of sixteen neighbouring lanes, in all of them
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  auto step = [&](auto ctrl) {
    const uint32_t o =
        (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xF, 0xF, false);
    v = o > v ? o : v;
  };
  step(std::integral_constant<int, 0xB1>{});   // lane ^ 1
  step(std::integral_constant<int, 0x4E>{});   // lane ^ 2
  step(std::integral_constant<int, 0x141>{});  // row_half_mirror
  step(std::integral_constant<int, 0x140>{});  // row_mirror
  return v;
}

// the elements of a vector from the n-th on set to 0
template <typename T>
__device__ __forceinline__ void clear_from(Raw<T>& r, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] &= n >= 2 * i + 2 ? ~0u : n == 2 * i + 1 ? 0xFFFFu : 0u;
}
__device__ __forceinline__ void clear_from(Raw<float>& r, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.a[i] = i < n ? r.a[i] : 0.f;
    r.b[i] = i + 4 < n ? r.b[i] : 0.f;
  }
}

template <typename T>
__device__ constexpr float largest_of() {
  return std::is_same<T, f16_t>::value ? 65504.f : std::is_same<T, bf16_t>::value ? 3.38953139e38f : 3.40282347e38f;
}

// whether a block's codes, times its scale, may pass T's range (or the scale is inf)
template <typename T, int FORMAT>
__device__ __forceinline__ bool may_pass(float scale) {
  return fabsf(scale) > largest_of<T>() / (FORMAT == ECHO_E4M3 ? 448.f : 57344.f);
}
// Code times scale, then rounded to a 16-bit type, is rounded once: binary32 holds the product
// where a scale has no more than 20 digits, which makes 24 with a code's, and lies above the
// subnormal numbers; of others a number halfway between two of the type may be one that the
// product was rounded to.
__device__ __forceinline__ bool may_lose(float scale) {
  const uint32_t b = __float_as_uint(scale);
  return (b & 15) != 0 || ((b & 0x007FFFFFu) != 0 && fabsf(scale) < 0x1p-100f);
}
// Whether one of eight may lie halfway between two numbers of T.  Its last 16 bits say so
// for bfloat16; for half, whose subnormal numbers have their digits further up, the last 12
// are 0, as they are for 0, which is looked for only then.
template <typename T>
__device__ __forceinline__ bool any_halfway(const float (&f)[8]) {
  constexpr bool kHalf = std::is_same<T, f16_t>::value;
  uint32_t least = ~0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(f[i]);
    least = min(least, kHalf ? b << 20 : (b << 16) + 0x80000000u);
  }
  if (least > 0 || !kHalf) return least == 0;
  bool any = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) any |= (__float_as_uint(f[i]) & 0xFFFu) == 0 && f[i] != 0.f;
  return any;
}
// The product rounded to odd: of the two binary32 numbers around one that is neither, that
// with its last bit set, which lies halfway between no two of a 16-bit type and on the
// product's side.  `up` lifts products of small scales from below binary32's smallest number.
// Unpacked with scales of all digits 32768 x 1024 takes 16.5 us (bf16) and 16.2 (f16), as with
// powers of two; every product to odd took 20.2, its remainder from binary64 23.
__device__ __forceinline__ float times_to_odd(float code, float scale) {
  const float v = code * scale, up = fabsf(scale) < 1.f ? 0x1p64f : 1.f;
  const float rest = fmaf(code, scale * up, -(v * up));
  const uint32_t b = __float_as_uint(v);
  const int outwards = (int)(__float_as_uint(rest) ^ b) >> 31 | 1;  // 1: the product is larger
  return __uint_as_float((b & 1) == 0 && (rest < 0.f || rest > 0.f) ? b + outwards : b);
}

// eight codes times their scale, to be rounded to T; finite codes stay finite
template <typename T, int FORMAT>
__device__ __forceinline__ void values_of(u32x2 w, float scale, float (&f)[8]) {
  values_of<FORMAT>(w, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] *= scale;
  if constexpr (sizeof(T) == 2) {
    if (may_lose(scale)) {
      if (any_halfway<T>(f)) {
        values_of<FORMAT>(w, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = times_to_odd(f[i], scale);
      }
    }
  }
  if (may_pass<T, FORMAT>(scale)) {
    float c[8];
    values_of<FORMAT>(w, c);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(f[i]) > largest_of<T>() && fabsf(c[i]) < __builtin_inff()) f[i] = copysignf(largest_of<T>(), f[i]);
  }
}

}  // namespace echo
