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
// a code's value before its rounding to T; finite codes stay finite
template <typename T>
__device__ __forceinline__ float value_of(float code, float scale) {
  const float v = code * scale;
  return fabsf(v) > largest_of<T>() && fabsf(code) < __builtin_inff() ? copysignf(largest_of<T>(), v) : v;
}

// eight codes times their scale
template <typename T, int FORMAT>
__device__ __forceinline__ void values_of(u32x2 w, float scale, float (&f)[8]) {
  values_of<FORMAT>(w, f);
  if (may_pass<T, FORMAT>(scale)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = value_of<T>(f[i], scale);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= scale;
  }
}

}  // namespace echo
