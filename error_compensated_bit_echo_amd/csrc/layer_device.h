// layer_device.h -- gfx950 device helpers of the layer operators: element
// types, 8-element vectors of any alignment, sums over a wavefront.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace echo {

struct bf16_t { uint16_t bits; };
typedef _Float16 f16_t;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// The same 16 bytes at an address aligned to one element only: the global
// load and store instructions of gfx950 take any alignment, so rows of odd
// lengths need no second code path.
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

__device__ __forceinline__ float to_f32(bf16_t v) { return __uint_as_float((uint32_t)v.bits << 16); }
__device__ __forceinline__ float to_f32(f16_t v) { return (float)v; }
__device__ __forceinline__ float to_f32(float v) { return v; }

// round to nearest even (v_cvt_pk_bf16_f32, v_cvt_f16_f32)
__device__ __forceinline__ uint32_t pack2(float a, float b, bf16_t) {
  typedef __bf16 h2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, h2));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, f16_t) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, h2));
}
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  const uint16_t b = (uint16_t)pack2(v, v, T{});
  return __builtin_bit_cast(T, b);
}
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

__device__ __forceinline__ void unpack8(u32x4 w, float (&f)[8], bf16_t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack8(u32x4 w, float (&f)[8], f16_t) {
  typedef _Float16 h8 __attribute__((ext_vector_type(8)));
  const h8 h = __builtin_bit_cast(h8, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = (float)h[i];
}

// Eight elements at p (element-aligned) as binary32; of the last vector of a
// row only the first n < 8 exist and the others read as `fill`.  NT marks a
// tensor that is read once.
template <bool NT, typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(p);
  u32x4 w;
  if constexpr (NT) w = __builtin_nontemporal_load(q);
  else w = *q;
  unpack8(w, f, T{});
}
template <bool NT>
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const f32x4_a4* q = reinterpret_cast<const f32x4_a4*>(p);
  f32x4 a, b;
  if constexpr (NT) {
    a = __builtin_nontemporal_load(q);
    b = __builtin_nontemporal_load(q + 1);
  } else {
    a = q[0];
    b = q[1];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = a[i];
    f[4 + i] = b[i];
  }
}
template <bool NT, typename T>
__device__ __forceinline__ void load_n(const T* p, int n, float (&f)[8], float fill = 0.f) {
  if (n >= 8) return load8<NT>(p, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = i < n ? to_f32(p[i]) : fill;
}

template <bool NT, typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2(f[2 * i], f[2 * i + 1], T{});
  u32x4_a2* q = reinterpret_cast<u32x4_a2*>(p);
  if constexpr (NT) __builtin_nontemporal_store(w, q);
  else *q = w;
}
template <bool NT>
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  f32x4_a4* q = reinterpret_cast<f32x4_a4*>(p);
  const f32x4 a = {f[0], f[1], f[2], f[3]}, b = {f[4], f[5], f[6], f[7]};
  if constexpr (NT) {
    __builtin_nontemporal_store(a, q);
    __builtin_nontemporal_store(b, q + 1);
  } else {
    q[0] = a;
    q[1] = b;
  }
}
template <bool NT, typename T>
__device__ __forceinline__ void store_n(T* p, int n, const float (&f)[8]) {
  if (n >= 8) return store8<NT>(p, f);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = from_f32<T>(f[i]);
}

// The same for W = 4 or 8 elements of a 16-bit type.
template <typename T, int W>
__device__ __forceinline__ void load_w(const T* p, int n, float (&f)[W]) {
  if constexpr (W == 8) {
    load_n<false>(p, n, f);
  } else {
    u32x2 w = {0, 0};
    if (n >= 4) {
      w = *reinterpret_cast<const u32x2_a2*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) w[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[i]) << (i % 2 * 16);
    }
    float g[8];
    unpack8(u32x4{w[0], w[1], 0, 0}, g, T{});
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = g[i];
  }
}
template <typename T, int W>
__device__ __forceinline__ void store_w(T* p, int n, const float (&f)[W]) {
  if constexpr (W == 8) {
    store_n<false>(p, n, f);
  } else if (n >= 4) {
    const u32x2 w = {pack2(f[0], f[1], T{}), pack2(f[2], f[3], T{})};
    *reinterpret_cast<u32x2_a2*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < n) p[i] = from_f32<T>(f[i]);
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}

// Sum over the 64 lanes, the same value and the same order of additions in
// every lane (all lanes must be active).
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f32<0xB1>(v);   // quad_perm [1,0,3,2]: lane ^ 1
  v += dpp_f32<0x4E>(v);   // quad_perm [2,3,0,1]: lane ^ 2
  v += dpp_f32<0x141>(v);  // row_half_mirror
  v += dpp_f32<0x140>(v);  // row_mirror: the row of 16 holds its sum
  const int b = (int)__float_as_uint(v);
  const float r0 = __uint_as_float((uint32_t)__builtin_amdgcn_readlane(b, 0));
  const float r1 = __uint_as_float((uint32_t)__builtin_amdgcn_readlane(b, 16));
  const float r2 = __uint_as_float((uint32_t)__builtin_amdgcn_readlane(b, 32));
  const float r3 = __uint_as_float((uint32_t)__builtin_amdgcn_readlane(b, 48));
  return (r0 + r1) + (r2 + r3);
}

}  // namespace echo
