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

// A thread's vector of a row in two steps, so that every load of a row is on its
// way before the first is waited for: fetch() the raw words, unpack() later;
// neither has a branch, at whose end the loads would be waited for.
//   kWhole  rows are whole vectors;
//   kTail   the last vector of a row is short: it is fetched as the row's last
//           eight elements and moved into place by unpack();
//   kShort  rows of less than eight elements, fetched one by one.
// A thread past the row fetches its start and unpacks zeros.
enum RowEnd { kWhole, kTail, kShort };

template <typename T>
struct Raw { u32x4 w; };
template <>
struct Raw<float> { f32x4 a, b; };

template <typename T>
__device__ __forceinline__ void keep(Raw<T>& r) { asm volatile("" : "+v"(r.w)); }
__device__ __forceinline__ void keep(Raw<float>& r) {
  asm volatile("" : "+v"(r.a));
  asm volatile("" : "+v"(r.b));
}

template <bool NT, typename T>
__device__ __forceinline__ Raw<T> fetch_at(const T* p) {
  const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(p);
  if constexpr (NT) return {__builtin_nontemporal_load(q)};
  else return {*q};
}
template <bool NT>
__device__ __forceinline__ Raw<float> fetch_at(const float* p) {
  const f32x4_a4* q = reinterpret_cast<const f32x4_a4*>(p);
  if constexpr (NT) return {__builtin_nontemporal_load(q), __builtin_nontemporal_load(q + 1)};
  else return {q[0], q[1]};
}
__device__ __forceinline__ void unpack_raw(const Raw<float>& r, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = r.a[i];
    f[4 + i] = r.b[i];
  }
}
template <typename T>
__device__ __forceinline__ void unpack_raw(const Raw<T>& r, float (&f)[8]) {
  unpack8(r.w, f, T{});
}

// (the elements past the row are its last one again)
template <typename T>
__device__ __forceinline__ Raw<T> fetch_short(const T* row, int H) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (uint32_t)__builtin_bit_cast(uint16_t, row[min(2 * i, H - 1)]) |
           (uint32_t)__builtin_bit_cast(uint16_t, row[min(2 * i + 1, H - 1)]) << 16;
  return {w};
}
__device__ __forceinline__ Raw<float> fetch_short(const float* row, int H) {
  Raw<float> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.a[i] = row[min(i, H - 1)];
    r.b[i] = row[min(4 + i, H - 1)];
  }
  return r;
}

// where the mask has ones a's bit, else b's (v_bfi_b32)
__device__ __forceinline__ uint32_t merge(uint32_t mask, uint32_t a, uint32_t b) { return (a & mask) | (b & ~mask); }

// The eight elements moved down by `by` places.  Merged by masks: written as
// selections, the compiler turns the three steps into a search for each
// element's index.
struct MoveDown {
  uint32_t one, two, four;  // all ones if `by` has that bit
  __device__ __forceinline__ explicit MoveDown(int by)
      : one(0u - (by & 1)), two(0u - (by >> 1 & 1)), four(0u - (by >> 2 & 1)) {}
  __device__ __forceinline__ void operator()(Raw<float>& r) const {
    uint32_t f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = __float_as_uint(r.a[i]);
      f[4 + i] = __float_as_uint(r.b[i]);
    }
#pragma unroll
    for (int i = 0; i < 7; ++i) f[i] = merge(one, f[i + 1], f[i]);
#pragma unroll
    for (int i = 0; i < 6; ++i) f[i] = merge(two, f[i + 2], f[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = merge(four, f[i + 4], f[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.a[i] = __uint_as_float(f[i]);
      r.b[i] = __uint_as_float(f[4 + i]);
    }
  }
  template <typename T>
  __device__ __forceinline__ void operator()(Raw<T>& r) const {
#pragma unroll
    for (int i = 0; i < 3; ++i) r.w[i] = merge(two, r.w[i + 1], r.w[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) r.w[i] = merge(four, r.w[i + 2], r.w[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = __builtin_amdgcn_alignbit(i < 3 ? r.w[i + 1] : 0u, r.w[i], one & 16u);
  }
};

// The vector at `col` of a row of H elements, n = H - col of them its own.
template <RowEnd END>
struct Place {
  int from, n;  // where it is fetched
  MoveDown move;
  // all ones for the row's own elements, kept as words: as conditions the
  // eight would not fit the scalar registers
  uint32_t own[END == kWhole ? 1 : 8];
  __device__ __forceinline__ Place(int col, int H)
      : from(END == kTail && H - col > 0 && H - col < 8 ? H - 8 : H - col > 0 ? col : 0),
        n(H - col),
        move(H - col > 0 ? col - from : 0) {
    if constexpr (END != kWhole) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        own[i] = i < n ? ~0u : 0u;
        asm volatile("" : "+v"(own[i]));
      }
    }
  }
  template <bool NT, typename T>
  __device__ __forceinline__ Raw<T> fetch(const T* row, int H) const {
    if constexpr (END == kShort) return fetch_short(row, H);
    else return fetch_at<NT>(row + from);
  }
  // v where element e of the vector is the row's, else 0
  __device__ __forceinline__ float only(int e, float v) const {
    if constexpr (END == kWhole) return n > 0 ? v : 0.f;
    else return __uint_as_float(__float_as_uint(v) & own[e]);
  }
  template <typename T>
  __device__ __forceinline__ void unpack(Raw<T> r, float (&f)[8]) const {
    if constexpr (END == kTail) move(r);
    unpack_raw(r, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = only(i, f[i]);
  }
  template <bool NT, typename T>
  __device__ __forceinline__ void store(T* at, const float (&f)[8]) const {  // at: the vector's own place
    if (n <= 0) return;
    if constexpr (END == kWhole) store8<NT>(at, f);
    else store_n<NT>(at, n, f);
  }
};

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
