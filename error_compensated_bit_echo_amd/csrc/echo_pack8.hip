// echo_pack8.hip -- matrices to codes in 8-bit floating point with a scale for each
// block of 128, and back (include/echo_fp8.h).
//
// Bound by HBM: a 16-bit element is read in two bytes and written in one, or the
// other way round.  A thread has eight neighbours of a row, so that a wavefront's
// loads and stores are each one run, and sixteen threads have a block's 128 columns,
// whose largest magnitude comes from four steps over their lanes (DPP).  Two such
// vectors a thread, both on their way before the first is used, and stores that do not
// stay in the caches: 8192 x 4096 bf16 packed in 16.9 us (6.0 TB/s) and 32768 x 1024
// unpacked in 16.2 (6.3 TB/s; a large copy reaches 6.5), 17 to 20 us with one vector, with
// cached stores or with uncached loads, 31 with sixteen neighbours a thread.  256 x 4096
// takes 3.2 us, which is latency.  Rows are found by a multiplication and, where a
// wavefront stays in one row, in scalar registers (packed 21.0 -> 18.2 us with its launch,
// unpacked 23.4 -> 16.7; 4072 x 2051 f16 from e5m2 8.9 -> 7.7).  Dividing by the scale is
// a multiplication with its reciprocal, exact for a power of two.
// Other forms, a call each: binary32 packed (8192 x 4096) 29.7 us and unpacked 46 (floor 26),
// 128 x 128 blocks of 3584 x 4096 packed without the transpose 9.5 and unpacked 8.4, 10.6 of
// two parts (two launches); unpacked with scales that are no powers of two 16.5 (32768 x 1024).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "echo_fp8.h"
#include "fp8_device.h"
#include "fp8_host.h"
#include "host_checks.h"
#include "unpack8_device.h"

using namespace echo;

namespace {

// One matrix, or its parts: part q's elements, codes and scales begin x_part,
// c_part and s_part elements behind the part before.
struct Pack8Args {
  const void* x;
  void* codes;
  float* scales;
  void* codes_t;   // nullable
  float* scales_t;
  int64_t rows, cols;  // of a part
  int64_t ld_x, ld_c, ld_t;
  int64_t x_part, c_part, s_part;
  int64_t ld_s, ld_st;  // row pitches of the scales
  int64_t items;        // blocks of all parts
  uint32_t parts, across, down;  // blocks along a row of a part, and above each other
  Divisor per_row;               // blocks of 1 x 128: of a row
};

// the vector at p, of whose eight elements the row has n
template <typename T, bool WHOLE>
__device__ __forceinline__ void load_row(const T* p, int64_t n, float (&f)[8]) {
  if constexpr (WHOLE) {
    if (n > 0) return load8<false>(p, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.f;
  } else {
    load_n<false>(p, (int)(n < 8 ? n : 8), f);
  }
}

template <bool NT>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t n, u32x2 w) {
  if (n >= 8) {
    if constexpr (NT) __builtin_nontemporal_store(w, (u32x2_a1*)p);
    else *(u32x2_a1*)p = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) p[i] = (uint8_t)(w[i / 4] >> (i % 4 * 8));
}

// The largest magnitude's bits of a vector as it lies in memory.  Of a 16-bit type by
// pairs; inf and NaN, which have all exponent bits set, are the exception that has its
// own way.
template <typename T>
__device__ __forceinline__ uint32_t largest_of_raw(const Raw<T>& r) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, r.w[i] & 0x7FFF7FFFu));
  const uint16_t top = m[0] > m[1] ? m[0] : m[1];
  if (top >= (std::is_same<T, f16_t>::value ? 0x7C00 : 0x7F80)) {
    float f[8];
    uint32_t finite = 0;
    unpack_raw(r, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) finite = max(finite, magnitude(f[i]));
    return finite;
  }
  return __float_as_uint(to_f32(__builtin_bit_cast(T, top)));
}
__device__ __forceinline__ uint32_t largest_of_raw(const Raw<float>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(magnitude(r.a[i]), magnitude(r.b[i])));
  return m;
}

// Blocks of 1 x 128, sixteen threads each.  WHOLE: rows (of a part) are whole vectors;
// otherwise a last vector is fetched as the row's last eight elements and moved down, and
// rows under a vector are read element by element.  RUN: a row (of a part) is a multiple of
// four blocks, a wavefront's.
template <typename T, int FORMAT, bool WHOLE, bool RUN>
__global__ __launch_bounds__(kBlock) void k_pack8_rows(Pack8Args a) {
  constexpr int U = 2, kApart = kBlock / 16;
  const int tx = threadIdx.x & 15;
  for (int64_t t0 = (int64_t)blockIdx.x * U * kApart + threadIdx.x / 16; t0 < a.items;
       t0 += (int64_t)gridDim.x * U * kApart) {
    Raw<T> r[U];
    int n[U];
    uint8_t* to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {  // past the end the last block once more
      const int64_t t = RUN ? min(lead<RUN>(t0 + u * kApart), a.items - 4) : min(t0 + u * kApart, a.items - 1);
      const int64_t row = a.per_row.quotient(t);
      uint32_t g = (uint32_t)(t - row * a.per_row.d), q = 0;
      if (a.parts == 2 && g >= a.across) {
        g -= a.across;
        q = 1;
      }
      const int64_t first = (int64_t)g * ECHO_FP8_BLOCK;
      const int off = RUN ? (int)(threadIdx.x & 63) * 8 : tx * 8;
      n[u] = (int)min(a.cols - first, (int64_t)1 << 20) - off;
      to[u] = (uint8_t*)a.codes + row * a.ld_c + q * a.c_part + first;
      const T* const x = (const T*)a.x + row * a.ld_x + q * a.x_part;
      if (WHOLE || a.cols >= 8) r[u] = fetch_at<false>(x + first + (n[u] < 8 ? off + n[u] - 8 : off));
      else r[u] = fetch_short(x, (int)a.cols);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t0 + u * kApart >= a.items) break;
      if (!WHOLE && n[u] < 8 && n[u] > 0) {
        if (a.cols >= 8) MoveDown{8 - n[u]}(r[u]);
        clear_from(r[u], n[u]);
      }
      const uint32_t largest = n[u] > 0 ? largest_of_raw(r[u]) : 0;
      const int e = scale_exponent<FORMAT>(lanes_max(largest));
      const float inverse = power_of_two(254 - e);
      float f[8];
      unpack_raw(r[u], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= inverse;
      if (n[u] > 0) store_codes<true>(to[u] + (RUN ? (int)(threadIdx.x & 63) * 8 : tx * 8), n[u], codes_of<FORMAT>(f));
      if (tx == 0) a.scales[t0 + u * kApart] = power_of_two(e);
    }
  }
}

// bytes b of four words each: out[i] has byte i of all four, in their order
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  w[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  w[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  w[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  w[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// Blocks of 128 x 128, a workgroup each; a thread has eight columns of eight rows in
// registers, so the transposed codes need no second reading and no LDS.
// 3584 x 4096 bf16 with its transpose in 14.6 us (4.0 TB/s): 896 workgroups are one round
// whose loads, block's scale and stores follow each other, and the transposed rows' stores
// are eight bytes at a time, which the caches join.
template <typename T, int FORMAT, bool WHOLE, bool TURN>
__global__ __launch_bounds__(256) void k_pack8_blocks(Pack8Args a) {
  __shared__ uint32_t most[4];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int64_t t = blockIdx.x; t < a.items; t += gridDim.x) {
    const uint32_t b = (uint32_t)t, bj = b % a.across, bq = b / a.across, bi = bq % a.down, q = bq / a.down;
    const int64_t row = (int64_t)bi * ECHO_FP8_BLOCK + ty * 8, col = (int64_t)bj * ECHO_FP8_BLOCK + tx * 8;
    const int64_t n = a.cols - col, high = a.rows - row;
    float f[8][8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
      load_row<T, WHOLE>((const T*)a.x + q * a.x_part + (row + r) * a.ld_x + col, r < high ? n : 0, f[r]);
    uint32_t largest = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i) largest = max(largest, magnitude(f[r][i]));
    largest = lanes_max(largest);
    largest = max(max((uint32_t)__builtin_amdgcn_readlane((int)largest, 0), (uint32_t)__builtin_amdgcn_readlane((int)largest, 16)),
                  max((uint32_t)__builtin_amdgcn_readlane((int)largest, 32), (uint32_t)__builtin_amdgcn_readlane((int)largest, 48)));
    __syncthreads();  // the block before has read its four
    if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = largest;
    __syncthreads();
    const int e = scale_exponent<FORMAT>(max(max(most[0], most[1]), max(most[2], most[3])));
    const float inverse = power_of_two(254 - e);
    u32x2 w[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[r][i] *= inverse;
      w[r] = codes_of<FORMAT>(f[r]);
      if (r < high && n > 0) store_codes<!TURN>((uint8_t*)a.codes + q * a.c_part + (row + r) * a.ld_c + col, n, w[r]);
    }
    if (threadIdx.x == 0) a.scales[q * a.s_part + bi * a.ld_s + bj] = power_of_two(e);
    if constexpr (TURN) {
      const int64_t at = (int64_t)q * a.rows + row;  // of the transposed row
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t top[4] = {w[0][h], w[1][h], w[2][h], w[3][h]}, low[4] = {w[4][h], w[5][h], w[6][h], w[7][h]};
        transpose4(top);
        transpose4(low);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (h * 4 + i < n && high > 0)
            store_codes<false>((uint8_t*)a.codes_t + (col + h * 4 + i) * a.ld_t + at, high, u32x2{top[i], low[i]});
      }
      if (threadIdx.x == 0) a.scales_t[bj * a.ld_st + q * a.down + bi] = power_of_two(e);
    }
  }
}

template <typename T, int FORMAT, bool RUN>
__global__ __launch_bounds__(kBlock) void k_unpack8(Unpack8Args a) {
  unpack8<T, FORMAT, RUN>(a, blockIdx.x, gridDim.x);
}

// ---- host side ---------------------------------------------------------------------

struct Matrix {
  int64_t rows, cols;  // of a part
  int64_t ld_x, ld_c, ld_t, size;
  int64_t across, down;  // blocks of a part
  bool empty;
};

int check_desc(const echo_pack8_desc* d, bool turned, Matrix& m) {
  if (!d) return ECHO_ERR_INVALID_ARGUMENT;
  if (d->dtype != ECHO_BF16 && d->dtype != ECHO_F16 && d->dtype != ECHO_F32) return ECHO_ERR_TYPE;
  if (d->format != ECHO_E4M3 && d->format != ECHO_E5M2) return ECHO_ERR_TYPE;
  if (d->blocks != 0 && d->blocks != 1) return ECHO_ERR_TYPE;
  if (d->rows < 0 || d->cols < 0 || d->rows > (d->blocks ? ECHO_MAX_PITCH : ECHO_MAX_ROWS) || d->cols > ECHO_MAX_PITCH ||
      d->rows * d->cols > ECHO_MAX_PRODUCT || (d->parts != 1 && d->parts != 2))
    return ECHO_ERR_SHAPE;
  m.rows = d->blocks ? d->rows / d->parts : d->rows;
  m.cols = d->blocks ? d->cols : d->cols / d->parts;
  if ((d->blocks ? d->rows : d->cols) % d->parts) return ECHO_ERR_SHAPE;
  if (turned && (!d->blocks || (d->parts == 2 && m.rows % ECHO_FP8_BLOCK))) return ECHO_ERR_SHAPE;
  m.size = d->dtype == ECHO_F32 ? 4 : 2;
  m.ld_x = d->ld_x ? d->ld_x : d->cols;
  if (d->ld_x != 0 && (d->ld_x < d->cols || d->ld_x > ECHO_MAX_PITCH)) return ECHO_ERR_SHAPE;
  int rc = code_pitch(d->ld_c, d->cols, m.ld_c);
  if (rc == ECHO_SUCCESS && turned) rc = code_pitch(d->ld_t, d->rows, m.ld_t);
  m.across = blocks_of(m.cols);
  m.down = d->blocks ? blocks_of(m.rows) : m.rows;
  m.empty = d->rows == 0 || d->cols == 0;
  return rc;
}

template <typename T, int FORMAT>
int pack(const Pack8Args& a, bool blocks, bool whole, hipStream_t s) {
  if (!blocks) {
    const bool run = a.cols % (4 * ECHO_FP8_BLOCK) == 0;
    const dim3 grid(blocks_for_items((uint64_t)a.items * 8));  // 16 threads to a block, two blocks each
    if (run) return launch(k_pack8_rows<T, FORMAT, true, true>, grid, s, a);
    return whole ? launch(k_pack8_rows<T, FORMAT, true, false>, grid, s, a)
                 : launch(k_pack8_rows<T, FORMAT, false, false>, grid, s, a);
  }
  const dim3 grid((uint32_t)(a.items < (int64_t)kMaxBlocks ? a.items : kMaxBlocks));
  if (a.codes_t)
    return whole ? launch(k_pack8_blocks<T, FORMAT, true, true>, grid, dim3(256), s, a)
                 : launch(k_pack8_blocks<T, FORMAT, false, true>, grid, dim3(256), s, a);
  return whole ? launch(k_pack8_blocks<T, FORMAT, true, false>, grid, dim3(256), s, a)
               : launch(k_pack8_blocks<T, FORMAT, false, false>, grid, dim3(256), s, a);
}

template <typename T>
int pack(const Pack8Args& a, int32_t format, bool blocks, bool whole, hipStream_t s) {
  return format == ECHO_E4M3 ? pack<T, ECHO_E4M3>(a, blocks, whole, s) : pack<T, ECHO_E5M2>(a, blocks, whole, s);
}

template <typename T>
int unpack(const Unpack8Args& a, int32_t format, hipStream_t s) {
  const dim3 grid(unpack_blocks(a));
  if (a.runs())
    return format == ECHO_E4M3 ? launch(k_unpack8<T, ECHO_E4M3, true>, grid, s, a)
                               : launch(k_unpack8<T, ECHO_E5M2, true>, grid, s, a);
  return format == ECHO_E4M3 ? launch(k_unpack8<T, ECHO_E4M3, false>, grid, s, a)
                             : launch(k_unpack8<T, ECHO_E5M2, false>, grid, s, a);
}

int unpack(Unpack8Args a, int32_t format, int32_t dtype, hipStream_t s) {
  a.per_row = Divisor::of(a.parts * a.vectors, a.items);
  if (dtype == ECHO_F32) return unpack<float>(a, format, s);
  return dtype == ECHO_BF16 ? unpack<bf16_t>(a, format, s) : unpack<f16_t>(a, format, s);
}

}  // namespace

namespace echo {

int unpack_rows(const void* codes, int64_t ld_c, const float* scales, int32_t format, int64_t m, int64_t k, void* x,
                int64_t ld, int32_t dtype, hipStream_t s) {
  if (m == 0 || ld == 0) return ECHO_SUCCESS;
  return unpack(unpack_args(codes, ld_c, scales, m, k, x, ld), format, dtype, s);
}

}  // namespace echo

extern "C" {

int echo_pack8(const echo_pack8_desc* d, const void* x, void* codes, float* scales, void* codes_t,
               float* scales_t, echo_stream_t stream) {
  Matrix m = {};
  const bool turned = codes_t || scales_t;
  const int rc = check_desc(d, turned, m);
  if (rc) return rc;
  if (m.empty) return ECHO_SUCCESS;
  if (!x || !codes || !scales || (turned && (!codes_t || !scales_t))) return ECHO_ERR_INVALID_ARGUMENT;
  if (!aligned(x, m.size) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(codes_t, 16) || !aligned(scales_t, 4))
    return ECHO_ERR_ALIGNMENT;
  const int64_t side = d->parts * m.across * m.down;
  Aliases al;
  al.in(x, bytes_of(d->rows, d->cols, m.ld_x, m.size));
  al.out(codes, bytes_of(d->rows, d->cols, m.ld_c, 1));
  al.out(scales, side * 4);
  if (turned) {
    al.out(codes_t, bytes_of(d->cols, d->rows, m.ld_t, 1));
    al.out(scales_t, side * 4);
  }
  if (!al.ok()) return ECHO_ERR_ALIAS;
  Pack8Args a = {};
  a.x = x;
  a.codes = codes;
  a.scales = scales;
  a.codes_t = codes_t;
  a.scales_t = scales_t;
  a.rows = m.rows;
  a.cols = m.cols;
  a.ld_x = m.ld_x;
  a.ld_c = m.ld_c;
  a.ld_t = m.ld_t;
  a.x_part = d->blocks ? m.rows * m.ld_x : m.cols;
  a.c_part = d->blocks ? m.rows * m.ld_c : m.cols;
  a.s_part = m.down * m.across;
  a.ld_s = m.across;
  a.ld_st = d->parts * m.down;
  a.items = side;
  a.parts = (uint32_t)d->parts;
  a.across = (uint32_t)m.across;
  a.down = (uint32_t)m.down;
  a.per_row = Divisor::of(a.parts * a.across, a.items);
  const bool whole = m.cols % 8 == 0;
  const hipStream_t s = (hipStream_t)stream;
  if (d->dtype == ECHO_F32) return pack<float>(a, d->format, d->blocks != 0, whole, s);
  return d->dtype == ECHO_BF16 ? pack<bf16_t>(a, d->format, d->blocks != 0, whole, s)
                               : pack<f16_t>(a, d->format, d->blocks != 0, whole, s);
}

int echo_unpack8(const echo_pack8_desc* d, const void* codes, const float* scales, void* x,
                 echo_stream_t stream) {
  Matrix m = {};
  const int rc = check_desc(d, false, m);
  if (rc) return rc;
  if (m.empty) return ECHO_SUCCESS;
  if (!x || !codes || !scales) return ECHO_ERR_INVALID_ARGUMENT;
  if (!aligned(x, m.size) || !aligned(codes, 16) || !aligned(scales, 4)) return ECHO_ERR_ALIGNMENT;
  Aliases al;
  al.out(x, bytes_of(d->rows, d->cols, m.ld_x, m.size));
  al.in(codes, bytes_of(d->rows, d->cols, m.ld_c, 1));
  al.in(scales, d->parts * m.across * m.down * 4);
  if (!al.ok()) return ECHO_ERR_ALIAS;
  Unpack8Args a = {};
  a.codes = codes;
  a.scales = scales;
  a.x = x;
  a.rows = d->rows;
  a.cols = a.fill = m.cols;
  a.ld_x = m.ld_x;
  a.ld_c = m.ld_c;
  a.blocks = d->blocks;
  a.ld_s = d->blocks ? m.across : d->parts * m.across;
  // blocks: a second part's rows follow the first's, its scales the first's
  a.parts = d->blocks ? 1 : (uint32_t)d->parts;
  a.x_part = a.c_part = m.cols;
  a.s_part = m.across;
  a.vectors = (uint32_t)((m.cols + 7) / 8);
  const hipStream_t s = (hipStream_t)stream;
  if (!d->blocks) {
    a.items = d->rows * a.parts * a.vectors;
    return unpack(a, d->format, d->dtype, s);
  }
  for (int q = 0; q < d->parts; ++q) {
    Unpack8Args b = a;
    b.codes = (const uint8_t*)codes + q * m.rows * m.ld_c;
    b.scales = scales + q * m.down * m.across;
    b.x = (char*)x + q * m.rows * m.ld_x * m.size;
    b.rows = m.rows;
    b.items = m.rows * b.vectors;
    const int rc2 = unpack(b, d->format, d->dtype, s);
    if (rc2) return rc2;
  }
  return ECHO_SUCCESS;
}

}  // extern "C"
