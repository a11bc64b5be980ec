// echo_norm.hip -- the norms before and after a block, fused with the block's
// gate and residual scale, and their gradients: kernels and the host side of
// echo_norm and echo_norm_backward (include/echo_layer.h).
//
// Per token, with hat(v) = (v - mean) rstd the normalized row (mean 0 for the
// root mean square norm) and N(v) = hat(v) w + b:
//   forward   u = N_post(y);  h' = h + scale gate u;  z = N_pre(h')
//   backward  d = dz w_pre;   dh = dh' + rstd (d - hat mean(d hat) - mean(d))
//             du = scale gate dh, and dy from du in the same way
//             (the last mean only for the layer norm)
// Both are bound by HBM: the forward call has to read y, h and to write h', z,
// the backward call to read dz, dh', h', y and to write dh, dy, with a few tens
// of operations per element.  So a row is read once and stays in registers, in
// binary32, from its loads to its stores: a thread holds ITEMS vectors of 8
// elements, a row takes W wavefronts, and sums go over the lanes by DPP and over
// the wavefronts through a few words of LDS.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "echo_layer.h"
#include "host_checks.h"
#include "layer_device.h"

using namespace echo;

namespace {

struct NormArgs {
  const void *h, *y, *gate, *w_post, *b_post, *w_pre, *b_pre;
  void *h_out, *z;
  float* stats;
  int64_t tokens, ld_y, ld_h;
  uint32_t hidden, rows_per_gate;  // rows_per_gate 0: no gate
  int32_t post, pre;
  float scale, eps;
};

// WAVES = 1: a row to a wavefront, four rows side by side in a workgroup.
// WAVES > 1: a row to the workgroup, which has up to so many wavefronts (fewer
// leave the compiler more registers).
constexpr int kSideBySide = 4;
constexpr int kMostWaves = 16;
constexpr int threads_of(int WAVES) { return 64 * (WAVES > 1 ? WAVES : kSideBySide); }

// Sums over the wavefronts of a row, double-buffered by the row's parity: a slot
// is written again two rows later, and the barrier of the row between keeps a
// late reader apart from it.
template <bool MANY>
struct RowSums {
  float* lds;  // [2][4][kMostWaves]
  uint32_t wave, waves, parity;
  __device__ __forceinline__ float add(const float* p) const {
    float s = p[0];
    for (uint32_t i = 1; i < waves; ++i) s += p[i];
    return s;
  }
  __device__ __forceinline__ float sum(float v, int slot) {
    v = wave_sum(v);
    if constexpr (!MANY) return v;
    float* p = lds + (parity * 4 + slot) * kMostWaves;
    if ((threadIdx.x & 63) == 0) p[wave] = v;
    __syncthreads();
    return add(p);
  }
  // two sums behind one barrier
  __device__ __forceinline__ void sum2(float& a, float& b, int slot) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (MANY) {
      float* p = lds + (parity * 4 + slot) * kMostWaves;
      if ((threadIdx.x & 63) == 0) {
        p[wave] = a;
        p[kMostWaves + wave] = b;
      }
      __syncthreads();
      a = add(p);
      b = add(p + kMostWaves);
    }
  }
};

// Mean and reciprocal deviation of the row in v.  The layer norm's variance is
// the mean square about the mean, from registers, so a mean far from zero
// costs no digits.
template <RowEnd END, int ITEMS, typename Sums>
__device__ __forceinline__ void moments(const float (&v)[ITEMS][8], const Place<END> (&at)[ITEMS], int kind,
                                        float eps, float inv_h, Sums& sums, int slot, float& mean,
                                        float& rstd) {
  mean = 0.f;
  if (kind == ECHO_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += at[i].only(e, v[i][e]);
    mean = sums.sum(s, slot) * inv_h;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = at[i].only(e, v[i][e] - mean);
      q = fmaf(c, c, q);
    }
  rstd = 1.0f / sqrtf(sums.sum(q, slot + 1) * inv_h + eps);
}

// The thread's columns of a vector along the row (a weight, a bias, a gate row),
// fetched before they are needed; absent ones are `none`.
template <typename T, int ITEMS>
struct RowVector {
  Raw<T> raw[ITEMS];
  const T* row;
  template <typename P>
  __device__ __forceinline__ void fetch(const void* p, const P (&at)[ITEMS], int H) {
    row = (const T*)p;
    if (!row) return;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) raw[i] = at[i].template fetch<false>(row, H);
  }
  // keeps the words packed across a loop: unpacked ahead of it they would take
  // twice the registers
  __device__ __forceinline__ void keep_packed() {
    if (!row) return;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) keep(raw[i]);
  }
};

// A thread's vectors of a row, `across` threads to a row.
template <RowEnd END, int ITEMS>
struct Places;
template <RowEnd END>
struct Places<END, 1> {
  Place<END> at[1];
  int col[1];
  __device__ __forceinline__ Places(int thread, int, int H) : at{{thread * 8, H}}, col{thread * 8} {}
};
template <RowEnd END>
struct Places<END, 2> {
  Place<END> at[2];
  int col[2];
  __device__ __forceinline__ Places(int thread, int across, int H)
      : at{{thread * 8, H}, {(thread + across) * 8, H}}, col{thread * 8, (thread + across) * 8} {}
};

// v <- (v - mean) rstd w + b on the thread's columns
template <RowEnd END, typename T, int ITEMS>
__device__ __forceinline__ void apply_norm(float (&v)[ITEMS][8], const Place<END> (&at)[ITEMS], float mean,
                                           float rstd, const RowVector<T, ITEMS>& w,
                                           const RowVector<T, ITEMS>& b) {
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = (v[i][e] - mean) * rstd;
    if (w.row) {
      at[i].unpack(w.raw[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] *= f[e];
    }
    if (b.row) {
      at[i].unpack(b.raw[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] += f[e];
    }
  }
}

template <typename T, typename S, int WAVES, int ITEMS, RowEnd END>
__global__ __launch_bounds__(threads_of(WAVES)) void k_norm(NormArgs a) {
  constexpr bool MANY = WAVES > 1;
  constexpr int kRows = MANY ? 1 : kSideBySide;  // rows a workgroup works on at a time
  __shared__ float slots[MANY ? 2 * 4 * kMostWaves : 1];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int across = MANY ? (int)blockDim.x : 64;  // threads of a row
  RowSums<MANY> sums{slots, wave, blockDim.x >> 6, 0};
  const int H = (int)a.hidden;
  const float inv_h = 1.0f / (float)H;
  const Places<END, ITEMS> places(MANY ? (int)threadIdx.x : (int)(threadIdx.x & 63), across, H);
  const auto& at = places.at;
  const auto& col = places.col;
  for (int64_t row = (int64_t)blockIdx.x * kRows + (MANY ? 0 : wave); row < a.tokens;
       row += (int64_t)gridDim.x * kRows, sums.parity ^= 1) {
    float v[ITEMS][8], h[ITEMS][8];
    const S* hp = (const S*)a.h + row * a.ld_h;
    const T* yp = (const T*)a.y + row * a.ld_y;
    Raw<S> hr[ITEMS];
    Raw<T> yr[ITEMS];
    RowVector<T, ITEMS> gate, w_post, b_post, w_pre, b_pre;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      hr[i] = at[i].template fetch<true>(hp, H);
      if (a.y) yr[i] = at[i].template fetch<true>(yp, H);
    }
    w_post.fetch(a.w_post, at, H);
    b_post.fetch(a.b_post, at, H);
    gate.fetch(a.rows_per_gate ? (const T*)a.gate + (int64_t)((uint32_t)row / a.rows_per_gate) * H : nullptr,
                    at, H);
    w_pre.fetch(a.w_pre, at, H);
    b_pre.fetch(a.b_pre, at, H);
    float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) at[i].unpack(hr[i], h[i]);
    if (a.y) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) at[i].unpack(yr[i], v[i]);
      if (a.post != ECHO_NORM_NONE) {
        moments(v, at, a.post, a.eps, inv_h, sums, 0, mean1, rstd1);
        apply_norm<END, T, ITEMS>(v, at, mean1, rstd1, w_post, b_post);
      }
      if (gate.row) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          float f[8];
          at[i].unpack(gate.raw[i], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] *= f[e];
        }
      }
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = fmaf(a.scale, v[i][e], h[i][e]);
      if (a.h_out) {
        S* op = (S*)a.h_out + row * a.ld_h;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
          at[i].template store<true>(op + col[i], h[i]);
      }
    }
    if (a.pre != ECHO_NORM_NONE) {
      moments(h, at, a.pre, a.eps, inv_h, sums, 2, mean2, rstd2);
      apply_norm<END, T, ITEMS>(h, at, mean2, rstd2, w_pre, b_pre);
      T* zp = (T*)a.z + row * H;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        at[i].template store<true>(zp + col[i], h[i]);
    }
    if (a.stats && (MANY ? threadIdx.x : threadIdx.x & 63) == 0) {
      a.stats[row] = mean1;
      a.stats[a.tokens + row] = rstd1;
      a.stats[2 * a.tokens + row] = mean2;
      a.stats[3 * a.tokens + row] = rstd2;
    }
  }
}

// ---- backward --------------------------------------------------------------------

// How a gate row's gradient is summed.  R = tokens per gate row.
enum GateSum {
  kGateNone = 0,    // no gate gradient
  kGateRow = 1,     // R = 1: written with the row
  kGateWhole = 2,   // a workgroup's rows are whole groups: written by it
  kGatePart = 3     // a group takes several workgroups: partial sums
};

// Partial sums of a workgroup over its rows, [kParts][blocks][hidden] in the
// workspace.
enum Part { kDwPre = 0, kDbPre = 1, kDwPost = 2, kDbPost = 3, kDgate = 4, kParts = 5 };

struct NormBackArgs {
  const void *dz, *dh_out, *h_out, *y, *gate, *w_post, *b_post, *w_pre;
  const float* stats;
  void *dh, *dy, *dgate;
  float* part;
  int64_t tokens, ld_y, ld_h;
  int64_t chunk;  // rows of a workgroup
  uint32_t hidden, rows_per_gate, blocks_per_gate;
  int32_t post, pre, gate_sum;
  uint32_t want;  // bit p: partial sums of Part p are wanted
  float scale;
};

// One element of each 128 bytes of a row, a line to a thread: a load for the L2,
// whose value nobody uses.
template <typename E>
__device__ __forceinline__ float touch(const E* row, int H) {
  const int e = (int)threadIdx.x * (128 / (int)sizeof(E));
  return e < H ? to_f32(row[e]) : 0.f;
}

template <int ITEMS>
__device__ __forceinline__ void zero(float (&v)[ITEMS][8]) {
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
}

// The accumulators of a workgroup, its rows' wavefronts added in order, to
// out[hidden] (binary32 partial sums or, for a whole gate row, its gradient).
template <typename O, bool MANY, int ITEMS>
__device__ __forceinline__ void flush(float (&acc)[ITEMS][8], const int (&col)[ITEMS], O* out, int H,
                                      float* comb) {
  if constexpr (MANY) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (col[i] < H) store_n<false>(out + col[i], H - col[i], acc[i]);
  } else {
    __syncthreads();
    const uint32_t w = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
      if (col[i] < H) {
#pragma unroll
        for (int e = 0; e < 8; ++e) comb[w * (512 * ITEMS) + col[i] + e] = acc[i][e];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < H; c += 64 * kSideBySide) {
      float s = comb[c];
#pragma unroll
      for (int k = 1; k < kSideBySide; ++k) s += comb[k * (512 * ITEMS) + c];
      out[c] = from_f32<O>(s);
    }
  }
}

// FULL: with a post norm or a gate; else dy = scale dh and only the pre
// norm's parameters have gradients.  BIAS: with a bias's gradient.  Without them
// there are fewer accumulators, so more rows in flight.  A workgroup walks
// `chunk` consecutive rows and keeps the sums over them, so the row data is read
// once for all outputs.  The sums stand in registers; but more than eight
// wavefronts have 128 registers a lane, so dw1's, dg's and, where it fits, db1's
// stand in LDS there (4072 x 4100 f16 with all five sums, the same inputs each
// time: 143 us against 242 with all in registers, which spill, and 175 with db2's
// in LDS as well; 4072 x 8200: 600 against 673.  Up to eight wavefronts gain
// nothing by it.)  Sixteen wavefronts with two vectors a lane spill all the same,
// 103 registers and more: rows past 8192 take 4 times their floor and more.
template <typename T, typename S, int WAVES, int ITEMS, bool FULL, bool BIAS, RowEnd END>
__global__ __launch_bounds__(threads_of(WAVES), FULL && WAVES <= 8 && ITEMS == 1 ? 3 : 1) void k_norm_backward(
    NormBackArgs a) {
  constexpr bool MANY = WAVES > 1;
  constexpr bool IN_LDS = FULL && WAVES == kMostWaves;
  constexpr int kFar = BIAS && ITEMS == 1 ? 3 : 2;
  __shared__ f32x4 far[IN_LDS ? kFar * ITEMS * 2 : 1][IN_LDS ? threads_of(WAVES) : 1];
  constexpr int kRows = MANY ? 1 : kSideBySide;
  __shared__ float slots[MANY ? 2 * 4 * kMostWaves : 1];
  __shared__ float comb[MANY ? 1 : kSideBySide * 512 * ITEMS];
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int across = MANY ? (int)blockDim.x : 64;
  RowSums<MANY> sums{slots, wave, blockDim.x >> 6, 0};
  const int H = (int)a.hidden;
  const float inv_h = 1.0f / (float)H;
  const Places<END, ITEMS> places(MANY ? (int)threadIdx.x : (int)(threadIdx.x & 63), across, H);
  const auto& at = places.at;
  const auto& col = places.col;
  // the thread's columns of the weights stay in registers for all its rows
  RowVector<T, ITEMS> w_pre, w_post, b_post, gate;
  w_pre.fetch(a.w_pre, at, H);
  w_post.fetch(FULL ? a.w_post : nullptr, at, H);
  b_post.fetch(FULL ? a.b_post : nullptr, at, H);
  gate.row = nullptr;
  int64_t r0, r1;
  if (a.gate_sum == kGatePart) {
    const int64_t g = blockIdx.x / a.blocks_per_gate, s = blockIdx.x % a.blocks_per_gate;
    r0 = g * a.rows_per_gate + s * a.chunk;
    r1 = min(r0 + a.chunk, (g + 1) * (int64_t)a.rows_per_gate);
  } else {
    r0 = (int64_t)blockIdx.x * a.chunk;
    r1 = min(r0 + a.chunk, a.tokens);
  }
  float dw2[ITEMS][8], db2[BIAS ? ITEMS : 1][8], dw1[FULL ? ITEMS : 1][8], db1[FULL && BIAS ? ITEMS : 1][8],
      dg[FULL ? ITEMS : 1][8];
  zero(dw2);
  zero(db2);
  zero(dw1);
  zero(db1);
  zero(dg);
  // dw1, dg and db1 stand in registers or in the thread's own place in LDS
  enum { kFarW, kFarGate, kFarB };
  auto far_read = [&](int k, int i, float (&v)[8]) {
    if constexpr (IN_LDS) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = far[(k * ITEMS + i) * 2 + e / 4][threadIdx.x][e % 4];
    }
  };
  auto far_write = [&](int k, int i, const float (&v)[8]) {
    if constexpr (IN_LDS) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        far[(k * ITEMS + i) * 2 + q][threadIdx.x] = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    }
  };
#pragma unroll
  for (int k = 0; k < kFar; ++k)
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) far_write(k, i, dw2[i]);  // zeros
  int64_t s1;
  for (int64_t s0 = r0; s0 < r1; s0 = s1) {
    s1 = FULL && a.gate_sum == kGateWhole ? min(s0 + (int64_t)a.rows_per_gate, r1) : r1;
    for (int64_t row = s0 + (MANY ? 0 : wave); row < s1; row += kRows, sums.parity ^= 1) {
      float d[ITEMS][8];   // dh' + N_pre'(dz), then dh
      float hat[ITEMS][8], g[ITEMS][8];
      const T* dzp = (const T*)a.dz + row * H;
      const S* dhp = (const S*)a.dh_out + row * H;
      const S* hp = (const S*)a.h_out + row * a.ld_h;
      const T* yp = (const T*)a.y + row * a.ld_y;
      w_pre.keep_packed();
      w_post.keep_packed();
      b_post.keep_packed();
      Raw<S> dr[ITEMS], hr[ITEMS];
      Raw<T> zr[ITEMS], yr[ITEMS];
      float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f;
      if (a.pre != ECHO_NORM_NONE) {
        mean2 = a.stats[2 * a.tokens + row];
        rstd2 = a.stats[3 * a.tokens + row];
      }
      if (FULL && a.post != ECHO_NORM_NONE) {
        mean1 = a.stats[row];
        rstd1 = a.stats[a.tokens + row];
      }
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        if (a.pre != ECHO_NORM_NONE) {
          hr[i] = at[i].template fetch<true>(hp, H);
          zr[i] = at[i].template fetch<true>(dzp, H);
        }
        if (a.dh_out) dr[i] = at[i].template fetch<true>(dhp, H);
        if (FULL && a.y) yr[i] = at[i].template fetch<true>(yp, H);
      }
      if (FULL && a.rows_per_gate)
        gate.fetch((const T*)a.gate + (int64_t)((uint32_t)row / a.rows_per_gate) * H, at, H);
      // the next row into the L2 while this one waits at its barriers
      float ahead[4] = {0.f, 0.f, 0.f, 0.f};
      if (MANY && row + 1 < s1) {
        if (a.pre != ECHO_NORM_NONE) {
          ahead[0] = touch(hp + a.ld_h, H);
          ahead[1] = touch(dzp + H, H);
        }
        if (a.dh_out) ahead[2] = touch(dhp + H, H);
        if (FULL && a.y) ahead[3] = touch(yp + a.ld_y, H);
      }
      zero(d);
      if (a.pre != ECHO_NORM_NONE) {
        float sh = 0.f, sg = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          float w[8];
          at[i].unpack(hr[i], hat[i]);
          at[i].unpack(zr[i], g[i]);
          if (a.w_pre) at[i].unpack(w_pre.raw[i], w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            hat[i][e] = at[i].only(e, (hat[i][e] - mean2) * rstd2);
            dw2[i][e] = fmaf(g[i][e], hat[i][e], dw2[i][e]);
            if constexpr (BIAS) db2[i][e] += g[i][e];
            if (a.w_pre) g[i][e] *= w[e];
            sh = fmaf(g[i][e], hat[i][e], sh);
            sg += g[i][e];
          }
        }
        if (a.pre == ECHO_NORM_LAYER) {
          sums.sum2(sh, sg, 0);
          sg *= inv_h;
        } else {
          sh = sums.sum(sh, 0);
          sg = 0.f;
        }
        sh *= inv_h;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) d[i][e] = at[i].only(e, rstd2 * ((g[i][e] - sg) - hat[i][e] * sh));
      }
      if (a.dh_out) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          float f[8];
          at[i].unpack(dr[i], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) d[i][e] += f[e];
        }
      }
      S* op = (S*)a.dh + row * H;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
        at[i].template store<true>(op + col[i], d[i]);
      // du = scale gate dh; the gate's and the post norm's gradients from it
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) d[i][e] *= a.scale;
      T* dyp = (T*)a.dy + row * H;
      if constexpr (FULL) {
        float y[ITEMS][8];
        float sh = 0.f, sg = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          float w[8], b[8];
          if (a.y) at[i].unpack(yr[i], y[i]);
          if (a.w_post) at[i].unpack(w_post.raw[i], w);
          if (a.post != ECHO_NORM_NONE) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[i][e] = at[i].only(e, (y[i][e] - mean1) * rstd1);
          }
          if (a.rows_per_gate) {
            if (a.gate_sum != kGateNone) {
              float u[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) u[e] = a.w_post ? y[i][e] * w[e] : y[i][e];
              if (a.b_post) {
                at[i].unpack(b_post.raw[i], b);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] += b[e];
              }
              if (a.gate_sum == kGateRow) {
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] *= d[i][e];
                at[i].template store<true>((T*)a.dgate + row * H + col[i], u);
              } else {
                far_read(kFarGate, i, dg[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) dg[i][e] = fmaf(u[e], d[i][e], dg[i][e]);
                far_write(kFarGate, i, dg[i]);
              }
            }
            at[i].unpack(gate.raw[i], b);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[i][e] *= b[e];
          }
          if (a.post != ECHO_NORM_NONE) {
            far_read(kFarW, i, dw1[i]);
            if constexpr (kFar == 3) far_read(kFarB, i, db1[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              dw1[i][e] = fmaf(d[i][e], y[i][e], dw1[i][e]);
              if constexpr (BIAS) db1[i][e] += d[i][e];
            }
            far_write(kFarW, i, dw1[i]);
            if constexpr (kFar == 3) far_write(kFarB, i, db1[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if (a.w_post) d[i][e] *= w[e];
              sh = fmaf(d[i][e], y[i][e], sh);
              sg += d[i][e];
            }
          }
        }
        if (a.post != ECHO_NORM_NONE) {
          if (a.post == ECHO_NORM_LAYER) {
            sums.sum2(sh, sg, 2);
            sg *= inv_h;
          } else {
            sh = sums.sum(sh, 2);
            sg = 0.f;
          }
          sh *= inv_h;
#pragma unroll
          for (int i = 0; i < ITEMS; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) d[i][e] = rstd1 * ((d[i][e] - sg) - y[i][e] * sh);
        }
      }
      if constexpr (MANY) asm volatile("" ::"v"(ahead[0]), "v"(ahead[1]), "v"(ahead[2]), "v"(ahead[3]));
      if (a.dy)
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
          at[i].template store<true>(dyp + col[i], d[i]);
    }
    if constexpr (FULL) {
      if (a.gate_sum == kGateWhole) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) far_read(kFarGate, i, dg[i]);
        flush<T, MANY, ITEMS>(dg, col, (T*)a.dgate + s0 / a.rows_per_gate * H, H, comb);
        zero(dg);
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) far_write(kFarGate, i, dg[i]);
      }
    }
  }
  const int64_t plane = (int64_t)gridDim.x * H;
  float* p = a.part + (int64_t)blockIdx.x * H;
  if (a.want >> kDwPre & 1) flush<float, MANY, ITEMS>(dw2, col, p + kDwPre * plane, H, comb);
  if constexpr (BIAS)
    if (a.want >> kDbPre & 1) flush<float, MANY, ITEMS>(db2, col, p + kDbPre * plane, H, comb);
  if constexpr (FULL) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      far_read(kFarW, i, dw1[i]);
      far_read(kFarGate, i, dg[i]);
      if constexpr (kFar == 3) far_read(kFarB, i, db1[i]);
    }
    if (a.want >> kDwPost & 1) flush<float, MANY, ITEMS>(dw1, col, p + kDwPost * plane, H, comb);
    if constexpr (BIAS)
      if (a.want >> kDbPost & 1) flush<float, MANY, ITEMS>(db1, col, p + kDbPost * plane, H, comb);
    if (a.want >> kDgate & 1) flush<float, MANY, ITEMS>(dg, col, p + kDgate * plane, H, comb);
  }
}

// out[r][c] = sum of part[b][c] over the `per_row` blocks of row r, in a fixed
// order: 32 columns to a workgroup, 32 runs of blocks side by side.
struct PartSumArgs {
  const float* part[kParts];
  void* out[kParts];
  uint32_t rows[kParts], per_row[kParts];
  uint32_t hidden;
};

template <typename T>
__global__ __launch_bounds__(1024) void k_norm_part_sum(PartSumArgs a) {
  __shared__ float lds[32][33];
  const uint32_t c = threadIdx.x & 31, k = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  const uint32_t p = blockIdx.z;
  for (uint32_t r = blockIdx.y; r < a.rows[p]; r += gridDim.y) {
    const uint32_t nb = a.per_row[p];
    const float* src = a.part[p] + (int64_t)r * nb * a.hidden;
    float s = 0.f;
    if (col < a.hidden) {
      uint32_t b = k;
      for (; b + 7 * 32 < nb; b += 8 * 32) {  // eight loads on their way at once
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = src[(int64_t)(b + e * 32) * a.hidden + col];
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[e];
      }
      for (; b < nb; b += 32) s += src[(int64_t)b * a.hidden + col];
    }
    __syncthreads();
    lds[k][c] = s;
    __syncthreads();
    if (k == 0 && col < a.hidden) {
#pragma unroll
      for (int i = 1; i < 32; ++i) s += lds[i][c];
      ((T*)a.out[p])[(int64_t)r * a.hidden + col] = from_f32<T>(s);
    }
  }
}

// ---- host side ---------------------------------------------------------------------

bool type_ok(int32_t t) { return t == ECHO_BF16 || t == ECHO_F16 || t == ECHO_F32; }
bool kind_ok(int32_t k) { return k == ECHO_NORM_NONE || k == ECHO_NORM_RMS || k == ECHO_NORM_LAYER; }
int64_t size_of(int32_t t) { return t == ECHO_F32 ? 4 : 2; }

struct Geometry {
  int64_t T, H, ld_y, ld_h, e, s;  // e, s: bytes of an element, of a stream element
  int64_t y_bytes, h_bytes, dense, dense_s;
};

int64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t size) {
  return rows == 0 ? 0 : ((rows - 1) * ld + cols) * size;
}

int check_shape(const echo_norm_desc* d) {
  if (!d) return ECHO_ERR_INVALID_ARGUMENT;
  if (d->tokens < 0 || d->tokens > ECHO_MAX_ROWS || d->hidden < 1 || d->hidden > ECHO_MAX_HIDDEN)
    return ECHO_ERR_SHAPE;
  if (d->gate_rows < 0 || d->gate_rows > ECHO_MAX_ROWS ||
      (d->gate_rows > 0 && d->tokens % d->gate_rows != 0))
    return ECHO_ERR_SHAPE;
  if ((d->ld_y != 0 && (d->ld_y < d->hidden || d->ld_y > ECHO_MAX_PITCH)) ||
      (d->ld_h != 0 && (d->ld_h < d->hidden || d->ld_h > ECHO_MAX_PITCH)))
    return ECHO_ERR_SHAPE;
  return ECHO_SUCCESS;
}

int check_desc(const echo_norm_desc* d, Geometry& g) {
  const int rc = check_shape(d);
  if (rc) return rc;
  if (!type_ok(d->dtype) || (d->stream_dtype != d->dtype && d->stream_dtype != ECHO_F32))
    return ECHO_ERR_TYPE;
  if (!kind_ok(d->post) || !kind_ok(d->pre)) return ECHO_ERR_TYPE;
  if (!(d->eps >= 0.f)) return ECHO_ERR_SHAPE;
  g.T = d->tokens;
  g.H = d->hidden;
  g.ld_y = d->ld_y ? d->ld_y : g.H;
  g.ld_h = d->ld_h ? d->ld_h : g.H;
  g.e = size_of(d->dtype);
  g.s = size_of(d->stream_dtype);
  g.y_bytes = span(g.T, g.H, g.ld_y, g.e);
  g.h_bytes = span(g.T, g.H, g.ld_h, g.s);
  g.dense = g.T * g.H * g.e;
  g.dense_s = g.T * g.H * g.s;
  return ECHO_SUCCESS;
}

// Wavefronts of a row and vectors of a thread.  Short rows take one wavefront and
// need no barrier; longer ones as many as hold them.  The forward pass holds two
// vectors a thread past 2048 elements (8192 x 4096: 45.6 us against 51.7 with one,
// which has twice the wavefronts to wait for at a barrier); the backward pass,
// whose accumulators fill the registers, one (without a post norm and a gate two to
// 1024, so that such rows need no barrier; and two past 8192, where a workgroup
// has no more wavefronts).
struct RowShape {
  int waves, items, threads;  // waves: the kernel's WAVES
  int64_t rows;               // of a workgroup at a time
};
enum Pass { kForward, kBackPlain, kBackFull };

RowShape shape_of(int64_t hidden, Pass pass) {
  if (hidden <= 512) return {1, 1, 64 * kSideBySide, kSideBySide};
  if (hidden <= 1024 && pass != kBackFull) return {1, 2, 64 * kSideBySide, kSideBySide};
  const int items = hidden <= (pass == kForward ? 2048 : 512 * kMostWaves) ? 1 : 2;
  const int waves = (int)((hidden + 512 * items - 1) / (512 * items));
  return {waves <= 8 ? 8 : kMostWaves, items, waves * 64, 1};
}

// Rows of a workgroup of the backward pass, and how many workgroups that is.
struct Walk {
  int64_t chunk;
  uint32_t blocks, blocks_per_gate;
  int32_t gate_sum;
};

Walk walk_of(int64_t T, int64_t H, int64_t gate_rows, bool want_gate, Pass pass) {
  const RowShape shape = shape_of(H, pass);
  const int64_t rows = shape.rows;
  // as many workgroups as are in residence, by the kernels' registers
  const int resident = pass == kBackFull ? 12 : 16;  // wavefronts of a compute unit
  const int64_t most = 256 * (resident * 64 >= shape.threads ? resident * 64 / shape.threads : 1);
  Walk w = {};
  int64_t chunk = (T + most - 1) / most;
  chunk = (chunk + rows - 1) / rows * rows;
  if (chunk < rows) chunk = rows;
  w.chunk = chunk;
  w.blocks_per_gate = 1;
  w.gate_sum = kGateNone;
  if (want_gate && gate_rows > 0 && T > 0) {
    const int64_t R = T / gate_rows;
    if (R == 1) {
      w.gate_sum = kGateRow;
    } else if (R <= chunk) {
      w.gate_sum = kGateWhole;
      w.chunk = chunk / R * R;
    } else {
      w.gate_sum = kGatePart;
      w.blocks_per_gate = (uint32_t)((R + chunk - 1) / chunk);
      w.blocks = (uint32_t)gate_rows * w.blocks_per_gate;
      return w;
    }
  }
  w.blocks = (uint32_t)((T + w.chunk - 1) / w.chunk);
  return w;
}

template <typename T, typename S, RowEnd END>
int launch_norm(const NormArgs& a, hipStream_t s) {
  const RowShape r = shape_of(a.hidden, kForward);
  const int64_t want = (a.tokens + r.rows - 1) / r.rows;
  const int64_t cap = 0xFFFFFFFFu / (uint32_t)r.threads;
  const dim3 grid((uint32_t)(want < cap ? want : cap)), block(r.threads);
  if constexpr (END == kShort) return launch(k_norm<T, S, 1, 1, END>, grid, block, s, a);
  else switch (r.waves * 4 + r.items) {
    case 4 + 1: return launch(k_norm<T, S, 1, 1, END>, grid, block, s, a);
    case 4 + 2: return launch(k_norm<T, S, 1, 2, END>, grid, block, s, a);
    case 32 + 1: return launch(k_norm<T, S, 8, 1, END>, grid, block, s, a);
    case 32 + 2: return launch(k_norm<T, S, 8, 2, END>, grid, block, s, a);
    default: return launch(k_norm<T, S, 16, 2, END>, grid, block, s, a);
  }
}

template <typename T, typename S>
int launch_norm(const NormArgs& a, hipStream_t s) {
  if (a.hidden < 8) return launch_norm<T, S, kShort>(a, s);
  return a.hidden % 8 ? launch_norm<T, S, kTail>(a, s) : launch_norm<T, S, kWhole>(a, s);
}

template <typename T, typename S, bool FULL, bool BIAS, RowEnd END>
int launch_norm_backward(const NormBackArgs& a, uint32_t blocks, hipStream_t s) {
  const RowShape r = shape_of(a.hidden, FULL ? kBackFull : kBackPlain);
  const dim3 grid(blocks), block(r.threads);
  if constexpr (END == kShort) return launch(k_norm_backward<T, S, 1, 1, FULL, BIAS, END>, grid, block, s, a);
  else switch (r.waves * 4 + r.items) {
    case 4 + 1: return launch(k_norm_backward<T, S, 1, 1, FULL, BIAS, END>, grid, block, s, a);
    case 4 + 2:
      if constexpr (!FULL) return launch(k_norm_backward<T, S, 1, 2, FULL, BIAS, END>, grid, block, s, a);
      return ECHO_ERR_SHAPE;
    case 32 + 1: return launch(k_norm_backward<T, S, 8, 1, FULL, BIAS, END>, grid, block, s, a);
    case 64 + 1: return launch(k_norm_backward<T, S, 16, 1, FULL, BIAS, END>, grid, block, s, a);
    default: return launch(k_norm_backward<T, S, 16, 2, FULL, BIAS, END>, grid, block, s, a);
  }
}

template <typename T, typename S, RowEnd END>
int launch_norm_backward(const NormBackArgs& a, uint32_t blocks, bool full, hipStream_t s) {
  const bool bias = a.want >> kDbPre & 1 || a.want >> kDbPost & 1;
  if (full)
    return bias ? launch_norm_backward<T, S, true, true, END>(a, blocks, s)
                : launch_norm_backward<T, S, true, false, END>(a, blocks, s);
  return bias ? launch_norm_backward<T, S, false, true, END>(a, blocks, s)
              : launch_norm_backward<T, S, false, false, END>(a, blocks, s);
}

template <typename T, typename S>
int launch_norm_backward(const NormBackArgs& a, uint32_t blocks, bool full, hipStream_t s) {
  if (a.hidden < 8) return launch_norm_backward<T, S, kShort>(a, blocks, full, s);
  return a.hidden % 8 ? launch_norm_backward<T, S, kTail>(a, blocks, full, s)
                      : launch_norm_backward<T, S, kWhole>(a, blocks, full, s);
}

int run_norm(const NormArgs& a, int32_t t, int32_t st, hipStream_t s) {
  if (t == ECHO_F32) return launch_norm<float, float>(a, s);
  if (t == ECHO_BF16)
    return st == t ? launch_norm<bf16_t, bf16_t>(a, s) : launch_norm<bf16_t, float>(a, s);
  return st == t ? launch_norm<f16_t, f16_t>(a, s) : launch_norm<f16_t, float>(a, s);
}

int run_norm_backward(const NormBackArgs& a, uint32_t blocks, bool full, int32_t t, int32_t st,
                      hipStream_t s) {
  if (t == ECHO_F32) return launch_norm_backward<float, float>(a, blocks, full, s);
  if (t == ECHO_BF16)
    return st == t ? launch_norm_backward<bf16_t, bf16_t>(a, blocks, full, s)
                   : launch_norm_backward<bf16_t, float>(a, blocks, full, s);
  return st == t ? launch_norm_backward<f16_t, f16_t>(a, blocks, full, s)
                 : launch_norm_backward<f16_t, float>(a, blocks, full, s);
}

int run_part_sum(const PartSumArgs& a, uint32_t parts, uint32_t rows, int32_t t, hipStream_t s) {
  const dim3 grid((a.hidden + 31) / 32, rows < 1024 ? rows : 1024, parts), block(1024);
  if (t == ECHO_F32) return launch(k_norm_part_sum<float>, grid, block, s, a);
  if (t == ECHO_BF16) return launch(k_norm_part_sum<bf16_t>, grid, block, s, a);
  return launch(k_norm_part_sum<f16_t>, grid, block, s, a);
}

}  // namespace

extern "C" {

int echo_norm(const echo_norm_desc* d, const void* h, const void* y, const void* gate,
              const void* w_post, const void* b_post, const void* w_pre, const void* b_pre,
              void* h_out, void* z, float* stats, echo_stream_t stream) {
  Geometry g;
  const int rc = check_desc(d, g);
  if (rc) return rc;
  if (g.T == 0) return ECHO_SUCCESS;
  const bool post = d->post != ECHO_NORM_NONE, pre = d->pre != ECHO_NORM_NONE;
  if (!h || (z != nullptr) != pre || (gate != nullptr) != (d->gate_rows > 0))
    return ECHO_ERR_INVALID_ARGUMENT;
  if (!y && (post || gate || h_out)) return ECHO_ERR_INVALID_ARGUMENT;
  if ((!post && (w_post || b_post)) || (!pre && (w_pre || b_pre))) return ECHO_ERR_INVALID_ARGUMENT;
  if (!z && !h_out) return ECHO_ERR_INVALID_ARGUMENT;  // nothing to compute
  for (const void* p : {y, gate, w_post, b_post, w_pre, b_pre, (const void*)z})
    if (!aligned(p, g.e)) return ECHO_ERR_ALIGNMENT;
  if (!aligned(h, g.s) || !aligned(h_out, g.s) || !aligned(stats, 4)) return ECHO_ERR_ALIGNMENT;
  Aliases al;
  al.out(h_out, g.h_bytes);
  al.out(z, g.dense);
  al.out(stats, 16 * g.T);
  al.in(h, g.h_bytes);
  al.in(y, g.y_bytes);
  al.in(gate, d->gate_rows * g.H * g.e);
  for (const void* p : {w_post, b_post, w_pre, b_pre}) al.in(p, g.H * g.e);
  al.allow_identical(h_out, h);
  if (!al.ok()) return ECHO_ERR_ALIAS;
  NormArgs a = {};
  a.h = h;
  a.y = y;
  a.gate = gate;
  a.w_post = w_post;
  a.b_post = b_post;
  a.w_pre = w_pre;
  a.b_pre = b_pre;
  a.h_out = h_out;
  a.z = z;
  a.stats = stats;
  a.tokens = g.T;
  a.ld_y = g.ld_y;
  a.ld_h = g.ld_h;
  a.hidden = (uint32_t)g.H;
  a.rows_per_gate = d->gate_rows ? (uint32_t)(g.T / d->gate_rows) : 0;
  a.post = d->post;
  a.pre = d->pre;
  a.scale = d->scale;
  a.eps = d->eps;
  return run_norm(a, d->dtype, d->stream_dtype, (hipStream_t)stream);
}

int64_t echo_norm_backward_workspace(const echo_norm_desc* d) {
  const int rc = check_shape(d);
  if (rc) return rc;
  if (d->tokens == 0) return 0;
  // whatever norms, and whether the gate's gradient is wanted or not
  uint32_t most = 0;
  for (const Pass pass : {kBackPlain, kBackFull})
    for (const bool want_gate : {false, true}) {
      const uint32_t blocks = walk_of(d->tokens, d->hidden, d->gate_rows, want_gate, pass).blocks;
      if (blocks > most) most = blocks;
    }
  return (int64_t)kParts * most * d->hidden * 4;
}

int echo_norm_backward(const echo_norm_desc* d, const void* dz, const void* dh_out,
                       const void* h_out, const void* y, const float* stats, const void* gate,
                       const void* w_post, const void* b_post, const void* w_pre, void* dh,
                       void* dy, void* dgate, void* dw_post, void* db_post, void* dw_pre,
                       void* db_pre, void* workspace, int64_t workspace_bytes,
                       echo_stream_t stream) {
  Geometry g;
  int rc = check_desc(d, g);
  if (rc) return rc;
  const bool post = d->post != ECHO_NORM_NONE, pre = d->pre != ECHO_NORM_NONE;
  if ((!post && (w_post || b_post || dw_post || db_post)) || (!pre && (w_pre || dw_pre || db_pre)))
    return ECHO_ERR_INVALID_ARGUMENT;
  if (d->gate_rows == 0 && (gate || dgate)) return ECHO_ERR_INVALID_ARGUMENT;
  if (g.T > 0) {
    if (!dh || (dz != nullptr) != pre || (gate != nullptr) != (d->gate_rows > 0))
      return ECHO_ERR_INVALID_ARGUMENT;
    if ((pre && !h_out) || ((post || dgate) && !y) || ((pre || post) && !stats))
      return ECHO_ERR_INVALID_ARGUMENT;
  }
  void* const outs[kParts] = {dw_pre, db_pre, dw_post, db_post, dgate};
  const bool sums = dw_pre || db_pre || dw_post || db_post || dgate;
  const int64_t need = echo_norm_backward_workspace(d);
  if (sums && need > 0) {
    if (!workspace) return ECHO_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return ECHO_ERR_WORKSPACE;
  }
  for (const void* p : {dz, y, gate, w_post, b_post, w_pre, (const void*)dy, (const void*)dgate,
                        (const void*)dw_post, (const void*)db_post, (const void*)dw_pre,
                        (const void*)db_pre})
    if (!aligned(p, g.e)) return ECHO_ERR_ALIGNMENT;
  if (!aligned(dh_out, g.s) || !aligned(h_out, g.s) || !aligned(dh, g.s) || !aligned(stats, 4) ||
      !aligned(workspace, 16))
    return ECHO_ERR_ALIGNMENT;
  Aliases al;
  al.out(dh, g.dense_s);
  al.out(dy, g.dense);
  al.out(dgate, d->gate_rows * g.H * g.e);
  for (void* p : {dw_post, db_post, dw_pre, db_pre}) al.out(p, g.H * g.e);
  if (sums) al.out(workspace, need);
  al.in(dz, g.dense);
  al.in(dh_out, g.dense_s);
  al.in(h_out, g.h_bytes);
  al.in(y, g.y_bytes);
  al.in(stats, 16 * g.T);
  al.in(gate, d->gate_rows * g.H * g.e);
  for (const void* p : {w_post, b_post, w_pre}) al.in(p, g.H * g.e);
  al.allow_identical(dh, dh_out);
  if (!al.ok()) return ECHO_ERR_ALIAS;

  const bool full = post || d->gate_rows > 0;
  const Walk w = walk_of(g.T, g.H, d->gate_rows, dgate != nullptr, full ? kBackFull : kBackPlain);
  PartSumArgs ps = {};
  ps.hidden = (uint32_t)g.H;
  uint32_t parts = 0, rows = 1, want = 0;
  const int64_t plane = (int64_t)w.blocks * g.H;
  for (int p = 0; p < kParts; ++p) {
    // a gate row of the whole or row kind is written by the row kernel
    // itself; without tokens there are zeros to write
    if (!outs[p] || (p == kDgate && g.T > 0 && w.gate_sum != kGatePart)) continue;
    want |= 1u << p;
    ps.part[parts] = (const float*)workspace + p * plane;
    ps.out[parts] = outs[p];
    ps.rows[parts] = p == kDgate ? (uint32_t)d->gate_rows : 1;
    ps.per_row[parts] = g.T == 0 ? 0 : p == kDgate ? w.blocks_per_gate : w.blocks;
    if (ps.rows[parts] > rows) rows = ps.rows[parts];
    ++parts;
  }
  if (g.T > 0) {
    NormBackArgs a = {};
    a.dz = dz;
    a.dh_out = dh_out;
    a.h_out = h_out;
    a.y = (post || dgate) ? y : nullptr;
    a.stats = stats;
    a.gate = gate;
    a.w_post = w_post;
    a.b_post = b_post;
    a.w_pre = w_pre;
    a.dh = dh;
    a.dy = dy;
    a.dgate = dgate;
    a.part = (float*)workspace;
    a.tokens = g.T;
    a.ld_y = g.ld_y;
    a.ld_h = g.ld_h;
    a.chunk = w.chunk;
    a.hidden = (uint32_t)g.H;
    a.rows_per_gate = d->gate_rows ? (uint32_t)(g.T / d->gate_rows) : 0;
    a.blocks_per_gate = w.blocks_per_gate;
    a.post = d->post;
    a.pre = d->pre;
    a.gate_sum = w.gate_sum;
    a.want = want;
    a.scale = d->scale;
    rc = run_norm_backward(a, w.blocks, full, d->dtype, d->stream_dtype, (hipStream_t)stream);
    if (rc) return rc;
  }
  if (parts == 0) return ECHO_SUCCESS;
  return run_part_sum(ps, parts, rows, d->dtype, (hipStream_t)stream);
}

}  // extern "C"
