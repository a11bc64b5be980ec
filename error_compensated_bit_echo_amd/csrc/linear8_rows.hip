// linear8_rows.hip -- the product in 8-bit floating point for a few rows of x: a
// decode step's.
//
// As in linear_rows.hip: every weight is read once, straight into registers, and
// meets at most 16 rows, so the call is bound by reading w from HBM, and by latency
// where w is small.  A workgroup takes 16 rows of w (gated, the gate and up rows of
// 8 outputs), its 8 wavefronts deal the contraction's blocks of 128 among them, and
// the eight sums of an output are added through LDS in a fixed order.  Lane 16 g +
// rho holds the 32 bytes 32 g .. + 31 of a block of row rho, of w and of x.
#include "linear8_device.h"

namespace echo {
namespace {

constexpr int kWaves8 = 8;

// U: blocks whose weights are held at once
template <typename T, int X, int U, bool GATED>
__global__ __launch_bounds__(64 * kWaves8) void k_rows8(Tile8Args a) {
  constexpr int OUT = GATED ? 8 : 16;
  __shared__ f32x4 lds[kWaves8][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, rho = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t j0 = (int64_t)blockIdx.x * OUT;
  const int64_t kb = (a.C + kC8 - 1) / kC8, down = (a.J + ECHO_FP8_BLOCK - 1) / ECHO_FP8_BLOCK;
  // rows past the end repeat the last one; their sums are not written
  const int64_t wrow = min(j0 + rho % OUT, a.J - 1) + (rho < OUT ? 0 : a.J);
  const uint8_t* const w = (const uint8_t*)a.b + wrow * a.ldb + g * 32;
  const int64_t xrow = min((int64_t)rho, a.I - 1);
  const uint8_t* const x = (const uint8_t*)a.a + xrow * a.lda + g * 32;
  const float* const sx = a.sx + xrow * kb;
  // the lane's sums are of rows 4 g .. + 3 of w: gated, gate rows or up rows
  const float* const sw = a.sw + (j0 / ECHO_FP8_BLOCK + (GATED && g >= 2 ? down : 0)) * kb;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto add = [&](i32x8 fw, i32x8 fx, float s) {
    const f32x4 t = mfma8<X>(fw, fx, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = fmaf(t[e], s, acc[e]);
  };

  // a block past the end repeats the last one's loads and is not multiplied
  const int full = (int)(a.C / kC8), rest = (int)(a.C % kC8);
  auto block_at = [&](int s) { return (int64_t)min(s, full - 1); };
  u32x4 fw[2][U][2];
  auto load_w = [&](u32x4 (&f)[U][2], int s) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        f[u][q] = __builtin_nontemporal_load((const u32x4*)(w + block_at(s + u * kWaves8) * kC8 + q * 16));
  };
  auto multiply = [&](const u32x4 (&f)[U][2], int s) {
    u32x4 fx[U][2];
    float ss[U], ts[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = block_at(s + u * kWaves8);
#pragma unroll
      for (int q = 0; q < 2; ++q) fx[u][q] = *(const u32x4*)(x + at * kC8 + q * 16);
      ss[u] = sx[at];
      ts[u] = sw[at];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u * kWaves8 < full) add(join16(f[u][0], f[u][1]), join16(fx[u][0], fx[u][1]), ss[u] * ts[u]);
  };
  constexpr int kGroup = kWaves8 * U;
  if (wave < full) {
    load_w(fw[0], wave);
    for (int s = wave; s < full; s += 2 * kGroup) {
      if (s + kGroup < full) load_w(fw[1], s + kGroup);
      multiply(fw[0], s);
      if (s + 2 * kGroup < full) load_w(fw[0], s + 2 * kGroup);
      if (s + kGroup < full) multiply(fw[1], s + kGroup);
    }
  }
  if (rest && wave == full % kWaves8) {
    const int64_t c = (int64_t)full * kC8;
    u32x4 cw[2], cx[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int n = rest - g * 32 - q * 16;
      cw[q] = cx[q] = u32x4{0, 0, 0, 0};
      if (n > 0) {  // a chunk with one byte of the row lies within its pitch
        cw[q] = chunk_before(*(const u32x4*)(w + c + q * 16), n);
        cx[q] = chunk_before(*(const u32x4*)(x + c + q * 16), n);
      }
    }
    add(join16(cw[0], cw[1]), join16(cx[0], cx[1]), sx[full] * sw[full]);
  }
  lds[wave][lane] = acc;
  __syncthreads();
  // the first wavefront finishes: a lane has four rows of w for one of x; gated,
  // the up rows are 32 lanes after their gate's
  const int64_t col = j0 + g * 4;
  if (wave > 0 || lane >= OUT * 4 || rho >= a.I || col >= a.J) return;
  float v[4], u[4];
  f32x4 sum = lds[0][lane];
#pragma unroll
  for (int k = 1; k < kWaves8; ++k) sum += lds[k][lane];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = sum[e];
  if constexpr (GATED) {
    sum = lds[0][lane + 32];
#pragma unroll
    for (int k = 1; k < kWaves8; ++k) sum += lds[k][lane + 32];
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = sum[e];
  }
  finish<T, 4, GATED>(a, rho, col, (int)min(a.J - col, (int64_t)4), v, u);
}

template <typename T, int X, bool GATED>
int rows(const Tile8Args& a, hipStream_t s) {
  const int64_t out = GATED ? 8 : 16;
  const dim3 grid((uint32_t)((a.J + out - 1) / out)), block(64 * kWaves8);
  return launch(k_rows8<T, X, 4, GATED>, grid, block, s, a);
}

template <typename T, int X>
int rows(const Tile8Args& a, bool gated, hipStream_t s) {
  return gated ? rows<T, X, true>(a, s) : rows<T, X, false>(a, s);
}

}  // namespace

int rows8_forward(const Tile8Args& a, int32_t dtype, int32_t format, bool gated, hipStream_t s) {
  if (dtype == ECHO_BF16) return format == ECHO_E4M3 ? rows<bf16_t, 0>(a, gated, s) : rows<bf16_t, 1>(a, gated, s);
  return format == ECHO_E4M3 ? rows<f16_t, 0>(a, gated, s) : rows<f16_t, 1>(a, gated, s);
}

}  // namespace echo
