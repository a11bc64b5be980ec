// linear8_rows.hip -- the product in 8-bit floating point for a few rows of x: a
// decode step's.
//
// As in linear_rows.hip: every weight is read once, straight into registers, and
// meets at most 16 rows, so the call is bound by reading w from HBM, and by latency
// where w is small.  A workgroup's eight wavefronts share 16 rows of w (gated, the gate
// and up rows of 8 outputs), deal the contraction's blocks of 128 among them, and add
// their sums of an output through LDS in a fixed order.  Lane 16 g + rho holds bytes
// 16 g .. + 15 of both halves of a block of row rho, of w and of x, so a load takes 64
// neighbours of each row.
// One row of x, weights from HBM: 32768 x 4096 in 28.8 us (4.7 TB/s), 8192 x 8192 in 16.4
// (4.1), 4096 x 4096 in 6.1, 4096 x 1792 in 4.2, 1792 x 4096 gated in 5.9; 16 rows 1 to 7 us
// more, for x, which every workgroup reads from the second-level cache.  What bounds the
// small ones is one wavefront's way through its loads; 16 wavefronts took 16.6 us for 8192
// x 8192 and 5.8 for 4096 x 4096, but 15.3 for 9.6 of 32768 x 1024.  Loads that leave the
// weights out of the caches took 17.2 us where w fits them (8192 x 8192), these 13.2.
#include "linear8_device.h"

namespace echo {
namespace {

constexpr int KW = 8;  // wavefronts

// U: blocks that are fetched together
template <typename T, int X, int U, bool GATED>
__global__ __launch_bounds__(64 * KW, 4) void k_rows8(Tile8Args a) {
  constexpr int OUT = GATED ? 8 : 16;
  __shared__ f32x4 lds[KW][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, rho = lane & 15;
  const int turn = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t j0 = (int64_t)blockIdx.x * OUT;
  const int64_t kb = (a.C + kC8 - 1) / kC8, down = (a.J + ECHO_FP8_BLOCK - 1) / ECHO_FP8_BLOCK;
  // rows past the end repeat the last one; their sums are not written
  const int64_t wrow = min(j0 + rho % OUT, a.J - 1) + (rho < OUT ? 0 : a.J);
  const uint8_t* const w = (const uint8_t*)a.b + wrow * a.ldb + g * 16;
  const int64_t xrow = min((int64_t)rho, a.I - 1);
  const uint8_t* const x = (const uint8_t*)a.a + xrow * a.lda + g * 16;
  const float* const sx = a.sx + xrow * kb;
  // the lane's sums are of rows 4 g .. + 3 of w: gated, gate rows or up rows
  const float* const sw = a.sw + (j0 / ECHO_FP8_BLOCK + (GATED && g >= 2 ? down : 0)) * kb;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto add = [&](i32x8 fw, i32x8 fx, float s) {
    const f32x4 t = mfma8<X>(fw, fx, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = fmaf(t[e], s, acc[e]);
  };

  // U blocks' operands and scales, fetched together: fetched later, x would be waited for
  // with the weights after it.  A block past the end repeats the last one's loads and is
  // not multiplied.
  const int full = (int)(a.C / kC8), rest = (int)(a.C % kC8);
  struct Group {
    u32x4 w[U][2], x[U][2];
    float sx[U], sw[U];
  } f[2];
  auto fetch = [&](Group& q, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = min(s + u * KW, full - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        q.w[u][h] = *(const u32x4*)(w + at * kC8 + h * 64);
        q.x[u][h] = *(const u32x4*)(x + at * kC8 + h * 64);
      }
      q.sx[u] = sx[at];
      q.sw[u] = sw[at];
    }
  };
  auto multiply = [&](const Group& q, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u * KW < full) add(join16(q.w[u][0], q.w[u][1]), join16(q.x[u][0], q.x[u][1]), q.sx[u] * q.sw[u]);
  };
  constexpr int kGroup = KW * U;
  if (turn < full) {
    fetch(f[0], turn);
    for (int s = turn; s < full; s += 2 * kGroup) {
      if (s + kGroup < full) fetch(f[1], s + kGroup);
      multiply(f[0], s);
      if (s + 2 * kGroup < full) fetch(f[0], s + 2 * kGroup);
      if (s + kGroup < full) multiply(f[1], s + kGroup);
    }
  }
  if (rest && turn == full % KW) {
    const int64_t c = (int64_t)full * kC8;
    u32x4 cw[2], cx[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int n = rest - g * 16 - q * 64;
      cw[q] = cx[q] = u32x4{0, 0, 0, 0};
      if (n > 0) {  // a chunk with one byte of the row lies within its pitch
        cw[q] = chunk_before(*(const u32x4*)(w + c + q * 64), n);
        cx[q] = chunk_before(*(const u32x4*)(x + c + q * 64), n);
      }
    }
    add(join16(cw[0], cw[1]), join16(cx[0], cx[1]), sx[full] * sw[full]);
  }
  lds[turn][lane] = acc;
  __syncthreads();
  // the first of them finishes: a lane has four rows of w for one of x; gated,
  // the up rows are 32 lanes after their gate's
  const int64_t col = j0 + g * 4;
  if (turn > 0 || lane >= OUT * 4 || rho >= a.I || col >= a.J) return;
  float v[4], u[4];
  f32x4 sum = lds[0][lane];
#pragma unroll
  for (int k = 1; k < KW; ++k) sum += lds[k][lane];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = sum[e];
  if constexpr (GATED) {
    sum = lds[0][lane + 32];
#pragma unroll
    for (int k = 1; k < KW; ++k) sum += lds[k][lane + 32];
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = sum[e];
  }
  finish<T, 4, GATED>(a, rho, col, (int)min(a.J - col, (int64_t)4), v, u);
}

// Two blocks a wavefront fetches together where it has four or more, else one: 32768 x
// 1024 9.7 us with one and 15.6 with two, 16384 x 2048 8.7 and 10.1, 4096 x 4096 6.4 and
// 6.1, 8192 x 4096 9.9 and 9.2.
template <typename T, int X, bool GATED>
int rows(const Tile8Args& a, hipStream_t s) {
  constexpr int kOut = GATED ? 8 : 16;
  const dim3 grid((uint32_t)((a.J + kOut - 1) / kOut)), block(64 * KW);
  if (a.C <= 2 * KW * kC8) return launch(k_rows8<T, X, 1, GATED>, grid, block, s, a);
  return launch(k_rows8<T, X, 2, GATED>, grid, block, s, a);
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
