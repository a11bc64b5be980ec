// linear8_tile.h -- the tile kernel of the product in 8-bit floating point
// (linear8_device.h has the mathematics and the layout of a fragment).
#pragma once

#include "linear8_device.h"

namespace echo {
namespace {

// four bytes per lane from memory into LDS, as dma16 does it with sixteen
__device__ __forceinline__ void dma4(u32x4 range, lds_short* lds, int offset) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 4\n\t"
      "buffer_load_dword %1, %2, 0 offen lds"
      :
      : "s"((uint32_t)(uintptr_t)lds), "v"(offset), "s"(range)
      : "memory");
}

// a wavefront's descriptor in scalar registers
__device__ __forceinline__ u32x4 uniform(u32x4 r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (uint32_t)__builtin_amdgcn_readfirstlane((int)r[i]);
  return r;
}

// A workgroup computes a BI x BJ tile of sums in steps of one block.  Both
// operands' tiles, rows of 128 bytes, arrive in LDS by direct loads, S stages on
// their way or in use, with chunks permuted as OperandTile has them; so do the
// step's scales, one load a wavefront: the first wavefronts' lanes fetch the tile
// rows' scales of x, the next one's the scale of each fragment of w, and the
// others load as much again to keep one count for all.
// A step whose scales are all powers of two, as echo_pack8 makes them, leaves
// them to the matrix cores; otherwise each fragment pair's product of a block is
// multiplied by its two scales on its way to the sum, four fused multiply-adds for
// 32 cycles of the matrix core.
// Gated, w's tile alternates runs of 32 gate rows and the 32 up rows of the same
// outputs; a wavefront's loads are of one kind, so each kind has a range of its own.
template <typename T, int X, int BI, int BJ, int WI, int WJ, bool GATED, int S>
__global__ __launch_bounds__(64 * WI * WJ, 2) void k_tile8(Tile8Args a) {
  constexpr int NT = 64 * WI * WJ, NW = WI * WJ, TI = BI / WI / 16, TJ = BJ / WJ / 16;
  constexpr int OUT = GATED ? BJ / 2 : BJ;
  static_assert(!GATED || TJ % 4 == 0, "a gated run is 64 rows of one wavefront");
  static_assert(BI / 64 + 1 <= NW && BJ <= 1024, "a wavefront for each scale load");
  static_assert(128 % (BJ / WJ) == 0, "one block of w to a wavefront's columns");
  constexpr int PA = BI * 8 / NT, PB = BJ * 8 / NT;  // chunks of a thread
  constexpr int kTileBytes = (BI + BJ) * kC8, kStage = (kTileBytes + NW * 256) / 2;  // in shorts
  constexpr int kLoads = PA + PB + 1;
  static_assert((S - 1) * kLoads < 64, "loads in flight");
  constexpr int kEpilogue = kEpilogueFloats<TJ>;
  __shared__ union {
    short stage[S * kStage];
    float sums[NW][kEpilogue];
  } mem;
  lds_short* const lds = (lds_short*)mem.stage;
  typedef __attribute__((address_space(3))) const u32x4 lds_chunk;
  typedef __attribute__((address_space(3))) const float lds_float;

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, rho = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wi = wave % WI * (BI / WI), wj = wave / WI * (BJ / WJ);
  const uint32_t b = blockIdx.y * gridDim.x + blockIdx.x;
  if (b >= a.workgroups) return;
  uint32_t ti, tj, split;
  tile_of(b, a.workgroups, a.tiles_i, a.tiles_j, ti, tj, split);
  const int64_t i0 = (int64_t)ti * BI, j0 = (int64_t)tj * OUT;
  const int64_t c0 = (int64_t)split * a.chunk, c1 = min(a.C, c0 + a.chunk);
  const int steps = (int)((c1 - c0 + kC8 - 1) / kC8);
  const int64_t rows_a = min(a.I - i0, (int64_t)BI), rows_b = min(a.J - j0, (int64_t)OUT);
  const int64_t kb = (a.C + kC8 - 1) / kC8;  // blocks along a row

  // Byte offsets of the thread's first chunks; the other chunks and the later steps
  // move the ranges, in scalar registers.  Every one of a thread's chunks has the
  // same place in its row, and gated its rows of w are 32 apart for each 64.
  const int ca = ((tid & 7) ^ (tid >> 3 & 7)) * 16;
  const int oa = (int)(tid / 8 * a.lda) + ca;
  const int ob = (int)((GATED ? tid / 8 & 31 : tid / 8) * a.ldb) + ca;
  const char* const pa = (const char*)a.a + i0 * a.lda + c0;
  const char* const pb = (const char*)a.b + j0 * a.ldb + c0;
  // a last chunk's filling is its row's own
  const int64_t whole = (c1 - c0 + 15) & ~(int64_t)15;
  const int64_t end_a = (rows_a - 1) * a.lda + whole, end_b = (rows_b - 1) * a.ldb + whole;
  // the scale that the lane fetches
  int os;
  u32x4 rs;
  if (wave < BI / 64) {
    os = (int)(min((int64_t)(wave * 64 + lane), rows_a - 1) * kb * 4);
    rs = range_of(a.sx + i0 * kb, rows_a * kb * 4);
  } else {
    const int r = min(lane, BJ / 16 - 1) * 16;
    const int64_t j = min(j0 + (GATED ? (r >> 6) * 32 + (r & 31) : r), a.J - 1), first = j0 / ECHO_FP8_BLOCK;
    const int64_t down = (a.J + ECHO_FP8_BLOCK - 1) / ECHO_FP8_BLOCK;
    os = (int)((j / ECHO_FP8_BLOCK - first + (GATED && (r >> 5 & 1) ? down : 0)) * kb * 4);
    rs = range_of(a.sw + first * kb, ((GATED ? 2 : 1) * down - first) * kb * 4);
  }
  os += (int)(c0 / kC8) * 4;
  rs = uniform(rs);
  constexpr int kPast = 0x7FFFFFF0;  // an offset past every range

  // past the last step nothing is in range, so every step issues as many loads
  auto stage = [&](lds_short* la, int s) {
    const int64_t left = c1 - c0 - (int64_t)s * kC8;  // of the contraction, from this step on
    const bool past = ca >= left;
    const int va = past ? kPast : oa, vb = past ? kPast : ob;
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int64_t on = i * (NT / 8) * a.lda + s * kC8;
      dma16(uniform(range_of(pa + on, end_a - on)), la + (i * NT + wave * 64) * 8, va);
    }
    lds_short* lb = la + BI * kC8 / 2;
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      const bool up = GATED && ((i * (NT / 8) + wave * 8) >> 5 & 1);
      const int64_t on = (GATED ? i * (NT / 8) / 64 * 32 : i * (NT / 8)) * a.ldb + s * kC8;
      dma16(uniform(range_of(pb + on + (up ? a.J * a.ldb : 0), end_b - on)), lb + (i * NT + wave * 64) * 8, vb);
    }
    dma4(rs, la + kTileBytes / 2 + wave * 128, left <= 0 ? kPast : os + s * 4);
  };

  // the two chunks of row `row` that the lane holds
  auto fragment = [&](const lds_short* t, int row) {
    const lds_short* p = t + row * (kC8 / 2);
    return join16(*(lds_chunk*)(p + (g ^ (row & 7)) * 8), *(lds_chunk*)(p + ((g + 4) ^ (row & 7)) * 8));
  };

  f32x4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // what a row's last chunk holds past the row's end: the last step's rows are cut
  // there, in LDS
  const int odd = (int)((c1 - c0) & 15), last = (int)((c1 - c0) & (kC8 - 1)) >> 4;
  auto cut = [&](lds_short* la) {
    typedef __attribute__((address_space(3))) u32x4 chunk;
    for (int r = tid; r < BI + BJ; r += NT) {
      chunk* p = (chunk*)(la + r * (kC8 / 2) + (last ^ (r & 7)) * 8);
      *p = chunk_before(*p, odd);
    }
    __syncthreads();
  };

  // One step's scales, and whether every lane's are powers of two.
  float xs[TI], ws[GATED ? 2 : 1];
  auto read_scales = [&](const lds_short* la) {
    lds_float* scales = (lds_float*)(la + kTileBytes / 2);
    bool powers = true;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      xs[i] = scales[wi + i * 16 + rho];
      powers = powers && is_power(__float_as_uint(xs[i]));
    }
#pragma unroll
    for (int q = 0; q < (GATED ? 2 : 1); ++q) {
      ws[q] = scales[BI + wj / 16 + q * 2];
      powers = powers && is_power(__float_as_uint(ws[q]));
    }
    return __builtin_amdgcn_ballot_w64(!powers) == 0;
  };
  // The step's products, w's fragments read one ahead.  `load` issues the loads of
  // the step S - 1 ahead behind this step's first reads of LDS.
  // (The empty assembly keeps a fragment's sums in their place: moved below the
  // step's other products they would not fit the registers.)
  auto products = [&](const lds_short* la, auto load, auto pair) {
    const lds_short* lb = la + BI * kC8 / 2;
    i32x8 fa[TI], fb[2];
#pragma unroll
    for (int i = 0; i < TI; ++i) fa[i] = fragment(la, wi + i * 16 + rho);
    fb[0] = fragment(lb, wj + rho);
    load();
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      if (j + 1 < TJ) fb[(j + 1) & 1] = fragment(lb, wj + (j + 1) * 16 + rho);
#pragma unroll
      for (int i = 0; i < TI; ++i) pair(fb[j & 1], fa[i], i, j);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto arrived = [&](lds_short* la, int s) {
    dma_wait<(S - 2) * kLoads>();
    __syncthreads();
    if (odd && s == steps - 1) cut(la);
  };

#pragma unroll
  for (int u = 0; u < S - 1; ++u) stage(lds + u * kStage, u);
  lds_short *now = lds, *next = lds + (S - 1) * kStage;
  auto turn = [&] {
    now = now == lds + (S - 1) * kStage ? lds : now + kStage;
    next = next == lds + (S - 1) * kStage ? lds : next + kStage;
  };
  int s = 0;
  bool powers = true;
  for (; s < steps; ++s) {
    arrived(now, s);
    powers = read_scales(now);
    if (!powers) break;
    int ex[TI], ew[GATED ? 2 : 1];
#pragma unroll
    for (int i = 0; i < TI; ++i) ex[i] = (int)(__float_as_uint(xs[i]) >> 23);
#pragma unroll
    for (int q = 0; q < (GATED ? 2 : 1); ++q) ew[q] = (int)(__float_as_uint(ws[q]) >> 23);
    products(now, [&] { stage(next, s + S - 1); }, [&](i32x8 w, i32x8 x, int i, int j) {
      acc[i][j] = mfma8<X>(w, x, acc[i][j], ew[GATED ? j >> 1 & 1 : 0], ex[i]);
    });
    turn();
  }
  // from the first step with another scale on (a wavefront of its own accord: both
  // loops have the same barriers)
  for (; s < steps; ++s) {
    if (powers) {
      arrived(now, s);
      read_scales(now);
    }
    powers = true;
    f32x4 t[2][TI];
    auto add = [&](int j) {
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const float both = xs[i] * ws[GATED ? j >> 1 & 1 : 0];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(t[j & 1][i][e], both, acc[i][j][e]);
        asm volatile("" : "+v"(acc[i][j]));
      }
    };
    products(now, [&] { stage(next, s + S - 1); }, [&](i32x8 w, i32x8 x, int i, int j) {
      t[j & 1][i] = mfma8<X>(w, x, f32x4{0.f, 0.f, 0.f, 0.f});
      if (i == TI - 1 && j > 0) add(j - 1);
    });
    add(TJ - 1);
    turn();
  }
  // nothing may arrive in LDS that the epilogue uses, or after the workgroup has left it
  dma_wait<0>();
  __syncthreads();
  write_tile<T, GATED, TI, TJ>(a, acc, mem.sums[wave], i0 + wi, j0 + (GATED ? wj / 2 : wj), split, lane);
}

template <typename T, int X, int BI, int BJ, int WI, int WJ, bool GATED, int S>
int launch_tile8(Tile8Args a, hipStream_t s) {
  const int64_t out = GATED ? BJ / 2 : BJ;
  const int64_t ti = (a.I + BI - 1) / BI, tj = (a.J + out - 1) / out;
  constexpr int NT = 64 * WI * WJ;
  if (ti * tj == 0) return ECHO_SUCCESS;
  a.tiles_i = (uint32_t)ti;
  a.tiles_j = (uint32_t)tj;
  a.workgroups = a.tiles_i * a.tiles_j * a.splits;  // below 2^32 by ECHO_MAX_PRODUCT
  const TileGrid g = grid_of(a.workgroups, NT);
  return launch(k_tile8<T, X, BI, BJ, WI, WJ, GATED, S>, dim3(g.x, g.y), dim3(NT), s, a);
}

template <typename T, int X, bool GATED>
int forward8(const Tile8Args& a, int tile, hipStream_t s) {
  constexpr int SI = GATED ? 4 : 2, SJ = GATED ? 1 : 2;  // a gated run is 64 rows of w, in one wavefront
  switch (tile) {
    case kTile256: return launch_tile8<T, X, 256, 256, 4, 2, GATED, 2>(a, s);
    case kTile256x128: return launch_tile8<T, X, 256, 128, 4, 2, GATED, 3>(a, s);
    case kTile128: return launch_tile8<T, X, 128, 128, 2, 2, GATED, 2>(a, s);
    default: return launch_tile8<T, X, 64, 64, SI, SJ, GATED, 4>(a, s);
  }
}

}  // namespace
}  // namespace echo
