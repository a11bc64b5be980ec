// linear8_tile.h -- the tile kernel of the product in 8-bit floating point
// (linear8_device.h has the mathematics and the layout of a fragment).
#pragma once

#include "linear8_device.h"

namespace echo {
namespace {

// As dma16, with `step` more bytes in a scalar register, and with one word a lane.  (A
// range is checked with or without `step`: what the calls below mean to be past its end is
// so by the lane's offset alone.)
__device__ __forceinline__ void dma16(u32x4 range, lds_short* lds, int offset, int step) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 4\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"((uint32_t)(uintptr_t)lds), "v"(offset), "s"(range), "s"(step)
      : "memory");
}
__device__ __forceinline__ void dma4(u32x4 range, lds_short* lds, int offset, int step) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 4\n\t"
      "buffer_load_dword %1, %2, %3 offen lds"
      :
      : "s"((uint32_t)(uintptr_t)lds), "v"(offset), "s"(range), "s"(step)
      : "memory");
}

// a wavefront's descriptor in scalar registers
__device__ __forceinline__ u32x4 uniform(u32x4 r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (uint32_t)__builtin_amdgcn_readfirstlane((int)r[i]);
  return r;
}

// A wavefront's sums to the epilogue or to a split's partial sums, through LDS as
// write_tile has them.  A short contraction's time is this one's: the bias is the same for
// all of a lane's rows and is read once, the residual of a pass is on its way three passes
// before it is added (two: 5 % more), and the passes are unrolled.  26490 x 480 x 94 with
// bias, residual and p kept 35.7 -> 26.9 us, 8192 x 4096 x 256 with residual 54.1 -> 45.6,
// 8192 x 4096 x 1792 94.1 -> 85.3, 131072 x 1792 x 4096 913 -> 905.  With exact GELU's gate
// (23589 x 2944 x 128: 112 us) it is bound by the activation's arithmetic.
template <typename T, bool GATED, int TI, int TJ>
__device__ __forceinline__ void write_tile8(const TileArgs& a, const f32x4 (&acc)[TI][TJ], float* lds, int64_t i0,
                                            int64_t j0, uint32_t split, int lane) {
  constexpr int kPitch = TJ * 16, kOut = GATED ? TJ * 8 : TJ * 16;  // outputs of the wavefront's tile
  constexpr int kLanes = kOut / 8, kRowsOf = 64 / kLanes;          // lanes to a row, rows to a pass
  constexpr int kTurn = TJ * 4 < 16 ? TJ * 4 - 1 : 15;             // bits of a row's number that permute
  constexpr int kAhead = 3;
  const int g = lane >> 4, rho = lane & 15;
  const int64_t cols = GATED ? 2 * a.J : a.J;
  const int c = lane % kLanes * 8, in_pass = lane / kLanes;
  const int at = (GATED ? c / 32 * 64 + c % 32 : c) / 4;
  const int64_t col = j0 + c;
  const int n = (int)min(a.J - col, (int64_t)8);
  const bool joins = a.splits == 1, whole = n == 8;
  float bg[8], bu[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) bg[e] = bu[e] = 0.f;
  if (joins && a.bias) {
    load_n<false>((const T*)a.bias + col, n, bg);
    if (GATED) load_n<false>((const T*)a.bias + a.J + col, n, bu);
  }
  const bool adds = joins && a.residual;
  u32x4 res[kAhead] = {};
  auto fetch = [&](int r) {  // the residual of the pass at row r of the tile
    const int64_t row = min(i0 + r + in_pass, a.I - 1);
    return *(const u32x4_a2*)((const T*)a.residual + row * a.ldr + col);
  };
  if (adds && whole)
#pragma unroll
    for (int p = 0; p < kAhead; ++p) res[p] = fetch(p * kRowsOf);
  auto read = [&](int r, float (&v)[8], float (&u)[8]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const f32x4 x = *(const f32x4*)(lds + r * kPitch + ((at + e) ^ (r & kTurn)) * 4);
      const f32x4 y = GATED ? *(const f32x4*)(lds + r * kPitch + ((at + 8 + e) ^ (r & kTurn)) * 4) : x;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[e * 4 + q] = x[q];
        u[e * 4 + q] = y[q];
      }
    }
  };
#pragma unroll
  for (int i = 0; i < TI; ++i) {
#pragma unroll
    for (int j = 0; j < TJ; ++j) *(f32x4*)(lds + rho * kPitch + ((j * 4 + g) ^ (rho & kTurn)) * 4) = acc[i][j];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r = 0; r < 16; r += kRowsOf) {
      float v[8], u[8];
      read(r + in_pass, v, u);
      u32x4 next = {};
      if (adds && whole) next = fetch(i * 16 + r + kAhead * kRowsOf);
      const int64_t row = i0 + i * 16 + r + in_pass;
      if (row < a.I && n > 0) {
        if (!joins) {
          float* p = a.part + ((int64_t)split * a.I + row) * cols + col;
          store_n<false>(p, n, v);
          if (GATED) store_n<false>(p + a.J, n, u);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] += bg[e];
            if (GATED) u[e] += bu[e];
          }
          if (a.p) {
            T* p = (T*)a.p + row * cols + col;
            store_n<false>(p, n, v);
            if (GATED) store_n<false>(p + a.J, n, u);
          }
          with_act(a.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float slope;
              act_slope<decltype(act)::value>(v[e], v[e], slope);
            }
          });
          float f[8];
          if (adds) {
            if (whole) unpack8(res[0], f, T{});
            else load_n<false>((const T*)a.residual + row * a.ldr + col, n, f);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (GATED) v[e] *= u[e];
            if (adds) v[e] += f[e];
          }
          store_n<false>((T*)a.out + row * a.ldo + col, n, v);
        }
      }
#pragma unroll
      for (int p = 0; p + 1 < kAhead; ++p) res[p] = res[p + 1];
      res[kAhead - 1] = next;
    }
    __builtin_amdgcn_wave_barrier();
  }
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
// WK sets of wavefronts take the blocks in turn, each with stages and scales of its
// own, and their sums are added at the end: a small tile's step is bound by the way
// from the barrier through LDS to its few products, not by their number.
//
// What bounds it: a step of 256 x 256 takes 1.7 us, and 1.14 of them without its loads
// (products and fragments alone; the matrix cores' own 2048 cycles are .85 at 2.4 GHz):
// the 64 KB from the second-level cache to LDS, 30 bytes a cycle and compute
// unit, do not hide whole.  A tile's filling and epilogue are another 11 us, 8 of them
// stores, which nothing of a lone workgroup covers.  131072 x 1792 x 4096 in 876 to 905 us
// (2.13 to 2.20 PFLOP/s), 8192 x 1792 x 4096 gated in 124 with powers of two and 132 with
// other scales, 256 x 4096 x 1792 in 10.5 (64 x 64, four sets).
// Measured and slower: a step with scales whose product is below 2^-126 added once more, by
// one scale after the other (a branch at the end of each step with other scales: 8192 x 1792
// x 4096 gated 124 -> 128 us, 131072 x 1792 x 4096 985 -> 1005; the header has what such
// products lose); fragments read across the steps' barrier; four wavefronts of 128 x
// 128 (1.86 us a step); loads into the second-level cache ahead of the tile's; two stages
// more for lone small tiles; outputs stored around the caches; workgroups that go on to a
// next tile with its first loads under the epilogue (2 to 4 % slower).
template <typename T, int X, int BI, int BJ, int WI, int WJ, bool GATED, int S, int WK>
__global__ __launch_bounds__(64 * WI * WJ * WK, WI * WJ * WK / 4 < 2 ? 2 : WI * WJ * WK / 4) void k_tile8(Tile8Args a) {
  constexpr int NT = 64 * WI * WJ, NW = WI * WJ, TI = BI / WI / 16, TJ = BJ / WJ / 16;  // NT, NW: of a set
  constexpr int OUT = GATED ? BJ / 2 : BJ;
  static_assert(!GATED || TJ % 4 == 0, "a gated run is 64 rows of one wavefront");
  static_assert(BI / 64 + 1 <= NW && BJ <= 1024, "a wavefront for each scale load");
  static_assert(128 % (BJ / WJ) == 0, "one block of w to a wavefront's columns");
  constexpr int PA = BI * 8 / NT, PB = BJ * 8 / NT;  // chunks of a thread
  constexpr int kStage = (BI + BJ) * kC8 / 2;  // in shorts
  constexpr int kLoads = PA + PB;              // and in some steps one of scales
  static_assert((S - 1) * (kLoads + 1) < 64, "loads in flight");
  constexpr int kScales = BI / 64 + 1;  // wavefronts that load scales
  // steps whose scales are there: a group of four is loaded over one that every
  // wavefront has left behind
  constexpr int kRing = WK > 1 ? 4 : 8;
  static_assert(S <= (WK > 1 ? kRing : kRing - 3), "scales in flight");
  constexpr int kEpilogue = kEpilogueFloats<TJ>;
  __shared__ union {
    struct {
      short stage[WK][S * kStage];
      float scales[WK][kRing][kScales * 64];
    };
    struct {
      float sums[NW][kEpilogue];
      f32x4 others[WK > 1 ? WK - 1 : 1][WK > 1 ? NW : 1][TI * TJ][64];
    };
  } mem;
  typedef __attribute__((address_space(3))) const float lds_float;
  typedef __attribute__((address_space(3))) const u32x4 lds_chunk;

  const int lane = threadIdx.x & 63, g = lane >> 4, rho = lane & 15;
  const int part = WK > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / NW : 0;  // the set
  const int tid = threadIdx.x - part * NT;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  lds_short* const lds = (lds_short*)mem.stage[part];
  float* const scales_at = mem.scales[part][0];
  lds_float* const lds_scales = (lds_float*)scales_at;
  const int wi = wave % WI * (BI / WI), wj = wave / WI * (BJ / WJ);
  const uint32_t b = blockIdx.y * gridDim.x + blockIdx.x;
  if (b >= a.workgroups) return;
  uint32_t ti, tj, split;
  tile_of(b, a.workgroups, a.tiles_i, a.tiles_j, ti, tj, split);
  const int64_t i0 = (int64_t)ti * BI, j0 = (int64_t)tj * OUT;
  const int64_t c0 = (int64_t)split * a.chunk, c1 = min(a.C, c0 + a.chunk);
  const int blocks = (int)((c1 - c0 + kC8 - 1) / kC8), steps = (blocks + WK - 1) / WK;
  const int64_t rows_a = min(a.I - i0, (int64_t)BI), rows_b = min(a.J - j0, (int64_t)OUT);
  const int64_t kb = (a.C + kC8 - 1) / kC8;  // blocks along a row

  // Byte offsets of the thread's first chunks; the other chunks and the later steps
  // move the ranges, in scalar registers.  Every one of a thread's chunks has the
  // same place in its row, and gated its rows of w are 32 apart for each 64.
  const int ca = ((tid & 7) ^ (tid >> 3 & 7)) * 16;
  int oa[PA], ob[PB];
#pragma unroll
  for (int i = 0; i < PA; ++i) oa[i] = (int)((i * (NT / 8) + tid / 8) * a.lda) + ca;
#pragma unroll
  for (int i = 0; i < PB; ++i) {
    const int r = i * (NT / 8) + tid / 8;
    ob[i] = (int)((GATED ? (r >> 6) * 32 + (r & 31) : r) * a.ldb) + ca;
  }
  const char* const pa = (const char*)a.a + i0 * a.lda + c0;
  const char* const pb = (const char*)a.b + j0 * a.ldb + c0;
  // a last chunk's filling is its row's own
  const int64_t whole = (c1 - c0 + 15) & ~(int64_t)15;
  const int64_t end_a = (rows_a - 1) * a.lda + whole, end_b = (rows_b - 1) * a.ldb + whole;
  const u32x4 ra = uniform(range_of(pa, end_a)), rb = uniform(range_of(pb, end_b));
  const u32x4 ru = GATED ? uniform(range_of(pb + a.J * a.ldb, end_b)) : rb;
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

  // The step's block of the set.  Past the last one nothing is in range, so every step
  // issues as many loads.
  auto stage = [&](lds_short* la, int step) {
    const int s = step * WK + part;
    const int64_t left = c1 - c0 - (int64_t)s * kC8;  // of the contraction, from this step on
    const bool past = ca >= left;
    if (wave < kScales) {
      // four steps' scales at once, where their rows begin at 16 bytes (8192 x 4096 x 4096
      // 139 us, 144 one by one; 32768 rows 539 and 559)
      if (WK == 1 && a.wide) {
        if (s % 4 == 0)
          dma16(rs, (lds_short*)(scales_at + (s % kRing / 4 * kScales + wave) * 256), left <= 0 ? kPast : os, s * 4);
      } else {
        dma4(rs, (lds_short*)(scales_at + (step % kRing * kScales + wave) * 64), left <= 0 ? kPast : os, s * 4);
      }
    }
#pragma unroll
    for (int i = 0; i < PA; ++i) dma16(ra, la + (i * NT + wave * 64) * 8, past ? kPast : oa[i], s * kC8);
    lds_short* lb = la + BI * kC8 / 2;
#pragma unroll
    for (int i = 0; i < PB; ++i)
      dma16(GATED && ((i * (NT / 8) + wave * 8) >> 5 & 1) ? ru : rb, lb + (i * NT + wave * 64) * 8, past ? kPast : ob[i], s * kC8);
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
    if ((blocks - 1) % WK == part) {
      for (int r = tid; r < BI + BJ; r += NT) {
        chunk* p = (chunk*)(la + r * (kC8 / 2) + (last ^ (r & 7)) * 8);
        *p = chunk_before(*p, odd);
      }
    }
    __syncthreads();
  };

  // One step's scales, and whether every lane's are powers of two.
  float xs[TI], ws[GATED ? 2 : 1];
  const int wide = WK == 1 && a.wide ? 4 : 1;
  auto read_scales = [&](int s) {
    lds_float* scales = lds_scales + (WK == 1 && a.wide ? s % kRing / 4 * kScales * 256 + s % 4 : s % kRing * kScales * 64);
    bool powers = true;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      xs[i] = scales[(wi + i * 16 + rho) * wide];
      powers = powers && is_power(__float_as_uint(xs[i]));
    }
#pragma unroll
    for (int q = 0; q < (GATED ? 2 : 1); ++q) {
      ws[q] = scales[(BI + wj / 16 + q * 2) * wide];
      powers = powers && is_power(__float_as_uint(ws[q]));
    }
    return __builtin_amdgcn_ballot_w64(!powers) == 0;
  };
  // A step begins with its first fragments and the loads of the step S - 1 ahead; its
  // scales are read behind them, so that nothing waits for their way to the branch
  // alone.
  i32x8 fa[TI], fb[2];
  lds_short *now = lds, *next = lds + (S - 1) * kStage;
  auto arrive = [&](int s) {
    dma_wait<(S - 2) * kLoads>();
    __syncthreads();
    if (odd && s == steps - 1) cut(now);
  };
  auto read_first = [&] {
#pragma unroll
    for (int i = 0; i < TI; ++i) fa[i] = fragment(now, wi + i * 16 + rho);
    fb[0] = fragment(now + BI * kC8 / 2, wj + rho);
  };
  // The step's products, w's fragments read one ahead.
  auto products = [&](auto pair) {
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      if (j + 1 < TJ) fb[(j + 1) & 1] = fragment(now + BI * kC8 / 2, wj + (j + 1) * 16 + rho);
#pragma unroll
      for (int i = 0; i < TI; ++i) pair(i, j);
      __builtin_amdgcn_sched_barrier(0);
    }
    now = now == lds + (S - 1) * kStage ? lds : now + kStage;
    next = next == lds + (S - 1) * kStage ? lds : next + kStage;
  };

#pragma unroll
  for (int u = 0; u < S - 1; ++u) stage(lds + u * kStage, u);
  int s = 0;
  bool powers = true;
  for (; s < steps; ++s) {
    arrive(s);
    read_first();
    stage(next, s + S - 1);
    powers = read_scales(s);
    if (!powers) break;
    int ex[TI], ew[GATED ? 2 : 1];
#pragma unroll
    for (int i = 0; i < TI; ++i) ex[i] = (int)(__float_as_uint(xs[i]) >> 23);
#pragma unroll
    for (int q = 0; q < (GATED ? 2 : 1); ++q) ew[q] = (int)(__float_as_uint(ws[q]) >> 23);
    products([&](int i, int j) { acc[i][j] = mfma8<X>(fb[j & 1], fa[i], acc[i][j], ew[GATED ? j >> 1 & 1 : 0], ex[i]); });
  }
  // From the first step with another scale on (a wavefront of its own accord: both loops
  // have the same barriers).  A fragment's products are added while the next one's are
  // made; the empty assembly keeps that place: moved below the step's other products they
  // would not fit the registers.
  for (; s < steps; ++s) {
    if (powers) arrive(s);
    read_first();
    if (powers) stage(next, s + S - 1);
    read_scales(s);
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
    products([&](int i, int j) {
      t[j & 1][i] = mfma8<X>(fb[j & 1], fa[i], f32x4{0.f, 0.f, 0.f, 0.f});
      if (i == TI - 1 && j > 0) add(j - 1);
    });
    add(TJ - 1);
  }
  // nothing may arrive in LDS that the epilogue uses, or after the workgroup has left it
  dma_wait<0>();
  __syncthreads();
  if constexpr (WK > 1) {
    f32x4* const mine = mem.others[part > 0 ? part - 1 : 0][wave][0] + lane;
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        if (part > 0) mine[(i * TJ + j) * 64] = acc[i][j];
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int p = 0; p < WK - 1; ++p)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] += mem.others[p][wave][i * TJ + j][lane];
  }
  write_tile8<T, GATED, TI, TJ>(a, acc, mem.sums[wave], i0 + wi, j0 + (GATED ? wj / 2 : wj), split, lane);
}

template <typename T, int X, int BI, int BJ, int WI, int WJ, bool GATED, int S, int WK = 1>
int launch_tile8(Tile8Args a, hipStream_t s) {
  const int64_t out = GATED ? BJ / 2 : BJ;
  const int64_t ti = (a.I + BI - 1) / BI, tj = (a.J + out - 1) / out;
  constexpr int NT = 64 * WI * WJ * WK;
  if (ti * tj == 0) return ECHO_SUCCESS;
  a.tiles_i = (uint32_t)ti;
  a.tiles_j = (uint32_t)tj;
  a.workgroups = a.tiles_i * a.tiles_j * a.splits;  // below 2^32 by ECHO_MAX_PRODUCT
  const TileGrid g = grid_of(a.workgroups, NT);
  return launch(k_tile8<T, X, BI, BJ, WI, WJ, GATED, S, WK>, dim3(g.x, g.y), dim3(NT), s, a);
}

// Where a tile's workgroups are no more than the compute units, one has a unit to itself
// and room for more sets of wavefronts (64 x 2048 x 2048 9.7 us, with one set 11.7; 1024 x
// 1024 x 4096 16.4 and 19.6; 2048 x 2048 x 2048 20.2 and 21.9; 256 x 4096 x 1792 11.5 and
// 11.7, weights from HBM).
template <typename T, int X, bool GATED>
int forward8(const Tile8Args& a, int tile, hipStream_t s) {
  constexpr int SI = GATED ? 4 : 2, SJ = GATED ? 1 : 2;  // a gated run is 64 rows of w, in one wavefront
  const TileCost& k = kCost8[tile];
  const int64_t cols = GATED ? 2 * a.J : a.J;
  const bool alone = ((a.I + k.bi - 1) / k.bi) * ((cols + k.bj - 1) / k.bj) * a.splits <= 256;
  switch (tile) {
    case kTile256: return launch_tile8<T, X, 256, 256, 4, 2, GATED, 2>(a, s);
    case kTile128:
      if (alone) return launch_tile8<T, X, 128, 128, 2, 2, GATED, 2, 2>(a, s);
      return launch_tile8<T, X, 128, 128, 2, 2, GATED, 2>(a, s);
    default:
      if (alone) return launch_tile8<T, X, 64, 64, SI, SJ, GATED, 2, 4>(a, s);
      return launch_tile8<T, X, 64, 64, SI, SJ, GATED, 4>(a, s);
  }
}

}  // namespace
}  // namespace echo
