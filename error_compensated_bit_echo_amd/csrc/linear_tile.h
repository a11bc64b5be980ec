// linear_tile.h -- the tile kernel of the matrix products (linear_device.h has
// its parts and the layout).  Each product's source file instantiates it.
#pragma once

#include "host_checks.h"
#include "linear_device.h"

namespace echo {
namespace {

// eight elements of which the first n exist, the others 0
template <typename T>
__device__ __forceinline__ u32x4 raw8(const T* p, int64_t n) {
  if (n >= 8) return *reinterpret_cast<const u32x4_a2*>(p);
  u32x4 w = {0, 0, 0, 0};
  if (n > 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) w[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[i]) << (i % 2 * 16);
  }
  return w;
}

// A wavefront's sums to the epilogue, or to a split's partial sums.  Lane 16 g +
// rho holds, for row rho of each of A's fragments, four neighbours along j of
// each of B's; written as they are, a store would cover 32 bytes of sixteen
// rows.  So they go through LDS, which the operands no longer need: one of A's
// fragments at a time into the wavefront's own part of it, and back with eight
// neighbours to a lane and whole lines of C to a store.  (The code of the
// epilogue proper then stands once for all of the wavefront's sums.)
// The groups of four sums of a row are permuted by an exclusive-or with its
// number against bank conflicts.
template <int TJ>
constexpr int kEpilogueFloats = 16 * TJ * 16;  // of a wavefront

template <typename T, bool GATED, int TI, int TJ>
__device__ __forceinline__ void write_tile(const TileArgs& a, const f32x4 (&acc)[TI][TJ], float* lds, int64_t i0,
                                           int64_t j0, uint32_t split, int lane) {
  constexpr int kPitch = TJ * 16, kOut = GATED ? TJ * 8 : TJ * 16;  // outputs of the wavefront's tile
  constexpr int kLanes = kOut / 8, kRowsOf = 64 / kLanes;          // lanes to a row, rows to a pass
  constexpr int kTurn = TJ * 4 < 16 ? TJ * 4 - 1 : 15;             // bits of a row's number that permute
  const int g = lane >> 4, rho = lane & 15;
  const int64_t cols = GATED ? 2 * a.J : a.J;
  const int c = lane % kLanes * 8, in_pass = lane / kLanes;
  // gated, runs of 32 gate sums and their 32 up sums alternate
  const int at = (GATED ? c / 32 * 64 + c % 32 : c) / 4;
  const int64_t col = j0 + c;
  const int n = (int)min(a.J - col, (int64_t)8);
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
    float v[8], u[8];
    read(in_pass, v, u);
#pragma unroll 1
    for (int r = 0; r < 16; r += kRowsOf) {
      float nv[8], nu[8];  // the next pass's sums on their way
      read(min(r + kRowsOf, 16 - kRowsOf) + in_pass, nv, nu);
      const int64_t row = i0 + i * 16 + r + in_pass;
      if (row < a.I && n > 0) {
        if (a.splits > 1) {
          float* p = a.part + ((int64_t)split * a.I + row) * cols + col;
          store_n<false>(p, n, v);
          if (GATED) store_n<false>(p + a.J, n, u);
        } else {
          finish<T, 8, GATED>(a, row, col, n, v, u);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = nv[e];
        u[e] = nu[e];
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Operands of any pitch and alignment: chunks go through registers, D steps
// ahead of their use, since a step of a small tile is far shorter than a load.
template <typename T, bool TA, bool TB, int BI, int BJ, int WI, int WJ, bool GATED, int D>
__global__ __launch_bounds__(64 * WI * WJ, 2) void k_tile(TileArgs a) {
  constexpr int NT = 64 * WI * WJ, TI = BI / WI / 16, TJ = BJ / WJ / 16;
  constexpr int OUT = GATED ? BJ / 2 : BJ;  // outputs of a tile row
  static_assert(!GATED || TJ % 4 == 0, "a gated run is 64 rows of one wavefront");
  typedef OperandTile<TA, BI, NT> A;
  typedef OperandTile<TB, BJ, NT> B;
  constexpr int kEpilogue = kEpilogueFloats<TJ>;
  __shared__ union {
    short stage[2][(BI + BJ) * kC];
    float sums[WI * WJ][kEpilogue];
  } mem;
  auto& lds = mem.stage;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wi = wave % WI * (BI / WI), wj = wave / WI * (BJ / WJ);
  const uint32_t b = blockIdx.y * gridDim.x + blockIdx.x;
  if (b >= a.workgroups) return;
  uint32_t ti, tj, split;
  tile_of(b, a.workgroups, a.tiles_i, a.tiles_j, ti, tj, split);
  const int64_t i0 = (int64_t)ti * BI, j0 = (int64_t)tj * OUT;
  const int64_t c0 = (int64_t)split * a.chunk, c1 = min(a.C, c0 + a.chunk);
  const int steps = (int)((c1 - c0 + kC - 1) / kC);

  // The thread's chunks of step 0.  Rows past an operand's end repeat its last
  // row: what they add up to is not written.  Across c a chunk that reaches past
  // the operand's edge is read as the row's last eight elements, `ea` or `eb`
  // places before its own, and moved when it is stored.
  const T *pa[A::kPer], *pb[B::kPer];
  int ca[A::kPer], cb[B::kPer];  // along c: the chunk's first element of the step; across: its row
  int ea[A::kPer], eb[B::kPer];
#pragma unroll
  for (int i = 0; i < A::kPer; ++i) {
    const int q = i * NT + tid, r = q / A::kRow, col = A::place(r, q % A::kRow) * 8;
    ca[i] = TA ? r : col;
    ea[i] = TA ? (int)max(i0 + col - (a.I - 8), (int64_t)0) : 0;
    pa[i] = (const T*)a.a + (TA ? (c0 + r) * a.lda + i0 + col - ea[i] : min(i0 + r, a.I - 1) * a.lda + c0 + col);
  }
#pragma unroll
  for (int i = 0; i < B::kPer; ++i) {
    const int q = i * NT + tid, r = q / B::kRow, col = B::place(r, q % B::kRow) * 8;
    cb[i] = TB ? r : col;
    eb[i] = TB ? (int)max(j0 + col - (a.J - 8), (int64_t)0) : 0;
    if constexpr (TB) {
      pb[i] = (const T*)a.b + (c0 + r) * a.ldb + j0 + col - eb[i];
    } else {
      const int64_t j = min(j0 + (GATED ? (r >> 6) * 32 + (r & 31) : r), a.J - 1);
      pb[i] = (const T*)a.b + (j + (GATED && (r >> 5 & 1) ? a.J : 0)) * a.ldb + c0 + col;
    }
  }
  // whole steps of rows of a chunk or more are loaded without a guard
  const bool wide = (!TA || a.I >= 8) && (!TB || a.J >= 8);
  const bool edge = (TA && i0 + BI > a.I) || (TB && j0 + BJ > a.J);
  auto whole = [&](int s) { return wide && c1 - c0 - (int64_t)s * kC >= kC; };
  u32x4 ra[D][A::kPer], rb[D][B::kPer];
  auto load = [&](u32x4 (&va)[A::kPer], u32x4 (&vb)[B::kPer], int s) {
    const int64_t c = (int64_t)s * kC, left = c1 - c0 - c;
    if (whole(s)) {
#pragma unroll
      for (int i = 0; i < A::kPer; ++i) va[i] = *(const u32x4_a2*)(pa[i] + (TA ? c * a.lda : c));
#pragma unroll
      for (int i = 0; i < B::kPer; ++i) vb[i] = *(const u32x4_a2*)(pb[i] + (TB ? c * a.ldb : c));
    } else if (left > 0) {
#pragma unroll
      for (int i = 0; i < A::kPer; ++i)
        va[i] = raw8(pa[i] + ea[i] + (TA ? c * a.lda : c), TA ? (ca[i] < left ? 8 - ea[i] : 0) : left - ca[i]);
#pragma unroll
      for (int i = 0; i < B::kPer; ++i)
        vb[i] = raw8(pb[i] + eb[i] + (TB ? c * a.ldb : c), TB ? (cb[i] < left ? 8 - eb[i] : 0) : left - cb[i]);
    }
  };
  auto stage = [&](const u32x4 (&va)[A::kPer], const u32x4 (&vb)[B::kPer], int s) {
    const bool move = edge && whole(s);
    auto put = [&](int place, u32x4 w, int by) {
      if (move) {  // (a chunk wholly past the edge holds anything)
        Raw<T> r = {w};
        MoveDown{by}(r);
        w = r.w;
      }
      *(u32x4*)(lds[s & 1] + place) = w;
    };
#pragma unroll
    for (int i = 0; i < A::kPer; ++i) put((i * NT + tid) * 8, va[i], ea[i]);
#pragma unroll
    for (int i = 0; i < B::kPer; ++i) put(BI * kC + (i * NT + tid) * 8, vb[i], eb[i]);
  };

  f32x4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int u = 0; u < D; ++u) load(ra[u], rb[u], u);
  if (steps > 0) {
    stage(ra[0], rb[0], 0);
    load(ra[0], rb[0], D);
  }
  __syncthreads();
  for (int s0 = 0; s0 < steps; s0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int s = s0 + d;
      if (s < steps) {
        const lds_short *la = (lds_short*)lds[s & 1], *lb = la + BI * kC;
#pragma unroll
        for (int kk = 0; kk < kC / 32; ++kk) {
          s16x8 fa[TI], fb[TJ];
#pragma unroll
          for (int i = 0; i < TI; ++i) fa[i] = A::fragment(la, i, kk, lane, wi);
#pragma unroll
          for (int j = 0; j < TJ; ++j) fb[j] = B::fragment(lb, j, kk, lane, wj);
#pragma unroll
          for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j) acc[i][j] = mfma(fb[j], fa[i], acc[i][j], T{});
        }
        if (s + 1 < steps) {
          stage(ra[(d + 1) % D], rb[(d + 1) % D], s + 1);
          load(ra[(d + 1) % D], rb[(d + 1) % D], s + 1 + D);
        }
        __syncthreads();
      }
    }
  }
  write_tile<T, GATED, TI, TJ>(a, acc, mem.sums[wave], i0 + wi, j0 + (GATED ? wj / 2 : wj), split, lane);
}

// One 16-byte chunk per lane from memory straight into LDS, the wavefront's 64
// chunks in lane order from `lds` on; chunks past the descriptor's range
// arrive as zeros.  In assembly because the compiler, which cannot tell the
// transposed reads of one stage from the stores to the other, waits for the
// loads in flight before it reads (dx, 8192 x 8192 x 4096: 535 us against 448).
// The instruction has no output register; its address and descriptor are read
// when it issues, its arrival is waited for by dma_wait.  s_nop covers the wait
// states after a write of m0 and after a vector write of the descriptor; nothing
// else in these kernels uses m0.
__device__ __forceinline__ void dma16(u32x4 range, lds_short* lds, int offset) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 4\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds"
      :
      : "s"((uint32_t)(uintptr_t)lds), "v"(offset), "s"(range)
      : "memory");
}

// wait until at most LEFT of this wavefront's loads are still on their way;
// they arrive in the order of their issue
template <int LEFT>
__device__ __forceinline__ void dma_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(LEFT) : "memory");
}

// descriptor of `bytes` bytes from p on, unformatted, checked byte by byte
__device__ __forceinline__ u32x4 range_of(const void* p, int64_t bytes) {
  const uint64_t at = (uint64_t)p;
  return u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, bytes < 0 ? 0u : (uint32_t)bytes, 0x00020000u};
}

// The same tile fed by direct loads into LDS, for operands whose 16-byte chunks
// are aligned and, along c, whole; no register holds a chunk on its way.  S
// stages are on their way or in use: while one is multiplied the S - 1 after it
// arrive.  A step waits for its own stage only, and its one barrier says both
// that every wavefront's part of the stage is there and that the stage before,
// whose place the next loads take, has been read.
// WK = 2: the two halves of a step's contraction go to two sets of wavefronts,
// whose sums are added at the end: a small tile's step is bound by the latency of
// one wavefront's reads and products, not by their number.
template <typename T, bool TA, bool TB, int BI, int BJ, int WI, int WJ, bool GATED, int S, int WK>
__global__ __launch_bounds__(64 * WI * WJ * WK, 2) void k_tile_dma(TileArgs a) {
  constexpr int NT = 64 * WI * WJ * WK, TI = BI / WI / 16, TJ = BJ / WJ / 16;
  constexpr int OUT = GATED ? BJ / 2 : BJ;
  static_assert(!GATED || TJ % 4 == 0, "a gated run is 64 rows of one wavefront");
  typedef OperandTile<TA, BI, NT> A;
  typedef OperandTile<TB, BJ, NT> B;
  constexpr int kStage = (BI + BJ) * kC, kLoads = A::kPer + B::kPer;
  static_assert((S - 1) * kLoads < 64, "loads in flight");
  constexpr int kEpilogue = kEpilogueFloats<TJ>;
  __shared__ union {
    short stage[S * kStage];
    struct {
      float sums[WI * WJ][kEpilogue];
      f32x4 halves[WK == 2 ? WI * WJ : 1][TI * TJ][64];
    };
  } mem;
  lds_short* const lds = (lds_short*)mem.stage;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int own = wave % (WI * WJ), half = wave / (WI * WJ);  // half: 0 where WK is 1
  const int wi = own % WI * (BI / WI), wj = own / WI * (BJ / WJ);
  const uint32_t b = blockIdx.y * gridDim.x + blockIdx.x;
  if (b >= a.workgroups) return;
  uint32_t ti, tj, split;
  tile_of(b, a.workgroups, a.tiles_i, a.tiles_j, ti, tj, split);
  const int64_t i0 = (int64_t)ti * BI, j0 = (int64_t)tj * OUT;
  const int64_t c0 = (int64_t)split * a.chunk, c1 = min(a.C, c0 + a.chunk);
  const int steps = (int)((c1 - c0 + kC - 1) / kC);
  const int64_t rows_a = min(a.I - i0, (int64_t)BI), rows_b = min(a.J - j0, (int64_t)OUT);

  // Byte offsets of the thread's chunks.  Along c they move by a step's bytes
  // and the ranges stay (a tile's rows span less than 2^31 bytes); across c the
  // ranges move and the offsets stay.
  int oa[A::kPer], ob[B::kPer];
  int ca[A::kPer], cb[B::kPer];  // along c: the chunk's first element in the step
#pragma unroll
  for (int i = 0; i < A::kPer; ++i) {
    const int q = i * NT + tid, r = q / A::kRow;
    ca[i] = A::place(r, q % A::kRow) * 8;
    oa[i] = (int)(r * a.lda + ca[i]) * 2;
  }
#pragma unroll
  for (int i = 0; i < B::kPer; ++i) {
    const int q = i * NT + tid, r = q / B::kRow;
    cb[i] = B::place(r, q % B::kRow) * 8;
    // gated, up rows lie J rows behind their gate's; a last tile's gate rows past J
    // are up rows then, whose sums are not written
    ob[i] = (int)(((GATED ? (r >> 6) * 32 + (r & 31) : r) + (GATED && (r >> 5 & 1) ? a.J : 0)) * a.ldb + cb[i]) * 2;
  }
  const T* pa = (const T*)a.a + (TA ? c0 * a.lda + i0 : i0 * a.lda + c0);
  const T* pb = (const T*)a.b + (TB ? c0 * a.ldb + j0 : j0 * a.ldb + c0);
  const int64_t whole = (c1 - c0 + 7) & ~(int64_t)7;  // a last chunk's filling is its row's own
  constexpr int kPast = 0x7FFFFFF0;  // an offset past every range
  // past the last step the ranges are empty, so every step issues as many loads
  auto stage = [&](lds_short* la, int s) {
    const int64_t left = c1 - c0 - (int64_t)s * kC;  // of the contraction, from this step on
    const bool tail = left < kC;
    if constexpr (TA) {
      // a range ends with whole words: an odd last column's word is its own row's
      const auto r = range_of(pa + (int64_t)s * kC * a.lda,
                              (((min(left, (int64_t)kC) - 1) * a.lda + (a.I - i0)) * 2 + 2) & ~(int64_t)3);
#pragma unroll
      for (int i = 0; i < A::kPer; ++i) dma16(r, la + (i * NT + wave * 64) * 8, oa[i]);
    } else {
      const auto r = range_of(pa, ((rows_a - 1) * a.lda + whole) * 2);
#pragma unroll
      for (int i = 0; i < A::kPer; ++i) {
        const int o = oa[i] + s * kC * 2;
        dma16(r, la + (i * NT + wave * 64) * 8, tail && ca[i] >= left ? kPast : o);
      }
    }
    lds_short* lb = la + BI * kC;
    if constexpr (TB) {
      const auto r = range_of(pb + (int64_t)s * kC * a.ldb,
                              (((min(left, (int64_t)kC) - 1) * a.ldb + (a.J - j0)) * 2 + 2) & ~(int64_t)3);
#pragma unroll
      for (int i = 0; i < B::kPer; ++i) dma16(r, lb + (i * NT + wave * 64) * 8, ob[i]);
    } else {
      const auto r = range_of(pb, ((rows_b - 1 + (GATED ? a.J : 0)) * a.ldb + whole) * 2);
#pragma unroll
      for (int i = 0; i < B::kPer; ++i) {
        const int o = ob[i] + s * kC * 2;
        dma16(r, lb + (i * NT + wave * 64) * 8, tail && cb[i] >= left ? kPast : o);
      }
    }
  };

  f32x4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // One step; `load` issues the loads of the step S - 1 ahead, behind this step's
  // first reads of LDS rather than before them (8192 x 8192 x 4096: 423 -> 399
  // us).  With both operands read across c the reads of the step's second half
  // are also spread over the products of its first (413 -> 393 us; along c that
  // costs as much, 399 -> 417).
  auto multiply = [&](const lds_short* la, auto load) {
    const lds_short* lb = la + BI * kC;
    static_assert(kC == 64, "two halves");
    s16x8 fa[2][TI], fb[2][TJ];
    auto read = [&](int kk) {
#pragma unroll
      for (int j = 0; j < TJ; ++j) fb[kk][j] = B::fragment(lb, j, kk, lane, wj);
#pragma unroll
      for (int i = 0; i < TI; ++i) fa[kk][i] = A::fragment(la, i, kk, lane, wi);
    };
    if constexpr (WK == 2) {
#pragma unroll
      for (int j = 0; j < TJ; ++j) fb[0][j] = B::fragment(lb, j, half, lane, wj);
#pragma unroll
      for (int i = 0; i < TI; ++i) fa[0][i] = A::fragment(la, i, half, lane, wi);
      load();
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = mfma(fb[0][j], fa[0][i], acc[i][j], T{});
      return;
    }
    read(0);
    load();
    if constexpr (TA && TB) read(1);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      if (kk == 1 && !(TA && TB)) read(1);
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = mfma(fb[kk][j], fa[kk][i], acc[i][j], T{});
    }
    if constexpr (TA && TB) {
#pragma unroll
      for (int q = 0; q < TI + TJ; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // a read of LDS,
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);  // two products
      }
    }
  };

#pragma unroll
  for (int u = 0; u < S - 1; ++u) stage(lds + u * kStage, u);
  for (int s = 0; s < steps; s += S) {
#pragma unroll
    for (int u = 0; u < S; ++u) {
      if (s + u < steps) {
        dma_wait<(S - 2) * kLoads>();
        __syncthreads();
        multiply(lds + u * kStage, [&] { stage(lds + (u + S - 1) % S * kStage, s + u + S - 1); });
      }
    }
  }
  // nothing may arrive in LDS that the epilogue uses, or after the workgroup has
  // left it
  dma_wait<0>();
  __syncthreads();
  if constexpr (WK == 2) {
    f32x4* const other = mem.halves[own][0] + lane;
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        if (half) other[(i * TJ + j) * 64] = acc[i][j];
    __syncthreads();
    if (half) return;
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] += other[(i * TJ + j) * 64];
  }
  write_tile<T, GATED, TI, TJ>(a, acc, mem.sums[own], i0 + wi, j0 + (GATED ? wj / 2 : wj), split, lane);
}

// whether every 16-byte chunk of both operands is aligned and, along c, whole or
// filled up with zeros, and within the loads' offsets
template <bool TA, bool TB>
bool chunked(const TileArgs& a, bool gated = false) {
  if (gated && (2 * a.J + 256) * a.ldb * 2 >= INT64_C(0x7FFFFFF0)) return false;  // 31-bit offsets in w
  return aligned(a.a, 16) && aligned(a.b, 16) && a.lda % 8 == 0 && a.ldb % 8 == 0 &&
         ((TA && TB) || a.C % 8 == 0 || a.padded);
}

// S: stages fed by direct loads, or, negative, steps loaded ahead through registers
template <typename T, bool TA, bool TB, int BI, int BJ, int WI, int WJ, bool GATED, int S, int WK = 1>
int launch_tile(TileArgs a, hipStream_t s) {
  const int64_t out = GATED ? BJ / 2 : BJ;
  const int64_t ti = (a.I + BI - 1) / BI, tj = (a.J + out - 1) / out;
  constexpr int NT = 64 * WI * WJ * WK;
  if (ti * tj == 0) return ECHO_SUCCESS;
  a.tiles_i = (uint32_t)ti;
  a.tiles_j = (uint32_t)tj;
  a.workgroups = a.tiles_i * a.tiles_j * a.splits;  // below 2^32 by ECHO_MAX_PRODUCT
  const TileGrid g = grid_of(a.workgroups, NT);
  const dim3 grid(g.x, g.y);
  if constexpr (S > 0) return launch(k_tile_dma<T, TA, TB, BI, BJ, WI, WJ, GATED, S, WK>, grid, dim3(NT), s, a);
  else return launch(k_tile<T, TA, TB, BI, BJ, WI, WJ, GATED, -S>, grid, dim3(NT), s, a);
}

}  // namespace

// The products, one source file each.
int tile_forward(const TileArgs& a, int32_t dtype, bool gated, int tile, hipStream_t s);
int tile_dx(const TileArgs& a, int32_t dtype, int tile, hipStream_t s);
int tile_dw(const TileArgs& a, int32_t dtype, int tile, hipStream_t s);
// the forward product of at most so many rows; from 17 on the 64 tile is as fast
// (4096 x 4096: 16 rows 12.5 us, 33 rows in a tile 12.6)
constexpr int64_t kFewRows = 16;
int rows_forward(const TileArgs& a, int32_t dtype, bool gated, hipStream_t s);

}  // namespace echo
