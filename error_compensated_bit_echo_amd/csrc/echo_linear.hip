// echo_linear.hip -- matrix products with bias, activation and residual in the
// epilogue, and their gradients: the host side of echo_linear and
// echo_linear_backward (include/echo_layer.h) and the kernels beside the tile
// kernel of linear_tile.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "echo_layer.h"
#include "host_checks.h"
#include "linear_device.h"
#include "linear_tile.h"

using namespace echo;

namespace {

// ---- dp: the gradient of the sums before the activation ---------------------------
// One pass over dout and p that writes dp, rounded, for both products, and sums
// its columns in binary32 for the bias.  A thread holds 8 columns and walks
// down the rows of its workgroup's run; `wide` threads lie side by side, 256 /
// wide above each other.  Bound by HBM: 2 bytes in per dout and p element, 2 out.
// The products read dp in 16 bits because the matrix cores do; the sums and the
// bias's gradient stay in binary32.  That is the rounding a caller who keeps dp as a
// tensor has too.  dp in two 16-bit parts, its rounding and the rest, would leave
// dx and dw the one rounding of their own, at twice the products: 32768 x 768 x
// 1024 bf16, root-mean-square error of dx and dw 0.0023 -> 0.0017 for 67 + 75 us ->
// 104 + 116; 8192 x 1792 x 4096 f16, 0.00029 -> 0.00021 for 120 + 129 us -> 199 +
// 209.  Half's range is the caller's to mind, by the scale of dout (echo_layer.h).
struct SlopeArgs {
  const void *dout;
  const void* p;  // nullable: no activation, dp is a copy of dout
  void* dp;       // nullable: dp is dout itself; rows filled up with zeros to ld_dp
  float* part;    // nullable: [runs][columns of dp] sums
  int64_t m, n, ld_out, ld_dp, run;
  int32_t act, gated, wide;  // wide: 8, 16 or 32
};

// Two rows' loads are on their way at once, without a branch at whose end they
// would be waited for.  WHOLE: rows are whole vectors.  Otherwise a row's last
// vector is read as the row's last eight elements and moved down, and rows
// under a vector are read element by element.
template <typename T, bool GATED, bool WHOLE>
__global__ __launch_bounds__(256) void k_slope(SlopeArgs a) {
  __shared__ float lds[GATED ? 2 : 1][256 * 8 + 32 * 8];
  const int tx = threadIdx.x & (a.wide - 1), ty = threadIdx.x / a.wide, high = 256 / a.wide;
  const int64_t col = ((int64_t)blockIdx.x * a.wide + tx) * 8;
  const int64_t r0 = (int64_t)blockIdx.y * a.run, r1 = min(r0 + a.run, a.m);
  const int n = (int)min(a.n - col, (int64_t)9);  // 8 or less: the row's last vector
  const int64_t cols = GATED ? 2 * a.n : a.n;
  float sg[8], su[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sg[e] = su[e] = 0.f;
  auto row = [&](int64_t r, float (&d)[8], float (&p)[8], float (&u)[8]) {
    if (a.p)
      with_act(a.act, [&](auto act) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float v, slope;
          act_slope<decltype(act)::value>(p[e], v, slope);
          if (GATED) {
            p[e] = d[e] * v;
            d[e] *= u[e];
          }
          d[e] *= slope;
        }
      });
    if (a.dp) {
      T* dp = (T*)a.dp + r * a.ld_dp;
      store_n<false>(dp + col, n, d);
      if (GATED) store_n<false>(dp + a.n + col, n, p);
      if (n <= 8)
        for (int64_t c = cols; c < a.ld_dp; ++c) dp[c] = from_f32<T>(0.f);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sg[e] += d[e];
      if (GATED) su[e] += p[e];
    }
  };
  const int back = !WHOLE && n < 8 ? 8 - n : 0;
  if ((WHOLE || a.n >= 8) && n > 0) {
    for (int64_t r = r0 + ty; r < r1; r += 2 * high) {
      Raw<T> d[2], p[2], u[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // past the end the last row once more
        const int64_t at = min(r + k * high, r1 - 1);
        d[k] = fetch_at<true>((const T*)a.dout + at * a.ld_out + col - back);
        if (a.p) p[k] = fetch_at<true>((const T*)a.p + at * cols + col - back);
        if (GATED && a.p) u[k] = fetch_at<true>((const T*)a.p + at * cols + a.n + col - back);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (r + k * high >= r1) continue;
        float fd[8], fp[8], fu[8];
        if constexpr (!WHOLE) {
          MoveDown{back}(d[k]);
          if (a.p) MoveDown{back}(p[k]);
          if (GATED && a.p) MoveDown{back}(u[k]);
        }
        unpack_raw(d[k], fd);
        if (a.p) unpack_raw(p[k], fp);
        if (GATED && a.p) unpack_raw(u[k], fu);
        row(r + k * high, fd, fp, fu);
      }
    }
  } else if (n > 0) {
    for (int64_t r = r0 + ty; r < r1; r += high) {
      float d[8], p[8], u[8];
      load_n<true>((const T*)a.dout + r * a.ld_out + col, n, d);
      if (a.p) {
        load_n<true>((const T*)a.p + r * cols + col, n, p);
        if (GATED) load_n<true>((const T*)a.p + r * cols + a.n + col, n, u);
      }
      row(r, d, p, u);
    }
  }
  if (!a.part) return;
  const int pitch = a.wide * 8 + 8;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lds[0][ty * pitch + tx * 8 + e] = sg[e];
    if constexpr (GATED) lds[1][ty * pitch + tx * 8 + e] = su[e];
  }
  __syncthreads();
  const int64_t c = (int64_t)blockIdx.x * a.wide * 8 + threadIdx.x;
  if ((int)threadIdx.x < a.wide * 8 && c < a.n)
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h) {
      float s = lds[h][threadIdx.x];
      for (int k = 1; k < high; ++k) s += lds[h][k * pitch + threadIdx.x];
      a.part[(int64_t)blockIdx.y * cols + h * a.n + c] = s;
    }
}

// ---- rows of odd lengths ------------------------------------------------------------
// Copies of up to two operands whose rows are no whole number of 16-byte chunks,
// each row filled up with zeros, for the tiles fed by direct loads: the copy
// moves each operand twice, the tiles save a third of the product's time.
struct PackArgs {
  const void* src[2];
  void* dst[2];
  int64_t rows[2], ld[2];
  int64_t cols, pitch;  // pitch: cols rounded up to 8
};

// a wavefront to a row
template <typename T>
__global__ __launch_bounds__(kBlock) void k_pack(PackArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t rows = a.rows[0] + a.rows[1];
  for (int64_t t = (int64_t)blockIdx.x * kWavesPerBlock + (threadIdx.x >> 6); t < rows;
       t += (int64_t)gridDim.x * kWavesPerBlock) {
    const int k = t >= a.rows[0];
    const int64_t r = k ? t - a.rows[0] : t;
    const T* src = (const T*)a.src[k] + r * a.ld[k];
    T* dst = (T*)a.dst[k] + r * a.pitch;
    for (int64_t c = lane * 8; c < a.pitch; c += 512) *(u32x4*)(dst + c) = raw8(src + c, a.cols - c);
  }
}

// out[c] = sum over the runs of part[run][c], in a fixed order
struct RunSumArgs {
  const float* part;
  void* out;
  int64_t cols;
  uint32_t runs;
};

template <typename T>
__global__ __launch_bounds__(1024) void k_run_sum(RunSumArgs a) {
  __shared__ float lds[32][33];
  const uint32_t c = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c;
  float s = 0.f;
  if (col < a.cols)
    for (uint32_t r = k; r < a.runs; r += 4 * 32) {  // four loads on their way at once
      float v[4];
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) v[e] = r + e * 32 < a.runs ? a.part[(r + e * 32) * a.cols + col] : 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) s += v[e];
    }
  lds[k][c] = s;
  __syncthreads();
  if (k == 0 && col < a.cols) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += lds[i][c];
    ((T*)a.out)[col] = from_f32<T>(s);
  }
}

// ---- joining splits ---------------------------------------------------------------
// The splits' sums added in order, then the epilogue; 8 outputs to a thread.
template <typename T, bool GATED>
__global__ __launch_bounds__(kBlock) void k_join(TileArgs a) {
  const int64_t cols = GATED ? 2 * a.J : a.J, vectors = (a.J + 7) / 8;
  const int64_t plane = a.I * cols, items = a.I * vectors;
  for (int64_t t = (int64_t)blockIdx.x * kBlock + threadIdx.x; t < items; t += (int64_t)gridDim.x * kBlock) {
    const int64_t i = t / vectors, j = (t - i * vectors) * 8;
    const int n = (int)min(a.J - j, (int64_t)8);
    const float* p = a.part + i * cols + j;
    float g[8], u[8], f[8];
    load_n<true>(p, n, g);
    if (GATED) load_n<true>(p + a.J, n, u);
    for (uint32_t s = 1; s < a.splits; ++s) {
      p += plane;
      load_n<true>(p, n, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] += f[e];
      if (GATED) {
        load_n<true>(p + a.J, n, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] += f[e];
      }
    }
    finish<T, 8, GATED>(a, i, j, n, g, u);
  }
}

// ---- host side ---------------------------------------------------------------------

struct Geometry {
  int64_t m, n, k, rows, ld_x, ld_w, ld_out, ld_r;
};

int64_t span(int64_t rows, int64_t cols, int64_t ld) {
  return rows == 0 || cols == 0 ? 0 : ((rows - 1) * ld + cols) * 2;
}

int pitch(int64_t ld, int64_t cols, int64_t& out) {
  out = ld ? ld : cols;
  return ld != 0 && (ld < cols || ld > ECHO_MAX_PITCH) ? ECHO_ERR_SHAPE : ECHO_SUCCESS;
}

int check_desc(const echo_linear_desc* d, Geometry& g) {
  if (!d) return ECHO_ERR_INVALID_ARGUMENT;
  if (d->dtype != ECHO_BF16 && d->dtype != ECHO_F16) return ECHO_ERR_TYPE;
  if (d->act < ECHO_ACT_NONE || d->act > ECHO_ACT_SILU) return ECHO_ERR_TYPE;
  if (d->gated != 0 && d->gated != 1) return ECHO_ERR_TYPE;
  if (d->m < 0 || d->m > ECHO_MAX_ROWS || d->n < 0 || d->k < 0 || d->k > ECHO_MAX_PITCH ||
      d->n > ECHO_MAX_PITCH / (d->gated ? 2 : 1))
    return ECHO_ERR_SHAPE;
  g.m = d->m;
  g.n = d->n;
  g.k = d->k;
  g.rows = d->gated ? 2 * d->n : d->n;
  if (g.m * g.k > ECHO_MAX_PRODUCT || g.m * g.rows > ECHO_MAX_PRODUCT) return ECHO_ERR_SHAPE;
  if (pitch(d->ld_x, g.k, g.ld_x) || pitch(d->ld_w, g.k, g.ld_w) || pitch(d->ld_out, g.n, g.ld_out) ||
      pitch(d->ld_r, g.n, g.ld_r))
    return ECHO_ERR_SHAPE;
  return ECHO_SUCCESS;
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// partial sums of either kind of operands fit
int64_t part_bytes(int64_t I, int64_t cols, int64_t C) {
  const int64_t a = plan_tiles(I, cols, C, true).part_bytes, b = plan_tiles(I, cols, C, false).part_bytes;
  return round_up(a > b ? a : b, 16);
}

// Rows of odd lengths.  Their chunks are neither aligned nor whole, so either
// the tiles stage them through registers, or copies with whole rows are made
// first (one launch, and every copied byte read and written) for the tiles fed
// by direct loads; the estimates decide.
int64_t copy_bytes(int64_t rows, int64_t cols) { return round_up(rows * round_up(cols, 8) * 2, 16); }
double copy_us(int64_t bytes) { return 3.5 + (double)bytes * 2.0 / 4.5e6; }

bool copy_forward(const Geometry& g) {
  return g.k % 8 != 0 && plan_tiles(g.m, g.rows, g.k, true).us + copy_us(copy_bytes(g.m + g.rows, g.k)) <
                             plan_tiles(g.m, g.rows, g.k, false).us;
}

int run_pack(const Geometry& g, const void* x, void* px, const void* w, void* pw, int32_t dtype,
             hipStream_t s) {
  PackArgs a = {};
  a.src[0] = x;
  a.dst[0] = px;
  a.rows[0] = x ? g.m : 0;
  a.ld[0] = g.ld_x;
  a.src[1] = w;
  a.dst[1] = pw;
  a.rows[1] = w ? g.rows : 0;
  a.ld[1] = g.ld_w;
  a.cols = g.k;
  a.pitch = round_up(g.k, 8);
  const uint64_t rows = (uint64_t)(a.rows[0] + a.rows[1]);
  if (rows == 0 || a.cols == 0) return ECHO_SUCCESS;
  const dim3 grid(blocks_for(rows)), block(kBlock);
  return dtype == ECHO_BF16 ? launch(k_pack<bf16_t>, grid, block, s, a) : launch(k_pack<f16_t>, grid, block, s, a);
}

int64_t forward_bytes(const Geometry& g) {
  if (g.m <= kFewRows) return 0;
  const int64_t copies = copy_forward(g) ? copy_bytes(g.m, g.k) + copy_bytes(g.rows, g.k) : 0;
  return copies + part_bytes(g.m, g.rows, g.k);
}

template <bool GATED>
int run_join(const TileArgs& a, int32_t dtype, hipStream_t s) {
  const uint64_t items = (uint64_t)a.I * (uint64_t)((a.J + 7) / 8);
  const dim3 grid(blocks_for_items(items)), block(kBlock);
  return dtype == ECHO_BF16 ? launch(k_join<bf16_t, GATED>, grid, block, s, a)
                            : launch(k_join<f16_t, GATED>, grid, block, s, a);
}

template <typename T, bool GATED>
int run_slope(const SlopeArgs& a, dim3 grid, dim3 block, hipStream_t s) {
  return a.n % 8 ? launch(k_slope<T, GATED, false>, grid, block, s, a)
                 : launch(k_slope<T, GATED, true>, grid, block, s, a);
}

void apply(const Plan& p, void* part, TileArgs& a) {
  a.splits = (uint32_t)p.splits;
  a.chunk = p.chunk;
  a.part = p.splits > 1 ? (float*)part : nullptr;
}

// The backward pass's workspace: dp where it differs from dout, copies of dout,
// x and w with whole rows where those pay, the bias's partial sums, one row for
// each run of rows, and the splits' sums.
struct BackPlan {
  bool copies;
  int32_t wide;
  int64_t ld_dp, dp_bytes, x_bytes, w_bytes, run, runs, bias_bytes, split_bytes;
  int64_t bytes() const { return dp_bytes + x_bytes + w_bytes + bias_bytes + split_bytes; }
};

BackPlan plan_back(const echo_linear_desc* d, const Geometry& g) {
  BackPlan b = {};
  const bool slope = d->act != ECHO_ACT_NONE || d->gated;
  const bool odd_k = g.k % 8 != 0, odd_n = !slope && g.n % 8 != 0;
  if (odd_k || odd_n) {
    const double copied = plan_tiles(g.m, g.k, g.rows, true).us + plan_tiles(g.rows, g.k, g.m, true).us;
    const double staged = plan_tiles(g.m, g.k, g.rows, false).us + plan_tiles(g.rows, g.k, g.m, false).us;
    const double cost = (odd_k ? copy_us(copy_bytes(g.m + g.rows, g.k)) : 0.0) +
                        (odd_n ? copy_us(copy_bytes(g.m, g.n)) : 0.0);
    b.copies = copied + cost < staged;
  }
  if (b.copies && odd_k) {
    b.x_bytes = copy_bytes(g.m, g.k);
    b.w_bytes = copy_bytes(g.rows, g.k);
  }
  if (slope || (b.copies && odd_n)) {
    b.ld_dp = round_up(g.rows, 8);
    b.dp_bytes = round_up(g.m * b.ld_dp * 2, 16);
  }
  // the widest strip of columns that wastes the fewest threads
  b.wide = 32;
  for (const int wide : {16, 8})
    if (round_up(g.n, wide * 8) < round_up(g.n, b.wide * 8)) b.wide = wide;
  const int64_t strips = (g.n + b.wide * 8 - 1) / (b.wide * 8);
  const int64_t most = strips ? (2048 + strips - 1) / strips : 1;  // workgroups along the rows
  b.run = round_up(g.m > 0 ? (g.m + most - 1) / most : 1, 512 / b.wide);
  b.runs = (g.m + b.run - 1) / b.run;
  b.bias_bytes = round_up(b.runs * g.rows * 4, 16);
  const int64_t dx = part_bytes(g.m, g.k, g.rows), dw = part_bytes(g.rows, g.k, g.m);
  b.split_bytes = dx > dw ? dx : dw;  // one after the other on the stream
  return b;
}

}  // namespace

extern "C" {

int64_t echo_linear_workspace(const echo_linear_desc* d) {
  Geometry g;
  const int rc = check_desc(d, g);
  return rc ? rc : forward_bytes(g);
}

int echo_linear(const echo_linear_desc* d, const void* x, const void* w, const void* bias,
                const void* residual, void* out, void* p, void* workspace,
                int64_t workspace_bytes, echo_stream_t stream) {
  Geometry g;
  int rc = check_desc(d, g);
  if (rc) return rc;
  if (g.m == 0 || g.n == 0) return ECHO_SUCCESS;
  if (!out || (g.k > 0 && (!x || !w))) return ECHO_ERR_INVALID_ARGUMENT;
  const int64_t need = forward_bytes(g);
  if (need > 0) {
    if (!workspace) return ECHO_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return ECHO_ERR_WORKSPACE;
  }
  for (const void* q : {x, w, bias, residual, (const void*)out, (const void*)p})
    if (!aligned(q, 2)) return ECHO_ERR_ALIGNMENT;
  if (!aligned(workspace, 16)) return ECHO_ERR_ALIGNMENT;
  Aliases al;
  al.out(workspace, need);
  al.out(out, span(g.m, g.n, g.ld_out));
  al.out(p, g.m * g.rows * 2);
  al.in(x, span(g.m, g.k, g.ld_x));
  al.in(w, span(g.rows, g.k, g.ld_w));
  al.in(bias, g.rows * 2);
  al.in(residual, span(g.m, g.n, g.ld_r));
  al.allow_identical(out, residual);
  if (!al.ok()) return ECHO_ERR_ALIAS;
  TileArgs a = {};
  a.a = x;
  a.b = w;
  a.lda = g.ld_x;
  a.ldb = g.ld_w;
  a.I = g.m;
  a.J = g.n;
  a.C = g.k;
  a.out = out;
  a.ldo = g.ld_out;
  a.p = p;
  a.bias = bias;
  a.residual = residual;
  a.ldr = g.ld_r;
  a.act = d->act;
  const hipStream_t s = (hipStream_t)stream;
  if (g.m <= kFewRows) return rows_forward(a, d->dtype, d->gated != 0, s);
  char* ws = (char*)workspace;
  if (copy_forward(g)) {
    char* pw = ws + copy_bytes(g.m, g.k);
    rc = run_pack(g, x, ws, w, pw, d->dtype, s);
    if (rc) return rc;
    a.a = ws;
    a.b = pw;
    a.lda = a.ldb = round_up(g.k, 8);
    a.padded = 1;
    ws = pw + copy_bytes(g.rows, g.k);
  }
  const Plan plan = plan_tiles(g.m, g.rows, g.k, chunked<false, false>(a, d->gated != 0));
  apply(plan, ws, a);
  rc = tile_forward(a, d->dtype, d->gated != 0, plan.tile, s);
  if (rc || plan.splits == 1) return rc;
  return d->gated ? run_join<true>(a, d->dtype, s) : run_join<false>(a, d->dtype, s);
}

int64_t echo_linear_backward_workspace(const echo_linear_desc* d) {
  Geometry g;
  const int rc = check_desc(d, g);
  if (rc) return rc;
  const BackPlan b = plan_back(d, g);
  return b.bytes();
}

int echo_linear_backward(const echo_linear_desc* d, const void* dout, const void* x,
                         const void* w, const void* p, void* dx, void* dw, void* dbias,
                         void* workspace, int64_t workspace_bytes, echo_stream_t stream) {
  Geometry g;
  int rc = check_desc(d, g);
  if (rc) return rc;
  const bool slope = d->act != ECHO_ACT_NONE || d->gated;
  const bool some = g.m > 0 && g.n > 0;
  if (some && (dx || dw || dbias)) {
    if (!dout || (slope && !p)) return ECHO_ERR_INVALID_ARGUMENT;
    if (g.k > 0 && ((dx && !w) || (dw && !x))) return ECHO_ERR_INVALID_ARGUMENT;
  }
  const BackPlan b = plan_back(d, g);
  const int64_t need = b.bytes();
  if (need > 0) {
    if (!workspace) return ECHO_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return ECHO_ERR_WORKSPACE;
  }
  for (const void* q : {dout, x, w, p, (const void*)dx, (const void*)dw, (const void*)dbias})
    if (!aligned(q, 2)) return ECHO_ERR_ALIGNMENT;
  if (!aligned(workspace, 16)) return ECHO_ERR_ALIGNMENT;
  Aliases al;
  al.out(dx, g.m * g.k * 2);
  al.out(dw, g.rows * g.k * 2);
  al.out(dbias, g.rows * 2);
  al.out(workspace, need);
  al.in(dout, span(g.m, g.n, g.ld_out));
  al.in(x, span(g.m, g.k, g.ld_x));
  al.in(w, span(g.rows, g.k, g.ld_w));
  if (slope) al.in(p, g.m * g.rows * 2);
  if (!al.ok()) return ECHO_ERR_ALIAS;

  const hipStream_t s = (hipStream_t)stream;
  const bool bf16 = d->dtype == ECHO_BF16;
  char* const px = (char*)workspace + b.dp_bytes;
  char* const pw = px + b.x_bytes;
  float* const part = (float*)(pw + b.w_bytes);
  const bool own_dp = b.dp_bytes > 0, pack = b.x_bytes + b.w_bytes > 0;
  const bool want_dp = own_dp && (dx || dw);
  if (some && (want_dp || dbias)) {
    SlopeArgs a = {};
    a.dout = dout;
    a.p = slope ? p : nullptr;
    a.dp = want_dp ? workspace : nullptr;
    a.part = dbias ? part : nullptr;
    a.m = g.m;
    a.n = g.n;
    a.ld_out = g.ld_out;
    a.ld_dp = b.ld_dp;
    a.run = b.run;
    a.act = d->act;
    a.gated = d->gated;
    a.wide = b.wide;
    const dim3 grid((uint32_t)((g.n + b.wide * 8 - 1) / (b.wide * 8)), (uint32_t)b.runs), block(256);
    if (d->gated)
      rc = bf16 ? run_slope<bf16_t, true>(a, grid, block, s) : run_slope<f16_t, true>(a, grid, block, s);
    else
      rc = bf16 ? run_slope<bf16_t, false>(a, grid, block, s) : run_slope<f16_t, false>(a, grid, block, s);
    if (rc) return rc;
  }
  if (dbias && g.rows > 0) {
    RunSumArgs a = {part, dbias, g.rows, some ? (uint32_t)b.runs : 0};
    const dim3 grid((uint32_t)((g.rows + 31) / 32)), block(1024);
    rc = bf16 ? launch(k_run_sum<bf16_t>, grid, block, s, a) : launch(k_run_sum<f16_t>, grid, block, s, a);
    if (rc) return rc;
  }
  TileArgs a = {};
  a.a = own_dp ? workspace : dout;
  a.lda = own_dp ? b.ld_dp : g.ld_out;
  a.padded = own_dp;
  void* const splits = (char*)part + b.bias_bytes;
  if (pack && some) {
    rc = run_pack(g, dw ? x : nullptr, px, dx ? w : nullptr, pw, d->dtype, s);
    if (rc) return rc;
  }
  if (dx) {
    a.b = pack ? pw : w;
    a.ldb = pack ? round_up(g.k, 8) : g.ld_w;
    a.I = g.m;
    a.J = g.k;
    a.C = g.rows;
    a.out = dx;
    a.ldo = g.k;
    const Plan plan = plan_tiles(a.I, a.J, a.C, chunked<false, true>(a));
    apply(plan, splits, a);
    rc = tile_dx(a, d->dtype, plan.tile, s);
    if (!rc && plan.splits > 1) rc = run_join<false>(a, d->dtype, s);
    if (rc) return rc;
  }
  if (dw) {
    a.b = pack ? px : x;
    a.ldb = pack ? round_up(g.k, 8) : g.ld_x;
    a.I = g.rows;
    a.J = g.k;
    a.C = g.m;
    a.out = dw;
    a.ldo = g.k;
    const Plan plan = plan_tiles(a.I, a.J, a.C, chunked<true, true>(a));
    apply(plan, splits, a);
    rc = tile_dw(a, d->dtype, plan.tile, s);
    if (!rc && plan.splits > 1) rc = run_join<false>(a, d->dtype, s);
  }
  return rc;
}

}  // extern "C"
