// echo_linear.hip -- matrix products with bias, activation and residual in the
// epilogue, and their gradients: the host side of echo_linear and
// echo_linear_backward (include/echo_layer.h) and the kernels beside the tile
// kernel of linear_tile.h.
#include <hip/hip_runtime.h>
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
// down the rows of its workgroup's run; 32 threads lie side by side, 8 above
// each other.  Bound by HBM: 2 bytes in per dout and p element, 2 out.
struct SlopeArgs {
  const void *dout, *p;
  void* dp;     // nullable: dp is dout itself
  float* part;  // nullable: [runs][columns of dp] sums
  int64_t m, n, ld_out, ld_dp, run;
  int32_t act, gated;
};

template <typename T>
__global__ __launch_bounds__(256) void k_slope(SlopeArgs a) {
  __shared__ float lds[2][8][256 + 8];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 256 + tx * 8;
  const int64_t r0 = (int64_t)blockIdx.y * a.run, r1 = min(r0 + a.run, a.m);
  const int n = (int)min(a.n - col, (int64_t)8);
  const int64_t cols = a.gated ? 2 * a.n : a.n;
  float sg[8], su[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sg[e] = su[e] = 0.f;
  if (n > 0)
    for (int64_t r = r0 + ty; r < r1; r += 8) {
      float d[8], p[8], u[8];
      load_n<false>((const T*)a.dout + r * a.ld_out + col, n, d);
      if (a.dp) {
        load_n<true>((const T*)a.p + r * cols + col, n, p);
        if (a.gated) load_n<true>((const T*)a.p + r * cols + a.n + col, n, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float v, slope;
          act_slope(p[e], a.act, v, slope);
          if (a.gated) {
            p[e] = d[e] * v;
            d[e] *= u[e];
          }
          d[e] *= slope;
        }
        store_n<false>((T*)a.dp + r * a.ld_dp + col, n, d);
        if (a.gated) store_n<false>((T*)a.dp + r * a.ld_dp + a.n + col, n, p);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sg[e] += d[e];
        if (a.gated) su[e] += p[e];
      }
    }
  if (!a.part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lds[0][ty][tx * 8 + e] = sg[e];
    if (a.gated) lds[1][ty][tx * 8 + e] = su[e];
  }
  __syncthreads();
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c < a.n)
    for (int h = 0; h <= a.gated; ++h) {
      float s = lds[h][0][threadIdx.x];
#pragma unroll
      for (int k = 1; k < 8; ++k) s += lds[h][k][threadIdx.x];
      a.part[(int64_t)blockIdx.y * cols + h * a.n + c] = s;
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
    for (uint32_t r = k; r < a.runs; r += 32) s += a.part[r * a.cols + col];
  lds[k][c] = s;
  __syncthreads();
  if (k == 0 && col < a.cols) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += lds[i][c];
    ((T*)a.out)[col] = from_f32<T>(s);
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
  if (pitch(d->ld_x, g.k, g.ld_x) || pitch(d->ld_w, g.k, g.ld_w) || pitch(d->ld_out, g.n, g.ld_out) ||
      pitch(d->ld_r, g.n, g.ld_r))
    return ECHO_ERR_SHAPE;
  return ECHO_SUCCESS;
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// The backward pass's workspace: dp where it differs from dout, and the bias's
// partial sums, one row for each run of rows.
struct BackPlan {
  int64_t ld_dp, dp_bytes, run, runs, part_bytes;
};

BackPlan plan_back(const echo_linear_desc* d, const Geometry& g) {
  BackPlan b = {};
  if (d->act != ECHO_ACT_NONE || d->gated) {
    b.ld_dp = round_up(g.rows, 8);
    b.dp_bytes = round_up(g.m * b.ld_dp * 2, 16);
  }
  const int64_t strips = (g.n + 255) / 256;
  const int64_t most = strips ? (2048 + strips - 1) / strips : 1;  // workgroups along the rows
  b.run = round_up((g.m + most - 1) / most, 8);
  if (b.run < 32) b.run = 32;
  b.runs = (g.m + b.run - 1) / b.run;
  b.part_bytes = round_up(b.runs * g.rows * 4, 16);
  return b;
}

int edge_of(int64_t I, int64_t cols) {
  // a larger tile reads less per output; a smaller one fills the 256 compute
  // units where there are few tiles
  for (int edge = 256; edge > 64; edge /= 2)
    if (((I + edge - 1) / edge) * ((cols + edge - 1) / edge) >= 192) return edge;
  return 64;
}

}  // namespace

extern "C" {

int64_t echo_linear_workspace(const echo_linear_desc* d) {
  Geometry g;
  const int rc = check_desc(d, g);
  return rc ? rc : 0;
}

int echo_linear(const echo_linear_desc* d, const void* x, const void* w, const void* bias,
                const void* residual, void* out, void* p, void* workspace,
                int64_t workspace_bytes, echo_stream_t stream) {
  Geometry g;
  int rc = check_desc(d, g);
  if (rc) return rc;
  if (g.m == 0 || g.n == 0) return ECHO_SUCCESS;
  if (!out || (g.k > 0 && (!x || !w))) return ECHO_ERR_INVALID_ARGUMENT;
  for (const void* q : {x, w, bias, residual, (const void*)out, (const void*)p})
    if (!aligned(q, 2)) return ECHO_ERR_ALIGNMENT;
  Aliases al;
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
  a.chunk = round_up(g.k, kC);
  a.splits = 1;
  a.out = out;
  a.ldo = g.ld_out;
  a.p = p;
  a.bias = bias;
  a.residual = residual;
  a.ldr = g.ld_r;
  a.act = d->act;
  return tile_forward(a, d->dtype, d->gated != 0, edge_of(g.m, g.rows), (hipStream_t)stream);
}

int64_t echo_linear_backward_workspace(const echo_linear_desc* d) {
  Geometry g;
  const int rc = check_desc(d, g);
  if (rc) return rc;
  const BackPlan b = plan_back(d, g);
  return b.dp_bytes + b.part_bytes;
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
  const int64_t need = b.dp_bytes + b.part_bytes;
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
  float* part = (float*)((char*)workspace + b.dp_bytes);
  const bool want_dp = slope && (dx || dw);
  if (some && (want_dp || dbias)) {
    SlopeArgs a = {};
    a.dout = dout;
    a.p = p;
    a.dp = slope ? workspace : nullptr;
    a.part = dbias ? part : nullptr;
    a.m = g.m;
    a.n = g.n;
    a.ld_out = g.ld_out;
    a.ld_dp = b.ld_dp;
    a.run = b.run;
    a.act = d->act;
    a.gated = d->gated;
    const dim3 grid((uint32_t)((g.n + 255) / 256), (uint32_t)b.runs), block(256);
    rc = bf16 ? launch(k_slope<bf16_t>, grid, block, s, a) : launch(k_slope<f16_t>, grid, block, s, a);
    if (rc) return rc;
  }
  if (dbias && g.rows > 0) {
    RunSumArgs a = {part, dbias, g.rows, some ? (uint32_t)b.runs : 0};
    const dim3 grid((uint32_t)((g.rows + 31) / 32)), block(1024);
    rc = bf16 ? launch(k_run_sum<bf16_t>, grid, block, s, a) : launch(k_run_sum<f16_t>, grid, block, s, a);
    if (rc) return rc;
  }
  TileArgs a = {};
  a.a = slope ? workspace : dout;
  a.lda = slope ? b.ld_dp : g.ld_out;
  a.splits = 1;
  if (dx) {
    a.b = w;
    a.ldb = g.ld_w;
    a.I = g.m;
    a.J = g.k;
    a.C = g.rows;
    a.chunk = round_up(a.C, kC);
    a.out = dx;
    a.ldo = g.k;
    rc = tile_dx(a, d->dtype, edge_of(a.I, a.J), s);
    if (rc) return rc;
  }
  if (dw) {
    a.b = x;
    a.ldb = g.ld_x;
    a.I = g.rows;
    a.J = g.k;
    a.C = g.m;
    a.chunk = round_up(a.C, kC);
    a.out = dw;
    a.ldo = g.k;
    rc = tile_dw(a, d->dtype, edge_of(a.I, a.J), s);
  }
  return rc;
}

}  // extern "C"
