// echo_linear8.hip -- the host side of echo_linear8 (include/echo_fp8.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "echo_fp8.h"
#include "fp8_host.h"
#include "host_checks.h"
#include "linear8_device.h"
#include "linear_join.h"

using namespace echo;

namespace echo {

int tile8_e4m3(const Tile8Args& a, int32_t dtype, bool gated, int tile, hipStream_t s);
int tile8_e5m2(const Tile8Args& a, int32_t dtype, bool gated, int tile, hipStream_t s);

}  // namespace echo

namespace {

int64_t workspace_of(const Shape8& g) { return g.m <= kFewRows ? 0 : plan_tiles8(g.m, g.rows, g.k).part_bytes; }

}  // namespace

extern "C" {

int64_t echo_linear8_workspace(const echo_linear8_desc* d) {
  Shape8 g;
  const int rc = check_shape8(d, g);
  return rc ? rc : workspace_of(g);
}

int echo_linear8(const echo_linear8_desc* d, const void* x, const float* sx, const void* w,
                 const float* sw, const void* bias, const void* residual, void* out, void* p,
                 void* workspace, int64_t workspace_bytes, echo_stream_t stream) {
  Shape8 g;
  int rc = check_shape8(d, g);
  if (!rc) rc = code_pitch(d->ld_w, g.k, g.ld_w);
  if (!rc && d->ld_r != 0 && (d->ld_r < g.n || d->ld_r > ECHO_MAX_PITCH)) rc = ECHO_ERR_SHAPE;
  if (rc) return rc;
  if (g.m == 0 || g.n == 0) return ECHO_SUCCESS;
  if (!out || (g.k > 0 && (!x || !sx || !w || !sw))) return ECHO_ERR_INVALID_ARGUMENT;
  const int64_t need = workspace_of(g), ld_r = d->ld_r ? d->ld_r : g.n;
  if (need > 0) {
    if (!workspace) return ECHO_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return ECHO_ERR_WORKSPACE;
  }
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(workspace, 16) || !aligned(sx, 4) || !aligned(sw, 4))
    return ECHO_ERR_ALIGNMENT;
  for (const void* q : {bias, residual, (const void*)out, (const void*)p})
    if (!aligned(q, 2)) return ECHO_ERR_ALIGNMENT;
  Aliases al;
  al.out(workspace, need);
  al.out(out, bytes_of(g.m, g.n, g.ld_out, 2));
  al.out(p, g.m * g.rows * 2);
  al.in(x, bytes_of(g.m, g.k, g.ld_x, 1));
  al.in(w, bytes_of(g.rows, g.k, g.ld_w, 1));
  al.in(sx, g.m * blocks_of(g.k) * 4);
  al.in(sw, (d->gated ? 2 : 1) * blocks_of(g.n) * blocks_of(g.k) * 4);
  al.in(bias, g.rows * 2);
  al.in(residual, bytes_of(g.m, g.n, ld_r, 2));
  al.allow_identical(out, residual);
  if (!al.ok()) return ECHO_ERR_ALIAS;
  Tile8Args a = {};
  a.a = x;
  a.b = w;
  a.sx = sx;
  a.sw = sw;
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
  a.ldr = ld_r;
  a.act = d->act;
  const hipStream_t s = (hipStream_t)stream;
  const bool gated = d->gated != 0;
  if (g.m <= kFewRows) return rows8_forward(a, d->dtype, d->x_format, gated, s);
  const Plan plan = plan_tiles8(g.m, g.rows, g.k);
  a.splits = (uint32_t)plan.splits;
  a.chunk = plan.chunk;
  a.part = plan.splits > 1 ? (float*)workspace : nullptr;
  a.wide = scales_in_fours(plan, g.k) && aligned(sx, 16) && aligned(sw, 16);
  rc = d->x_format == ECHO_E4M3 ? tile8_e4m3(a, d->dtype, gated, plan.tile, s)
                                : tile8_e5m2(a, d->dtype, gated, plan.tile, s);
  if (rc || plan.splits == 1) return rc;
  return gated ? run_join<true>(a, d->dtype, s) : run_join<false>(a, d->dtype, s);
}

}  // extern "C"
