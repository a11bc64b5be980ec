// fp8_host.h -- host helpers shared by the operators in 8-bit floating point.
#pragma once

#include "echo_fp8.h"
#include "host_checks.h"

namespace echo {

inline int64_t blocks_of(int64_t n) { return (n + ECHO_FP8_BLOCK - 1) / ECHO_FP8_BLOCK; }

// the pitch of `cols` codes that a descriptor's `ld` means, and its status
inline int code_pitch(int64_t ld, int64_t cols, int64_t& out) {
  out = ld ? ld : (cols + 15) / 16 * 16;
  if (ld != 0 && (ld < cols || ld > ECHO_MAX_PITCH)) return ECHO_ERR_SHAPE;
  return out % 16 ? ECHO_ERR_ALIGNMENT : ECHO_SUCCESS;
}

// bytes from a matrix's first element to its last
inline int64_t bytes_of(int64_t rows, int64_t cols, int64_t ld, int64_t size) {
  return rows == 0 || cols == 0 ? 0 : ((rows - 1) * ld + cols) * size;
}

// What echo_linear8 and echo_linear_backward8 check alike; ld_w, ld_r and ld_p are
// each call's own.
struct Shape8 {
  int64_t m, n, k, rows, ld_x, ld_w, ld_out;  // rows: of w
};

inline int check_shape8(const echo_linear8_desc* d, Shape8& g) {
  if (!d) return ECHO_ERR_INVALID_ARGUMENT;
  if (d->dtype != ECHO_BF16 && d->dtype != ECHO_F16) return ECHO_ERR_TYPE;
  if (d->act < ECHO_ACT_NONE || d->act > ECHO_ACT_SILU) return ECHO_ERR_TYPE;
  if (d->gated != 0 && d->gated != 1) return ECHO_ERR_TYPE;
  if (d->x_format != ECHO_E4M3 && d->x_format != ECHO_E5M2) return ECHO_ERR_TYPE;
  if (d->m < 0 || d->m > ECHO_MAX_ROWS || d->n < 0 || d->k < 0 || d->k > ECHO_MAX_PITCH ||
      d->n > ECHO_MAX_PITCH / (d->gated ? 2 : 1))
    return ECHO_ERR_SHAPE;
  g = {d->m, d->n, d->k, d->gated ? 2 * d->n : d->n, 0, 0, d->ld_out ? d->ld_out : d->n};
  if (g.m * g.k > ECHO_MAX_PRODUCT || g.m * g.rows > ECHO_MAX_PRODUCT) return ECHO_ERR_SHAPE;
  if (d->ld_out != 0 && (d->ld_out < g.n || d->ld_out > ECHO_MAX_PITCH)) return ECHO_ERR_SHAPE;
  return code_pitch(d->ld_x, g.k, g.ld_x);
}

// x (m rows of k, rows filled up with zeros to ld) of `dtype` from codes and scales
// in blocks of 1 x 128
int unpack_rows(const void* codes, int64_t ld_c, const float* scales, int32_t format, int64_t m, int64_t k, void* x,
                int64_t ld, int32_t dtype, hipStream_t s);

}  // namespace echo
