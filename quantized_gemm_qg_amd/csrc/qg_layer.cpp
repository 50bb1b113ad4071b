// C ABI of what stands around the products of a layer and behind the last one:
// the root-mean-square norm, the low-rank adapters and the cross entropy of a
// head.  Argument checks, workspaces and dispatch.
#include <algorithm>
#include <cmath>

#include "qg_internal.h"

using namespace qg;

// Checks of one matrix of 16-byte accesses: `el` bytes per element.
static qg_status matrix_check(const void *p, int64_t ld, int64_t columns, int el) {
  if (ld < columns) return QG_ERR_SHAPE;
  return aligned(p, 16) && ld * el % 16 == 0 ? QG_OK : QG_ERR_ALIGNMENT;
}
#define QG_TRY(check)                       \
  do {                                      \
    const qg_status st_ = (check);          \
    if (st_ != QG_OK) return st_;           \
  } while (0)

// Checks that the two directions of the norm share.
static qg_status norm_check(const void *weight, float eps, int64_t rows, int64_t k) {
  if (rows < 0 || k < 0 || !std::isfinite(eps) || !(eps > 0.f)) return QG_ERR_INVALID_ARGUMENT;
  if (k == 0 || k % 8 != 0) return QG_ERR_SHAPE;
  if (k > (1 << 24)) return QG_ERR_UNSUPPORTED;
  if (rows > 0 && !weight) return QG_ERR_INVALID_ARGUMENT;
  return aligned(weight, 16) ? QG_OK : QG_ERR_ALIGNMENT;
}

extern "C" qg_status qg_rmsnorm(const void *x, int32_t x_type, int64_t ldx, const void *residual, int32_t res_type,
                                int64_t ldr, void *sum, int64_t lds, const void *weight, float eps, int64_t rows,
                                int64_t k, void *y, int64_t ldy, int32_t q_type, void *q, int64_t ldq, void *q_scales,
                                hipStream_t stream) {
  QG_TRY(norm_check(weight, eps, rows, k));
  const bool added = residual || sum;
  if (!out_type(x_type) || (added && !out_type(res_type))) return QG_ERR_INVALID_ARGUMENT;
  if (q_type == QG_A_MXFP4) return QG_ERR_UNSUPPORTED;
  if (q_type != QG_A_BF16 && q_type != QG_A_INT8_TOKEN && q_type != QG_A_FP8_TOKEN && q_type != QG_A_FP8_BLOCK &&
      q_type != QG_A_MXFP8)
    return QG_ERR_INVALID_ARGUMENT;
  if (q_type == QG_A_MXFP8 && k % 32 != 0) return QG_ERR_SHAPE;
  if (rows > 0 && (!x || (!y && !q) || (q != nullptr) != (q_type != QG_A_BF16) || (q && !q_scales)))
    return QG_ERR_INVALID_ARGUMENT;
  QG_TRY(matrix_check(x, ldx, k, el_of(x_type)));
  if (residual) QG_TRY(matrix_check(residual, ldr, k, el_of(res_type)));
  if (sum) QG_TRY(matrix_check(sum, lds, k, el_of(res_type)));
  if (y) QG_TRY(matrix_check(y, ldy, k, 2));
  if (q) {
    if (ldq < k) return QG_ERR_SHAPE;
    if (!aligned(q, 8) || ldq % 8 != 0 || (q_type != QG_A_MXFP8 && !aligned(q_scales, 4))) return QG_ERR_ALIGNMENT;
  }
  if (rows == 0) return QG_OK;
  const NormArgs a{x, ldx, residual, ldr, sum, lds, weight, eps, rows, k, (uint16_t *)y, ldy, q_type, (uint8_t *)q, ldq, q_scales};
  return hip_status(launch_rmsnorm(a, x_type == QG_O_F32, !added ? 0 : res_type == QG_O_BF16 ? 1 : 2, stream));
}

extern "C" qg_status qg_rmsnorm_backward_workspace_size(int64_t rows, int64_t k, uint64_t *bytes) {
  if (!bytes || rows < 0 || k < 0) return QG_ERR_INVALID_ARGUMENT;
  *bytes = rows == 0 || k == 0 ? 0 : align_up((uint64_t)rmsnorm_back_parts(rows, k) * k * 4, 256);
  return QG_OK;
}

extern "C" qg_status qg_rmsnorm_backward(const void *s, int32_t s_type, int64_t lds, const void *weight, float eps,
                                         int64_t rows, int64_t k, const void *dy, int64_t lddy, const void *dsum,
                                         int64_t ldds, void *dx, int64_t lddx, void *dw, int32_t dw_type, void *ws,
                                         uint64_t ws_bytes, hipStream_t stream) {
  QG_TRY(norm_check(weight, eps, rows, k));
  if (!out_type(s_type) || (dw && !out_type(dw_type))) return QG_ERR_INVALID_ARGUMENT;
  if (rows > 0 && (!s || !dy)) return QG_ERR_INVALID_ARGUMENT;
  QG_TRY(matrix_check(s, lds, k, el_of(s_type)));
  QG_TRY(matrix_check(dy, lddy, k, 2));
  if (dsum) QG_TRY(matrix_check(dsum, ldds, k, el_of(s_type)));
  if (dx) QG_TRY(matrix_check(dx, lddx, k, el_of(s_type)));
  if (!aligned(dw, 16)) return QG_ERR_ALIGNMENT;
  if (!dw && (!dx || rows == 0)) return QG_OK;
  if (dw) {
    uint64_t need = 0;
    (void)qg_rmsnorm_backward_workspace_size(rows, k, &need);
    QG_TRY(ws_check(need, ws, ws_bytes));
  }
  const NormBackArgs a{s, lds, weight, eps, rows, k, (const uint16_t *)dy, lddy, dsum, ldds, dx, lddx, dw ? (float *)ws : nullptr};
  return hip_status(launch_rmsnorm_backward(a, s_type == QG_O_F32, dw, dw_type == QG_O_F32, stream));
}
