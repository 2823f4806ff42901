// C ABI: the layer norm (see include/metis.h for the contract).
#include "abi_common.h"
#include "abi_internal.h"
#include "layer_norm.h"

using namespace metis;

namespace {

metis_status check_vector(const void* v, int dtype) {
  if (!v) return METIS_OK;
  if (!valid_dtype(dtype)) return METIS_ERR_ARG;
  return reinterpret_cast<uintptr_t>(v) % dtype_size(dtype) ? METIS_ERR_ALIGN : METIS_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" metis_status metis_layer_norm_fwd(const void* X, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx,
                                             const void* weight, const void* bias, int32_t w_dtype, float eps,
                                             void* Y, int32_t y_dtype, int64_t ldy, float* mean, float* rstd,
                                             metis_act8_tensor* saved, void* stream) {
  METIS_TRY(check_any_dense(X, dtype, rows, cols, ldx));
  METIS_TRY(check_any_dense(Y, y_dtype, rows, cols, ldy));
  METIS_TRY(check_vector(weight, w_dtype));
  METIS_TRY(check_vector(bias, w_dtype));
  if (!(eps >= 0.f)) return METIS_ERR_ARG;
  if (!aligned4(mean) || !aligned4(rstd)) return METIS_ERR_ALIGN;
  if (saved) {
    METIS_TRY(check_act8(saved));
    if (saved->rows != rows || saved->cols != cols) return METIS_ERR_SHAPE;
  }
  if (!device_is_sm100()) return METIS_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (saved && cudaMemsetAsync(saved->amax, 0, METIS_ACT8_AMAX * sizeof(float), s) != cudaSuccess)
      return step_status("metis_layer_norm_fwd");
    return METIS_OK;
  }
  NormFwdParams p{};
  p.X = X;
  p.rows = rows;
  p.ldx = ldx;
  p.cols = static_cast<int>(cols);
  p.w = weight;
  p.b = bias;
  p.w_dtype = w_dtype;
  p.eps = eps;
  p.Y = Y;
  p.y_dtype = y_dtype;
  p.ldy = ldy;
  p.mean = mean;
  p.rstd = rstd;
  if (saved) p.save = act8_view(saved);
  launch_norm_fwd(p, dtype, device_sm_count(), s);
  return step_status("metis_layer_norm_fwd");
}

extern "C" metis_status metis_layer_norm_bwd(const void* dY, int32_t g_dtype, int64_t rows, int64_t cols, int64_t ldg,
                                             const void* X, int32_t x_dtype, int64_t ldx,
                                             const metis_act8_tensor* saved, const float* mean, const float* rstd,
                                             const void* weight, int32_t w_dtype, void* dX, int32_t dx_dtype,
                                             int64_t ldd, float* dweight, float* dbias, void* workspace,
                                             size_t* workspace_bytes, void* stream) {
  if (!workspace_bytes) return METIS_ERR_NULL;
  METIS_TRY(check_any_dense(dY, g_dtype, rows, cols, ldg));
  if (saved) {
    if (X) return METIS_ERR_ARG;
    METIS_TRY(check_act8(saved));
    if (saved->rows != rows || saved->cols != cols) return METIS_ERR_SHAPE;
  } else {
    METIS_TRY(check_any_dense(X, x_dtype, rows, cols, ldx));
  }
  if (rows > 0 && (!mean || !rstd)) return METIS_ERR_NULL;
  METIS_TRY(check_vector(weight, w_dtype));
  if (dX) METIS_TRY(check_any_dense(dX, dx_dtype, rows, cols, ldd));
  if (!dX && !dweight && !dbias && rows > 0) return METIS_ERR_NULL;
  if (!aligned4(mean) || !aligned4(rstd) || !aligned4(dweight) || !aligned4(dbias)) return METIS_ERR_ALIGN;
  NormBwdParams p{};
  p.dY = dY;
  p.g_dtype = g_dtype;
  p.rows = rows;
  p.ldg = ldg;
  p.cols = static_cast<int>(cols);
  p.X = saved ? nullptr : X;
  p.x_dtype = x_dtype;
  p.ldx = ldx;
  if (saved) p.saved = act8_view(saved);
  p.mean = mean;
  p.rstd = rstd;
  p.w = weight;
  p.w_dtype = w_dtype;
  p.inv_n = 1.f / static_cast<float>(cols);
  p.dX = dX;
  p.dx_dtype = dx_dtype;
  p.ldd = ldd;
  p.part_ld = (cols + 3) / 4 * 4;
  const int parts = rows > 0 ? norm_bwd_parts(p, device_sm_count()) : 1;
  Carver c(workspace);
  c.take<float>(1);
  float* pw = nullptr;
  float* pb = nullptr;
  if (parts > 1) {
    if (dweight) pw = c.take<float>(static_cast<size_t>(parts) * p.part_ld);
    if (dbias) pb = c.take<float>(static_cast<size_t>(parts) * p.part_ld);
  }
  if (!workspace) {
    *workspace_bytes = c.used;
    return METIS_OK;
  }
  if (*workspace_bytes < c.used || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return METIS_ERR_WORKSPACE;
  if (!device_is_sm100()) return METIS_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    const size_t n = static_cast<size_t>(cols) * sizeof(float);
    if ((dweight && cudaMemsetAsync(dweight, 0, n, s) != cudaSuccess) ||
        (dbias && cudaMemsetAsync(dbias, 0, n, s) != cudaSuccess))
      return step_status("metis_layer_norm_bwd");
    return METIS_OK;
  }
  p.part_w = parts > 1 ? pw : dweight;
  p.part_b = parts > 1 ? pb : dbias;
  launch_norm_bwd(p, parts, s);
  if (parts > 1 && (dweight || dbias))
    launch_norm_reduce(pw, pb, parts, p.part_ld, p.cols, dweight, dbias, s);
  return step_status("metis_layer_norm_bwd");
}
