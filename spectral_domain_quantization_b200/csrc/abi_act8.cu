// C ABI: activations kept in 8 bits (see include/metis.h for the contract).
#include <cstddef>

#include "abi_common.h"
#include "abi_internal.h"
#include "act8.h"

// The Python binding mirrors the struct field by field (ctypes).
static_assert(sizeof(metis_act8_tensor) == 48 && offsetof(metis_act8_tensor, rows) == 8 &&
                  offsetof(metis_act8_tensor, codes) == 24 && offsetof(metis_act8_tensor, amax) == 40,
              "metis_act8_tensor layout");

namespace metis {

metis_status check_act8(const metis_act8_tensor* t) {
  if (!t) return METIS_ERR_NULL;
  if (t->fmt != METIS_MXINT8 && t->fmt != METIS_MXFP8) return METIS_ERR_ARG;
  METIS_TRY(check_extent(t->rows, t->cols));
  if (!t->amax || (t->rows > 0 && (!t->codes || !t->scales))) return METIS_ERR_NULL;
  if (!aligned16(t->codes) || !aligned16(t->amax)) return METIS_ERR_ALIGN;
  return METIS_OK;
}

metis_status check_extent(int64_t rows, int64_t cols) {
  // columns are counted in 32 bits, and rows * (padded cols) stays far inside 63
  if (rows < 0 || cols <= 0 || rows > (int64_t{1} << 40) || cols > (int64_t{1} << 30) ||
      (rows > 0 && cols > (int64_t{1} << 50) / rows))
    return METIS_ERR_SHAPE;
  return METIS_OK;
}

metis_status check_any_dense(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld) {
  if (!valid_dtype(dtype)) return METIS_ERR_ARG;
  METIS_TRY(check_extent(rows, cols));
  if (ld < cols || (rows > 0 && ld > (int64_t{1} << 50) / rows)) return METIS_ERR_SHAPE;
  if (rows > 0 && !X) return METIS_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(X) % dtype_size(dtype)) return METIS_ERR_ALIGN;
  return METIS_OK;
}

}  // namespace metis

using namespace metis;

extern "C" {

size_t metis_act8_codes_bytes(int64_t rows, int64_t cols) {
  if (check_extent(rows, cols) != METIS_OK) return 0;
  return static_cast<size_t>(rows) * static_cast<size_t>(32 * act8_blocks(cols));
}

size_t metis_act8_scales_bytes(int64_t rows, int64_t cols) {
  if (check_extent(rows, cols) != METIS_OK) return 0;
  return static_cast<size_t>(rows) * static_cast<size_t>(act8_blocks(cols));
}

metis_status metis_act8_save(const void* X, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                             metis_act8_tensor* out, void* stream) {
  METIS_TRY(check_any_dense(X, dtype, rows, cols, ld));
  METIS_TRY(check_act8(out));
  if (out->rows != rows || out->cols != cols) return METIS_ERR_SHAPE;
  if (!device_is_sm100()) return METIS_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (cudaMemsetAsync(out->amax, 0, METIS_ACT8_AMAX * sizeof(float), s) != cudaSuccess)
      return step_status("metis_act8_save");
    return METIS_OK;
  }
  launch_act8_save(X, dtype, rows, cols, ld, act8_view(out), device_sm_count(), s);
  return step_status("metis_act8_save");
}

metis_status metis_act8_restore(const metis_act8_tensor* in, void* Y, int32_t dtype, int64_t ld, void* stream) {
  METIS_TRY(check_act8(in));
  METIS_TRY(check_any_dense(Y, dtype, in->rows, in->cols, ld));
  if (!device_is_sm100()) return METIS_ERR_UNSUPPORTED;
  if (in->rows == 0) return METIS_OK;
  launch_act8_restore(act8_view(in), in->rows, in->cols, Y, dtype, ld, device_sm_count(),
                      static_cast<cudaStream_t>(stream));
  return step_status("metis_act8_restore");
}

metis_status metis_act8_quantize_fp4(const metis_act8_tensor* in, int32_t block_axis, metis_fp4_tensor* out,
                                     void* stream) {
  METIS_TRY(check_act8(in));
  if (!out) return METIS_ERR_NULL;
  if (block_axis != 0 && block_axis != 1) return METIS_ERR_ARG;
  const int64_t outer = block_axis == 1 ? in->rows : in->cols;
  const int64_t inner = block_axis == 1 ? in->cols : in->rows;
  METIS_TRY(check_fp4(out, outer, inner, out->fmt));
  if (outer > (int64_t{1} << 36) || inner > (int64_t{1} << 36)) return METIS_ERR_SHAPE;   // tile counts in 32 bits
  if (out->inner_sum) return METIS_ERR_UNSUPPORTED;
  if (!device_is_sm100()) return METIS_ERR_UNSUPPORTED;
  launch_act8_quantize(act8_view(in), in->rows, in->cols, block_axis, out, device_sm_count(),
                       static_cast<cudaStream_t>(stream));
  return step_status("metis_act8_quantize_fp4");
}

}  // extern "C"
