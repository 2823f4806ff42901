// Activations kept in 8 bits (act8.cu): views of a metis_act8_tensor and the
// launch interface.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/metis.h"

namespace metis {

// A metis_act8_tensor as the kernels take it.
struct Act8View {
  int fmt;             // METIS_MXINT8 / METIS_MXFP8
  int64_t ldc;         // bytes between rows of codes (32 blocks)
  int64_t blocks;      // blocks (scale bytes) per row
  uint8_t* codes;
  uint8_t* scales;
  float* amax;         // METIS_ACT8_AMAX floats
};

inline int64_t act8_blocks(int64_t cols) { return (cols + 31) / 32; }

inline Act8View act8_view(const metis_act8_tensor* t) {
  Act8View v{};
  v.fmt = t->fmt;
  v.blocks = act8_blocks(t->cols);
  v.ldc = 32 * v.blocks;
  v.codes = t->codes;
  v.scales = t->scales;
  v.amax = t->amax;
  return v;
}

// X (rows x cols, leading dimension ld) -> 8 bits, and back.
void launch_act8_save(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld, const Act8View& out,
                      int num_sms, cudaStream_t s);
void launch_act8_restore(const Act8View& in, int64_t rows, int64_t cols, void* Y, int dtype, int64_t ld, int num_sms,
                         cudaStream_t s);
// 8 bits -> FP4 along the columns (axis 1) or the rows (axis 0); writes every
// byte of out's scales, the padding included.
void launch_act8_quantize(const Act8View& in, int64_t rows, int64_t cols, int axis, const metis_fp4_tensor* out,
                          int num_sms, cudaStream_t s);

}  // namespace metis
