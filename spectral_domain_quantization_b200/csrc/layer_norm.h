// Launch interface of the layer norm kernels (layer_norm_fwd.cu,
// layer_norm_bwd*.cu).
#pragma once

#include "act8.h"

namespace metis {

struct NormFwdParams {
  const void* X;
  int64_t rows, ldx;
  int cols;
  int slice;               // columns of a CTA of the cluster (a multiple of 32)
  const void* w;           // optional
  const void* b;           // optional
  int w_dtype;
  float eps;
  void* Y;
  int y_dtype;
  int64_t ldy;
  float* mean;             // optional
  float* rstd;             // optional
  Act8View save;           // codes == NULL: not wanted
};

struct NormBwdParams {
  const void* dY;
  int g_dtype;
  int64_t rows, ldg;
  int cols;
  int slice;
  const void* X;           // or NULL and `saved`
  int x_dtype;
  int64_t ldx;
  Act8View saved;
  const float* mean;
  const float* rstd;
  const void* w;           // optional
  int w_dtype;
  float inv_n;
  void* dX;                // optional
  int dx_dtype;
  int64_t ldd;
  float* part_w;           // optional: [parts] rows of part_ld floats
  float* part_b;
  int64_t part_ld;
};

// Widest matrix whose rows stay in registers (8 CTAs of a cluster, 4096 columns
// each); wider rows are read from memory in every pass.
constexpr int kNormMaxCols = 8 * 4096;

void launch_norm_fwd(const NormFwdParams& p, int dtype, int num_sms, cudaStream_t s);

// Rows of partial sums a backward call writes (1: the sums themselves).
int norm_bwd_parts(const NormBwdParams& p, int num_sms);
void launch_norm_bwd(const NormBwdParams& p, int parts, cudaStream_t s);
// out[c] = sum of part[0 .. parts)[c], for each of the two that is not NULL.
void launch_norm_reduce(const float* part_w, const float* part_b, int parts, int64_t part_ld, int cols, float* dw,
                        float* db, cudaStream_t s);

// One file per kind of X (and, inside, type of dY): the register kernels.
// Each returns the CTAs an SM holds when `occupancy` is set, and launches otherwise.
int norm_bwd_bf16(const NormBwdParams& p, int parts, bool occupancy, cudaStream_t s);
int norm_bwd_f32(const NormBwdParams& p, int parts, bool occupancy, cudaStream_t s);
int norm_bwd_act8(const NormBwdParams& p, int parts, bool occupancy, cudaStream_t s);

}  // namespace metis
