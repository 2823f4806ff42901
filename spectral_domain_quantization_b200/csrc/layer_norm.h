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
  int period, offset;      // rows of one shift, and the first row's (RowMode kPhase)
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
  int period, offset;
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

// Widest matrix whose rows stay in the registers of a cluster; wider rows are
// read from memory in every pass.
constexpr int kNormMaxCols = 32768;

void launch_norm_fwd(const NormFwdParams& p, int dtype, int num_sms, cudaStream_t s);
// One file per type of X; `narrow`: Y is bf16 too.
void norm_fwd_bf16(const NormFwdParams& p, int mode, bool save, bool narrow, int num_sms, cudaStream_t s);
void norm_fwd_f32(const NormFwdParams& p, int mode, bool save, int num_sms, cudaStream_t s);

// Rows of partial sums a backward call writes (1: the sums themselves).
int norm_bwd_parts(const NormBwdParams& p, int num_sms);
void launch_norm_bwd(const NormBwdParams& p, int parts, cudaStream_t s);
// out[c] = sum of part[0 .. parts)[c], for each of the two that is not NULL.
void launch_norm_reduce(const float* part_w, const float* part_b, int parts, int64_t part_ld, int cols, float* dw,
                        float* db, cudaStream_t s);

// One file per kind of X; `narrow`: every matrix is bf16.  Each launches, or
// (occupancy) returns how many CTAs or clusters run at once.
int norm_bwd_bf16(const NormBwdParams& p, int mode, bool narrow, int parts, bool occupancy, int num_sms,
                  cudaStream_t s);
int norm_bwd_f32(const NormBwdParams& p, int mode, bool narrow, int parts, bool occupancy, int num_sms,
                 cudaStream_t s);
int norm_bwd_act8(const NormBwdParams& p, int mode, bool narrow, int parts, bool occupancy, int num_sms,
                  cudaStream_t s);

}  // namespace metis
