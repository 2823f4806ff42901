// Layer norm, backward: the choice of kernel, the sum of the CTAs' partial
// sums, and rows wider than a cluster holds.
#include "layer_norm.cuh"

namespace metis {

namespace {

// out[c] = sum over the parts; 32 columns x 16 slices of the parts a CTA,
// blockIdx.y picks dweight or dbias.  592 parts of 4096 columns take 5.7 us (19 MB from L2,
// 256 CTAs that wait for it).
__global__ void __launch_bounds__(512) norm_reduce_kernel(const float* part_w, const float* part_b, int parts,
                                                          int64_t part_ld, int cols, float* dw, float* db) {
  __shared__ float acc[16][33];
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  float* out = blockIdx.y == 0 ? dw : db;
  wait_for_previous();
  if (!out) return;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + x;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int k = y; k < parts; k += 16) s += part[k * part_ld + c];
  }
  acc[y][x] = s;
  __syncthreads();
  if (y == 0 && c < cols) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += acc[k][x];
    out[c] = s;
  }
}

MDEV float wide_x(const NormBwdParams& p, int64_t row, int c) {
  if (p.X) return load_any(p.X, p.x_dtype, row * p.ldx + c);
  const uint32_t code = p.saved.codes[row * p.saved.ldc + c], sc = p.saved.scales[row * p.saved.blocks + (c >> 5)];
  return p.saved.fmt == METIS_MXINT8 ? act8_elem<METIS_MXINT8>(code) * act8_factor<METIS_MXINT8>(sc)
                                     : act8_elem<METIS_MXFP8>(code) * act8_factor<METIS_MXFP8>(sc);
}

// Rows wider than a cluster holds.  dw and db: a thread a column, over the rows
// y, y + gridDim.y, ...  (2000 x 40000 bf16: 729 us with the next kernel, 0.7 TB/s.)
__global__ void __launch_bounds__(256) norm_bwd_wide_cols_kernel(NormBwdParams p) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.cols) return;
  float aw = 0.f, ab = 0.f;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float dy = load_any(p.dY, p.g_dtype, row * p.ldg + c);
    aw = fmaf(dy, (wide_x(p, row, c) - p.mean[row]) * p.rstd[row], aw);
    ab += dy;
  }
  if (p.part_w) p.part_w[blockIdx.y * p.part_ld + c] = aw;
  if (p.part_b) p.part_b[blockIdx.y * p.part_ld + c] = ab;
}

// dx: a CTA a row, two passes over it.
__global__ void __launch_bounds__(1024) norm_bwd_wide_rows_kernel(NormBwdParams p) {
  __shared__ float buf[32];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float g = load_any(p.dY, p.g_dtype, row * p.ldg + c) * (p.w ? load_any(p.w, p.w_dtype, c) : 1.f);
      s1 = fmaf(g, (wide_x(p, row, c) - mean) * rstd, s1);
      s2 += g;
    }
    const float kd = -rstd * (rstd * (cta_sum(s1, buf) * p.inv_n)), k0 = -rstd * (cta_sum(s2, buf) * p.inv_n);
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float g = load_any(p.dY, p.g_dtype, row * p.ldg + c) * (p.w ? load_any(p.w, p.w_dtype, c) : 1.f);
      store_any(p.dX, p.dx_dtype, row * p.ldd + c, fmaf(g, rstd, fmaf(wide_x(p, row, c) - mean, kd, k0)));
    }
  }
}

int dispatch(const NormBwdParams& params, int parts, bool occupancy, int num_sms, cudaStream_t s) {
  NormBwdParams p = params;
  RowsOf m[3] = {{p.dY, p.ldg, p.g_dtype}};
  int count = 1;
  bool narrow = p.g_dtype == METIS_BF16;       // every matrix is bf16 (or 8 bits)
  if (p.X) {
    m[count++] = {p.X, p.ldx, p.x_dtype};
    narrow = narrow && p.x_dtype == METIS_BF16;
  }
  if (p.dX) {
    m[count++] = {p.dX, p.ldd, p.dx_dtype};
    narrow = narrow && p.dx_dtype == METIS_BF16;
  }
  // the 8-bit blocks are columns of the matrix: no shift
  const int mode = norm_mode(m, count, p.cols, p.X != nullptr, 8, &p.period, &p.offset);
  if (!p.X) return norm_bwd_act8(p, mode, narrow, parts, occupancy, num_sms, s);
  return p.x_dtype == METIS_BF16 ? norm_bwd_bf16(p, mode, narrow, parts, occupancy, num_sms, s)
                                 : norm_bwd_f32(p, mode, narrow, parts, occupancy, num_sms, s);
}

}  // namespace

int norm_bwd_parts(const NormBwdParams& p, int num_sms) {
  if (p.cols > kNormMaxCols) return static_cast<int>(imax64(1, imin64(p.rows, 16)));
  return dispatch(p, 0, true, num_sms, nullptr);
}

void launch_norm_bwd(const NormBwdParams& p, int parts, cudaStream_t s) {
  if (p.cols > kNormMaxCols) {
    // the column sums first: dX may be dY
    if (p.part_w || p.part_b)
      norm_bwd_wide_cols_kernel<<<dim3(static_cast<unsigned>((p.cols + 255) / 256), static_cast<unsigned>(parts)), 256,
                                  0, s>>>(p);
    if (p.dX) norm_bwd_wide_rows_kernel<<<static_cast<unsigned>(imin64(p.rows, 296)), 1024, 0, s>>>(p);
    return;
  }
  dispatch(p, parts, false, 0, s);
}

void launch_norm_reduce(const float* part_w, const float* part_b, int parts, int64_t part_ld, int cols, float* dw,
                        float* db, cudaStream_t s) {
  launch_dependent(norm_reduce_kernel, dim3(static_cast<unsigned>((cols + 31) / 32), 2), 512, 0, 1, s, part_w, part_b,
                   parts, part_ld, cols, dw, db);
}

}  // namespace metis
