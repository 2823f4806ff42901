// Layer norm, forward: the choice of kernel, and rows wider than a cluster holds.
#include "layer_norm_fwd.cuh"

namespace metis {

namespace {

// Three passes over the row in memory, an element a thread: 2000 x 40000 bf16 take 249
// us (1.3 TB/s of the one pass's bytes).
__global__ void __launch_bounds__(1024) norm_fwd_wide_kernel(NormFwdParams p, int dtype) {
  __shared__ float buf[32];
  const float n = static_cast<float>(p.cols);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t xr = row * p.ldx, yr = row * p.ldy;
    float s = 0.f, sq = 0.f, r = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += 1024) s += load_any(p.X, dtype, xr + c);
    const float m0 = __fdiv_rn(cta_sum(s, buf), n);
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float e = load_any(p.X, dtype, xr + c) - m0;
      sq = fmaf(e, e, sq);
      r += e;
    }
    sq = cta_sum(sq, buf);
    const float rest = sum_rest(m0, n, cta_sum(r, buf), sq);
    RowStats st;
    st.set(m0, __fdiv_rn(rest, n), fmaf(-rest, __fdiv_rn(rest, n), sq), __fdiv_rn(1.f, n), p.eps);
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = st.mean;
      if (p.rstd) p.rstd[row] = st.rstd;
    }
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float w = p.w ? load_any(p.w, p.w_dtype, c) : 1.f;
      const float b = p.b ? load_any(p.b, p.w_dtype, c) : 0.f;
      store_any(p.Y, p.y_dtype, yr + c, fmaf(fmaf(load_any(p.X, dtype, xr + c) - st.m0, st.rstd, st.off), w, b));
    }
  }
}

}  // namespace

void launch_norm_fwd(const NormFwdParams& params, int dtype, int num_sms, cudaStream_t s) {
  NormFwdParams p = params;
  bool save = p.save.codes != nullptr;
  if (p.cols > kNormMaxCols) {
    // the 8-bit copy first: Y may be X
    if (save) launch_act8_save(p.X, dtype, p.rows, p.cols, p.ldx, p.save, num_sms, s);
    const int grid = static_cast<int>(imin64(p.rows, 2 * num_sms));
    norm_fwd_wide_kernel<<<grid, 1024, 0, s>>>(p, dtype);
    return;
  }
  const RowsOf m[2] = {{p.X, p.ldx, dtype}, {p.Y, p.ldy, p.y_dtype}};
  const int mode = norm_mode(m, 2, p.cols, true, 8, &p.period, &p.offset);
  if (mode != kAligned && save) {
    // the 8-bit blocks are columns of the matrix and no lane has a whole word of
    // one: the copy is a kernel of its own (first, since Y may be X)
    launch_act8_save(p.X, dtype, p.rows, p.cols, p.ldx, p.save, num_sms, s);
    save = false;
  }
  const bool narrow = dtype == METIS_BF16 && p.y_dtype == METIS_BF16;
  if (dtype == METIS_BF16)
    norm_fwd_bf16(p, mode, save, narrow, num_sms, s);
  else
    norm_fwd_f32(p, mode, save, num_sms, s);
}

}  // namespace metis
