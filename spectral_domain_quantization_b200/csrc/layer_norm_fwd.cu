// Layer norm, forward: y = (x - mean) rstd w + b over the columns of each row,
// optionally keeping x in 8 bits from the same pass.
//
// Bound by HBM: every element is read once and written once (and once more as
// 1 + 1/32 bytes with the 8-bit copy).  A row stays in registers between its
// three passes: the mean; the mean of the deviations and their squares (the
// first corrects the mean's rounding, the second gives the variance without
// cancellation); the output.  The grid is no larger than what is resident at
// once, so a thread loads its columns' weight and bias once for all its rows.
#include "layer_norm.cuh"

namespace metis {

namespace {

template <int FMT, int G, int NV, int VEC, bool CL>
MDEV void save_row(const NormCols<G, NV, VEC, CL>& cs, const Act8View& out, int slice, int64_t row, bool active,
                   const float* v, float& top) {
  const int pad_end = CL ? min(static_cast<int>(out.ldc), cs.begin + slice) : static_cast<int>(out.ldc);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (VEC == 8) {
      // a block of 32 columns in 4 adjacent lanes
      float a = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) a = max_nan(a, fabsf(v[8 * i + j]));
      a = max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
      a = max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
      const int c = cs.col(i, 0);
      if (active && c < pad_end) {
        float enc, q[8];
        const uint32_t sc = act8_scale<FMT>(a, enc);
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = v[8 * i + j] * enc;
        uint2 codes = act8_pack8<FMT>(q);
        if (sc == 255u) codes = make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(out.codes + row * out.ldc + c) = codes;
        if ((cs.t & 3) == 0) out.scales[row * out.blocks + (c >> 5)] = static_cast<uint8_t>(sc);
        top = fmaxf(top, act8_block_amax<FMT>(a, enc, sc));
      }
    } else {
      // a block of 32 columns in the 32 lanes of a warp
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = cs.col(i, j);
        const float x = v[8 * i + j];
        const float a = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x) & 0x7FFFFFFFu));
        if (active && c < pad_end) {
          float enc;
          const uint32_t sc = act8_scale<FMT>(a, enc);
          const uint32_t code = act8_code<FMT>(x * enc);
          out.codes[row * out.ldc + c] = static_cast<uint8_t>(sc == 255u ? 0u : code);
          if ((cs.t & 31) == 0) out.scales[row * out.blocks + (c >> 5)] = static_cast<uint8_t>(sc);
          top = fmaxf(top, act8_block_amax<FMT>(a, enc, sc));
        }
      }
    }
  }
}

template <typename T, int G, int NV, int VEC, bool SAVE, bool CL>
__global__ void __launch_bounds__(norm_threads<G>()) norm_fwd_kernel(NormFwdParams p, int ctas) {
  constexpr int kThreads = norm_threads<G>();
  constexpr int kRows = kThreads / G;     // rows a CTA has at once
  __shared__ float2 sums[2 * RowSum<G, CL>::kEntries];
  const NormCols<G, NV, VEC, CL> cs(p.cols, p.slice);
  RowSum<G, CL> row_sum(sums, ctas);
  const int g = static_cast<int>(threadIdx.x) / G;
  const int64_t step = static_cast<int64_t>(CL ? gridDim.x / ctas : gridDim.x) * kRows;
  const T* X = static_cast<const T*>(p.X);
  if constexpr (CL) cluster_sync_all();   // every CTA of the cluster runs before its shared memory is written
  float w[NV * 8], b[NV * 8];
  load_vector(cs, p.w, p.w_dtype, 1.f, w);
  load_vector(cs, p.b, p.w_dtype, 0.f, b);
  const float n = static_cast<float>(p.cols);
  float top = 0.f;
  // the loop's bound is the same for the whole CTA (and cluster)
  for (int64_t r0 = norm_block<CL>(ctas) * kRows; r0 < p.rows; r0 += step) {
    const int64_t row = r0 + g;
    const bool active = row < p.rows;
    RawUnit<T, VEC> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) load_row_unit(cs, X + row * p.ldx, i, active, raw[i]);
    float v[NV * 8];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      raw[i].get(v + 8 * i);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[8 * i + j];
    }
    const float m0 = __fdiv_rn(row_sum(s, 0.f).x, n);
    float ss = 0.f, sd = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (VEC == 8 && cs.left(i) >= 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = v[8 * i + j] - m0;
          ss = fmaf(d, d, ss);
          sd += d;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = cs.has(i, j) ? v[8 * i + j] - m0 : 0.f;
          ss = fmaf(d, d, ss);
          sd += d;
        }
      }
    }
    const float2 dev = row_sum(ss, sd);
    const float m1 = __fdiv_rn(dev.y, n);             // what the first mean is off
    float var = fmaf(-m1, m1, __fdiv_rn(dev.x, n));
    var = var < 0.f ? 0.f : var;                  // keeps a NaN
    const float rstd = __fdiv_rn(1.f, __fsqrt_rn(var + p.eps));
    if (active && cs.t == 0 && (!CL || cluster_rank() == 0)) {
      if (p.mean) p.mean[row] = m0 + m1;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = fmaf(((v[8 * i + j] - m0) - m1) * rstd, w[8 * i + j], b[8 * i + j]);
      if constexpr (VEC == 8) {
        const int left = cs.left(i);
        if (active && left > 0) store_unit(p.Y, p.y_dtype, row * p.ldy + cs.col(i, 0), y, left);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (active && cs.has(i, j)) store_any(p.Y, p.y_dtype, row * p.ldy + cs.col(i, j), y[j]);
      }
    }
    if constexpr (SAVE) {
      if (p.save.fmt == METIS_MXINT8)
        save_row<METIS_MXINT8>(cs, p.save, p.slice, row, active, v, top);
      else
        save_row<METIS_MXFP8>(cs, p.save, p.slice, row, active, v, top);
    }
  }
  if constexpr (SAVE) {
    __shared__ float wm[kThreads / 32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
    if ((threadIdx.x & 31) == 0) wm[threadIdx.x >> 5] = top;
    __syncthreads();
    top = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, wm[i]);
    act8_write_amax(p.save.amax, top);
  }
}

template <typename T, int G, int NV, int VEC, bool SAVE, bool CL>
void launch(const NormFwdParams& p, int num_sms, cudaStream_t s) {
  constexpr int kThreads = norm_threads<G>();
  auto* kernel = norm_fwd_kernel<T, G, NV, VEC, SAVE, CL>;
  static const int per_sm = norm_occupancy(kernel, kThreads);
  const int ctas = CL ? norm_cluster(p.cols) : 1;
  const int64_t rows = (p.rows + kThreads / G - 1) / (kThreads / G);
  const int64_t most = imin64(static_cast<int64_t>(num_sms) * per_sm, METIS_ACT8_AMAX) / ctas;
  norm_launch(kernel, static_cast<int>(imin64(rows, imax64(1, most))) * ctas, kThreads, ctas, p, s);
}

template <typename T, int VEC, bool SAVE>
void launch_cols(const NormFwdParams& p, int num_sms, cudaStream_t s) {
  if (VEC == 8 && p.cols <= 64)
    launch<T, VEC == 8 ? 8 : 32, 1, VEC, SAVE, false>(p, num_sms, s);
  else if (p.cols <= 256)
    launch<T, 32, 1, VEC, SAVE, false>(p, num_sms, s);
  else if (p.cols <= 1024)
    launch<T, 32, 4, VEC, SAVE, false>(p, num_sms, s);
  else if (p.cols <= 2048)
    launch<T, 128, 2, VEC, SAVE, false>(p, num_sms, s);
  else if (p.cols <= 4096)
    launch<T, 256, 2, VEC, SAVE, false>(p, num_sms, s);
  else
    launch<T, 256, 2, VEC, SAVE, true>(p, num_sms, s);
}

// Rows wider than a cluster holds: three passes over the row in memory.
__global__ void __launch_bounds__(1024) norm_fwd_wide_kernel(NormFwdParams p, int dtype) {
  __shared__ float2 sums[2 * RowSum<1024, false>::kEntries];
  RowSum<1024, false> row_sum(sums, 1);
  const float n = static_cast<float>(p.cols);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t x0 = row * p.ldx, y0 = row * p.ldy;
    float s = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += 1024) s += load_any(p.X, dtype, x0 + c);
    const float m0 = __fdiv_rn(row_sum(s, 0.f).x, n);
    float ss = 0.f, sd = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float d = load_any(p.X, dtype, x0 + c) - m0;
      ss = fmaf(d, d, ss);
      sd += d;
    }
    const float2 dev = row_sum(ss, sd);
    const float m1 = __fdiv_rn(dev.y, n);
    float var = fmaf(-m1, m1, __fdiv_rn(dev.x, n));
    var = var < 0.f ? 0.f : var;
    const float rstd = __fdiv_rn(1.f, __fsqrt_rn(var + p.eps));
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = m0 + m1;
      if (p.rstd) p.rstd[row] = rstd;
    }
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float w = p.w ? load_any(p.w, p.w_dtype, c) : 1.f;
      const float b = p.b ? load_any(p.b, p.w_dtype, c) : 0.f;
      store_any(p.Y, p.y_dtype, y0 + c, fmaf(((load_any(p.X, dtype, x0 + c) - m0) - m1) * rstd, w, b));
    }
  }
}

}  // namespace

void launch_norm_fwd(const NormFwdParams& params, int dtype, int num_sms, cudaStream_t s) {
  NormFwdParams p = params;
  const bool save = p.save.codes != nullptr;
  if (p.cols > kNormMaxCols) {
    // the 8-bit copy first: Y may be X
    if (save) launch_act8_save(p.X, dtype, p.rows, p.cols, p.ldx, p.save, num_sms, s);
    const int grid = static_cast<int>(imin64(p.rows, 2 * num_sms));
    norm_fwd_wide_kernel<<<grid, 1024, 0, s>>>(p, dtype);
    return;
  }
  if (p.cols > 4096) p.slice = norm_slice(p.cols, norm_cluster(p.cols));
  const bool wide = ((reinterpret_cast<uintptr_t>(p.X) | reinterpret_cast<uintptr_t>(p.Y)) & 15u) == 0 &&
                    (p.ldx * (dtype == METIS_BF16 ? 2 : 4)) % 16 == 0 &&
                    (p.ldy * (p.y_dtype == METIS_BF16 ? 2 : 4)) % 16 == 0;
  auto go = [&](auto vec, auto sv) {
    if (dtype == METIS_BF16)
      launch_cols<__nv_bfloat16, decltype(vec)::value, decltype(sv)::value>(p, num_sms, s);
    else
      launch_cols<float, decltype(vec)::value, decltype(sv)::value>(p, num_sms, s);
  };
  using one = std::integral_constant<int, 1>;
  using eight = std::integral_constant<int, 8>;
  if (wide)
    save ? go(eight{}, std::true_type{}) : go(eight{}, std::false_type{});
  else
    save ? go(one{}, std::true_type{}) : go(one{}, std::false_type{});
}

}  // namespace metis
