// Layer norm, backward, for rows held in registers.
//
//   xh = (x - mean) rstd, g = dy w
//   dx = rstd (g - sum(g)/n - xh sum(g xh)/n),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Bound by HBM: dy and x (2 or 4 bytes, or 1 + 1/32 from the 8-bit copy) are
// read once and dx written once.  A thread owns the same columns in every row it
// sees, so dw and db are running sums in its registers; a CTA's rows end as one
// row of partial sums, and a second kernel adds those in a fixed order.
#pragma once

#include "layer_norm.cuh"

namespace metis {

// x of one unit: dense, or 8 codes and the block's factor.
struct Act8Tag {};

template <typename TX, int VEC>
struct XUnit {
  RawUnit<TX, VEC> r;
  template <int G, int NV, bool CL>
  MDEV void load(const NormCols<G, NV, VEC, CL>& cs, const NormBwdParams& p, int64_t row, int i, bool active) {
    load_row_unit(cs, static_cast<const TX*>(p.X) + row * p.ldx, i, active, r);
  }
  MDEV void get(const NormBwdParams&, float* v) const { r.get(v); }
};

template <>
struct XUnit<Act8Tag, 8> {
  uint2 q;
  uint32_t sc;
  template <int G, int NV, bool CL>
  MDEV void load(const NormCols<G, NV, 8, CL>& cs, const NormBwdParams& p, int64_t row, int i, bool active) {
    q = make_uint2(0u, 0u);
    sc = 0u;
    if (active && cs.left(i) > 0) {
      const int c = cs.col(i, 0);
      q = *reinterpret_cast<const uint2*>(p.saved.codes + row * p.saved.ldc + c);
      sc = p.saved.scales[row * p.saved.blocks + (c >> 5)];
    }
  }
  MDEV void get(const NormBwdParams& p, float* v) const {
    float f;
    if (p.saved.fmt == METIS_MXINT8) {
      f = act8_factor<METIS_MXINT8>(sc);
      act8_elems4<METIS_MXINT8>(q.x, v);
      act8_elems4<METIS_MXINT8>(q.y, v + 4);
    } else {
      f = act8_factor<METIS_MXFP8>(sc);
      act8_elems4<METIS_MXFP8>(q.x, v);
      act8_elems4<METIS_MXFP8>(q.y, v + 4);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= f;
  }
};

template <>
struct XUnit<Act8Tag, 1> {
  float e[8];
  template <int G, int NV, bool CL>
  MDEV void load(const NormCols<G, NV, 1, CL>& cs, const NormBwdParams& p, int64_t row, int i, bool active) {
    uint32_t code[8], sc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      code[j] = sc[j] = 0u;
      if (active && cs.has(i, j)) {
        const int c = cs.col(i, j);
        code[j] = p.saved.codes[row * p.saved.ldc + c];
        sc[j] = p.saved.scales[row * p.saved.blocks + (c >> 5)];
      }
    }
    if (p.saved.fmt == METIS_MXINT8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = act8_elem<METIS_MXINT8>(code[j]) * act8_factor<METIS_MXINT8>(sc[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = act8_elem<METIS_MXFP8>(code[j]) * act8_factor<METIS_MXFP8>(sc[j]);
    }
  }
  MDEV void get(const NormBwdParams&, float* v) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e[j];
  }
};

template <typename TX, typename TG, int G, int NV, int VEC, bool CL>
__global__ void __launch_bounds__(norm_threads<G>(), G >= 256 ? 2 : 1) norm_bwd_kernel(NormBwdParams p, int ctas) {
  constexpr int kThreads = norm_threads<G>();
  constexpr int kRows = kThreads / G;
  constexpr int kOwn = NV * 8;
  __shared__ float2 sums[2 * RowSum<G, CL>::kEntries];
  __shared__ float gather[kRows > 1 ? kThreads * kOwn : 1];
  const NormCols<G, NV, VEC, CL> cs(p.cols, p.slice);
  RowSum<G, CL> row_sum(sums, ctas);
  const int g = static_cast<int>(threadIdx.x) / G;
  const int64_t blk = norm_block<CL>(ctas);
  const int64_t step = static_cast<int64_t>(CL ? gridDim.x / ctas : gridDim.x) * kRows;
  if constexpr (CL) cluster_sync_all();   // every CTA of the cluster runs before its shared memory is written
  float w[kOwn], aw[kOwn], ab[kOwn];
  load_vector(cs, p.w, p.w_dtype, 1.f, w);
#pragma unroll
  for (int k = 0; k < kOwn; ++k) aw[k] = ab[k] = 0.f;
  for (int64_t r0 = blk * kRows; r0 < p.rows; r0 += step) {
    const int64_t row = r0 + g;
    const bool active = row < p.rows;
    XUnit<TX, VEC> xr[NV];
    RawUnit<TG, VEC> gr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_row_unit(cs, static_cast<const TG*>(p.dY) + row * p.ldg, i, active, gr[i]);
      xr[i].load(cs, p, row, i, active);
    }
    const float mean = active ? p.mean[row] : 0.f, rstd = active ? p.rstd[row] : 0.f;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float x[8], dy[8];
      xr[i].get(p, x);
      gr[i].get(dy);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = 8 * i + j;
        const float xh = (x[j] - mean) * rstd, gk = dy[j] * w[k];
        s1 = fmaf(gk, xh, s1);
        s2 += gk;
        aw[k] = fmaf(dy[j], xh, aw[k]);
        ab[k] += dy[j];
      }
    }
    if (p.dX) {
      const float2 t = row_sum(s1, s2);
      const float c1 = t.x * p.inv_n, c2 = t.y * p.inv_n;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float x[8], dy[8];
        xr[i].get(p, x);
        gr[i].get(dy);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = (x[j] - mean) * rstd;
          dy[j] = rstd * (fmaf(-xh, c1, dy[j] * w[8 * i + j] - c2));
        }
        if constexpr (VEC == 8) {
          const int n = cs.left(i);
          if (active && n > 0) store_unit(p.dX, p.dx_dtype, row * p.ldd + cs.col(i, 0), dy, n);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (active && cs.has(i, j)) store_any(p.dX, p.dx_dtype, row * p.ldd + cs.col(i, j), dy[j]);
        }
      }
    }
  }
  // this CTA's partial sums
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* part = which == 0 ? p.part_w : p.part_b;
    if (!part) continue;
    part += blk * p.part_ld;
    const float* a = which == 0 ? aw : ab;
    if constexpr (kRows > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          gather[g * (G * kOwn) + cs.col(i, j)] = a[8 * i + j];
      __syncthreads();
      for (int c = threadIdx.x; c < p.cols; c += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kRows; ++k) s += gather[k * (G * kOwn) + c];
        part[c] = s;
      }
    } else {
      const bool wide = VEC == 8 && (reinterpret_cast<uintptr_t>(part) & 15u) == 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (wide && cs.left(i) >= 8) {
          float4* d = reinterpret_cast<float4*>(part + cs.col(i, 0));
          d[0] = make_float4(a[8 * i], a[8 * i + 1], a[8 * i + 2], a[8 * i + 3]);
          d[1] = make_float4(a[8 * i + 4], a[8 * i + 5], a[8 * i + 6], a[8 * i + 7]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (cs.has(i, j)) part[cs.col(i, j)] = a[8 * i + j];
        }
      }
    }
  }
}

// Launches, or (occupancy) returns the CTAs an SM holds times the rows a CTA
// has at once, as (rows << 16) | CTAs.
template <typename TX, typename TG, int G, int NV, int VEC, bool CL>
int norm_bwd_go(const NormBwdParams& p, int parts, bool occupancy, cudaStream_t s) {
  constexpr int kThreads = norm_threads<G>();
  auto* kernel = norm_bwd_kernel<TX, TG, G, NV, VEC, CL>;
  if (occupancy) {
    static const int per_sm = norm_occupancy(kernel, kThreads);
    return ((kThreads / G) << 16) | per_sm;
  }
  const int ctas = CL ? norm_cluster(p.cols) : 1;
  norm_launch(kernel, parts * ctas, kThreads, ctas, p, s);
  return 0;
}

inline bool norm_bwd_aligned(const NormBwdParams& p) {
  auto ok = [](const void* q, int64_t ld, int dt) {
    return (reinterpret_cast<uintptr_t>(q) & 15u) == 0 && (ld * (dt == METIS_BF16 ? 2 : 4)) % 16 == 0;
  };
  return ok(p.dY, p.ldg, p.g_dtype) && (!p.X || ok(p.X, p.ldx, p.x_dtype)) && (!p.dX || ok(p.dX, p.ldd, p.dx_dtype));
}

template <typename TX, typename TG, int VEC>
int norm_bwd_cols(const NormBwdParams& p, int parts, bool occ, cudaStream_t s) {
  if (VEC == 8 && p.cols <= 64) return norm_bwd_go<TX, TG, VEC == 8 ? 8 : 32, 1, VEC, false>(p, parts, occ, s);
  if (p.cols <= 256) return norm_bwd_go<TX, TG, 32, 1, VEC, false>(p, parts, occ, s);
  if (p.cols <= 1024) return norm_bwd_go<TX, TG, 32, 4, VEC, false>(p, parts, occ, s);
  if (p.cols <= 2048) return norm_bwd_go<TX, TG, 128, 2, VEC, false>(p, parts, occ, s);
  if (p.cols <= 4096) return norm_bwd_go<TX, TG, 256, 2, VEC, false>(p, parts, occ, s);
  return norm_bwd_go<TX, TG, 256, 2, VEC, true>(p, parts, occ, s);
}

template <typename TX>
int norm_bwd_kind(const NormBwdParams& p, int parts, bool occ, cudaStream_t s) {
  const bool al = norm_bwd_aligned(p);
  if (p.g_dtype == METIS_BF16)
    return al ? norm_bwd_cols<TX, __nv_bfloat16, 8>(p, parts, occ, s)
              : norm_bwd_cols<TX, __nv_bfloat16, 1>(p, parts, occ, s);
  return al ? norm_bwd_cols<TX, float, 8>(p, parts, occ, s) : norm_bwd_cols<TX, float, 1>(p, parts, occ, s);
}

}  // namespace metis
