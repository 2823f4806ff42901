// What the layer norm's forward and backward kernels share: how a row is spread
// over threads, its loads and stores, and the sums over a row.
//
// A row is held in registers by G threads: part of a warp, a warp, a CTA, or a
// cluster of CTAs that take a slice of the columns each (sums meet in
// distributed shared memory).  Each thread has NV units of 8 columns:
//   VEC == 8: 8 consecutive columns a unit (rows on 16-byte boundaries), so a
//             warp's loads and stores are 16 bytes a lane;
//   VEC == 1: the unit's columns G apart, one element a lane (rows that start
//             anywhere: a warp still touches contiguous bytes).
#pragma once

#include "act8.cuh"
#include "layer_norm.h"

namespace metis {

template <int G>
constexpr int norm_threads() {
  return G >= 128 ? G : 128;
}

MDEV float load_any(const void* p, int dtype, int64_t i) { return load_elem(p, dtype, i); }

MDEV void unpack8(const uint4& u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

MDEV uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

MDEV void store_any(void* p, int dtype, int64_t i, float v) {
  if (dtype == METIS_BF16)
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<float*>(p)[i] = v;
}

// 8 values to 8 consecutive elements; n < 8 of them where the row ends.
MDEV void store_unit(void* p, int dtype, int64_t i, const float* v, int n) {
  if (n >= 8) {
    if (dtype == METIS_BF16) {
      *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p) + i) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                     pack_bf16x2(v[6], v[7]));
    } else {
      float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
      d[0] = make_float4(v[0], v[1], v[2], v[3]);
      d[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) store_any(p, dtype, i + j, v[j]);
  }
}

// The columns of one thread.
template <int G, int NV, int VEC, bool CL>
struct NormCols {
  int begin, end;   // this CTA's columns
  int t;            // thread within the row's threads of this CTA
  MDEV NormCols(int cols, int slice) {
    t = static_cast<int>(threadIdx.x) % G;
    begin = CL ? static_cast<int>(cluster_rank()) * slice : 0;
    end = CL ? min(cols, begin + slice) : cols;
  }
  MDEV int col(int i, int j) const { return VEC == 8 ? begin + (i * G + t) * 8 + j : begin + (i * 8 + j) * G + t; }
  // how many of unit i's columns exist (VEC == 8)
  MDEV int left(int i) const { return end - (begin + (i * G + t) * 8); }
  MDEV bool has(int i, int j) const { return col(i, j) < end; }
};

// Per-column vector (weight or bias) into registers; `none` where it is absent.
template <int G, int NV, int VEC, bool CL>
MDEV void load_vector(const NormCols<G, NV, VEC, CL>& cs, const void* p, int dtype, float none, float* out) {
  if (!p) {
#pragma unroll
    for (int k = 0; k < NV * 8; ++k) out[k] = none;
    return;
  }
  const bool wide = VEC == 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (wide && cs.left(i) >= 8) {
      if (dtype == METIS_BF16) {
        unpack8(*reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p) + cs.col(i, 0)), out + 8 * i);
      } else {
        const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + cs.col(i, 0));
        const float4 a = q[0], b = q[1];
        out[8 * i] = a.x; out[8 * i + 1] = a.y; out[8 * i + 2] = a.z; out[8 * i + 3] = a.w;
        out[8 * i + 4] = b.x; out[8 * i + 5] = b.y; out[8 * i + 6] = b.z; out[8 * i + 7] = b.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) out[8 * i + j] = cs.has(i, j) ? load_any(p, dtype, cs.col(i, j)) : 0.f;
    }
  }
}

// One unit of a dense row, as loaded.
template <typename T, int VEC>
struct RawUnit;

template <>
struct RawUnit<__nv_bfloat16, 8> {
  uint4 q;
  MDEV void zero() { q = make_uint4(0, 0, 0, 0); }
  MDEV void load(const __nv_bfloat16* p, int n) {
    if (n >= 8) {
      q = *reinterpret_cast<const uint4*>(p);
    } else {
      zero();
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) w[j >> 1] |= static_cast<uint32_t>(__bfloat16_as_ushort(p[j])) << (16 * (j & 1));
      q = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  MDEV void get(float* v) const { unpack8(q, v); }
};

template <>
struct RawUnit<float, 8> {
  float4 a, b;
  MDEV void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  MDEV void load(const float* p, int n) {
    if (n >= 8) {
      a = *reinterpret_cast<const float4*>(p);
      b = *reinterpret_cast<const float4*>(p + 4);
    } else {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < n ? p[j] : 0.f;
      a = make_float4(v[0], v[1], v[2], v[3]);
      b = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
  MDEV void get(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

template <typename T>
struct RawUnit<T, 1> {
  T e[8];
  MDEV void zero() {
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = static_cast<T>(0.f);
  }
  MDEV void get(float* v) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = static_cast<float>(e[j]);
  }
};

// Unit i of the row at `p`.
template <typename T, int G, int NV, int VEC, bool CL>
MDEV void load_row_unit(const NormCols<G, NV, VEC, CL>& cs, const T* p, int i, bool active, RawUnit<T, VEC>& r) {
  if constexpr (VEC == 8) {
    const int n = cs.left(i);
    if (active && n > 0)
      r.load(p + cs.col(i, 0), n);
    else
      r.zero();
  } else {
    r.zero();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (active && cs.has(i, j)) r.e[j] = p[cs.col(i, j)];
  }
}

// Sums of two values over a row, the same in all its threads.  Two buffers in
// turn: a buffer is written again only after every thread has passed the
// barrier that follows its last reading.
template <int G, bool CL>
struct RowSum {
  static constexpr int kWarps = G / 32 > 0 ? G / 32 : 1;
  static constexpr int kEntries = CL ? 8 * kWarps : kWarps;
  float2* buf;      // shared memory, 2 * kEntries
  int phase = 0;
  int ctas;         // CTAs of the cluster
  MDEV RowSum(float2* b, int n) : buf(b), ctas(n) {}
  MDEV float2 operator()(float x, float y) {
    constexpr int kSpan = G < 32 ? G : 32;
#pragma unroll
    for (int off = kSpan / 2; off > 0; off >>= 1) {
      x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
      y += __shfl_xor_sync(0xFFFFFFFFu, y, off);
    }
    if constexpr (G <= 32) {
      return make_float2(x, y);
    } else {
      float2* b = buf + phase * kEntries;
      phase ^= 1;
      const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % kWarps;
      float2 s = make_float2(0.f, 0.f);
      if constexpr (CL) {
        // every warp writes its sums into every CTA of the cluster
        if (lane < ctas) {
          const uint32_t dst =
              map_to_rank(smem_u32(b + static_cast<int>(cluster_rank()) * kWarps + warp), static_cast<uint32_t>(lane));
          asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dst), "f"(x), "f"(y) : "memory");
        }
        cluster_sync_all();
        const int n = ctas * kWarps;
        for (int k = lane; k < n; k += 32) {
          s.x += b[k].x;
          s.y += b[k].y;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
          s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, off);
          s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, off);
        }
      } else {
        if (lane == 0) b[warp] = make_float2(x, y);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          s.x += b[k].x;
          s.y += b[k].y;
        }
      }
      return s;
    }
  }
};

// Grid-wide: which block of rows' groups this CTA (or cluster) is.
template <bool CL>
MDEV int64_t norm_block(int ctas) {
  return CL ? blockIdx.x / ctas : blockIdx.x;
}

inline int norm_cluster(int cols) { return cols <= 2 * 4096 ? 2 : (cols <= 4 * 4096 ? 4 : 8); }
inline int norm_slice(int cols, int ctas) { return ((cols + ctas - 1) / ctas + 31) / 32 * 32; }

// Launch `kernel` on `grid` CTAs, in clusters of `ctas` where that is not 1.
template <typename P>
void norm_launch(void (*kernel)(P, int), int grid, int threads, int ctas, const P& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  cudaLaunchKernelEx(&cfg, kernel, p, ctas);
}

template <typename K>
int norm_occupancy(K kernel, int threads) {
  int per_sm = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0) != cudaSuccess || per_sm < 1)
    per_sm = 1;
  return per_sm;
}

}  // namespace metis
