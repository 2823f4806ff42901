// What the layer norm's forward and backward kernels share: how rows are spread
// over threads, and the sums over a row.
//
// A row is held in registers: by SPAN lanes of a warp (up to 1024 columns; 1536
// forward, and 1280 backward in units of 8), by the W warps of a CTA, 1024 columns
// each, or by a cluster of CTAs that take a slice of the columns each (sums meet in
// distributed shared memory).  Each thread has NV units of E consecutive columns
// (rows.cuh), the same columns in every row: 32 columns a thread, so what a row costs
// besides its elements (reductions, roots, addresses) is spread over many.  E is 8
// where every matrix is bf16 (16-byte words) and 4 where one is float32, so that a
// warp's words are contiguous.  The rows to come wait in a ring in shared memory, each
// warp's part in a ring of its own.
#pragma once

#include <atomic>
#include <type_traits>

#include "act8.cuh"
#include "dependent.cuh"
#include "layer_norm.h"
#include "pairs.cuh"
#include "rows.cuh"

namespace metis {

// How a kernel spreads rows: kLanes, the SPAN lanes of a warp hold a row, and a
// CTA of 128 threads takes 128 / SPAN of them; kCta, a CTA holds a row; kCluster;
// kTall, a CTA that fills an SM holds a row, for the widest that can.
enum NormShape { kLanes = 0, kCta = 1, kCluster = 2, kTall = 3 };

constexpr int kLaneThreads = 128;
constexpr int kWarpCols = 1024;        // columns of a warp of kCta and kCluster

// The columns and rows of one thread.
template <int SPAN, int NV, int E, int MODE, int SHAPE>
struct NormCols {
  static constexpr int kSpan = SPAN;
  static constexpr bool kMulti = SHAPE != kLanes;
  static constexpr bool kClustered = SHAPE == kCluster;
  static constexpr int kRows = kMulti ? 1 : kLaneThreads / SPAN;   // rows a CTA has at once
  static constexpr int kStride = SPAN * E;                         // columns between a thread's units
  static constexpr int kOwn = NV * E;
  static_assert(!kMulti || SPAN * kOwn == kWarpCols);
  int lo, hi;         // this CTA's columns
  int c0;             // this thread's first column (kPhase: may be outside)
  int shift;          // kPhase: columns that c0 is moved by
  int t;              // lane of the row's lanes in the warp
  int64_t row, step;  // first row, and from one to the next
  uint32_t all, any;  // kPhase: bit i, all or any of unit i's columns are the row's

  // kPhase: row r's first element is (offset + r ld) mod `width` elements behind a
  // period's begin; that of rows `period` apart is equal
  MDEV NormCols(int cols, int slice, int ctas, int64_t ld, int offset, int width) {
    t = static_cast<int>(threadIdx.x) % SPAN;
    const int64_t blocks = kClustered ? gridDim.x / ctas : gridDim.x;
    row = static_cast<int64_t>(kClustered ? blockIdx.x / ctas : blockIdx.x) * kRows + (kMulti ? 0 : threadIdx.x / SPAN);
    step = blocks * kRows;                // a multiple of the period
    shift = MODE == kPhase ? static_cast<int>((offset + row * ld) & (width - 1)) : 0;
    const int begin = (kClustered ? static_cast<int>(cluster_rank()) * slice : 0) - shift;
    c0 = begin + t * E + (kMulti ? static_cast<int>(threadIdx.x >> 5) * kWarpCols : 0);
    lo = max(begin, 0);
    hi = kClustered ? min(cols, begin + slice) : cols;
    all = any = 0u;
    if (MODE == kPhase) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (col(i) >= lo && col(i) + E <= hi) all |= 1u << i;
        if (col(i) < hi && col(i) + E > lo) any |= 1u << i;
      }
    }
  }
  MDEV int col(int i) const { return c0 + i * kStride; }
  MDEV int left(int i) const { return hi - col(i); }      // columns from unit i's first on
  MDEV bool some(int i) const { return MODE == kPhase ? (any >> i) & 1u : col(i) < hi; }
  MDEV bool whole(int i) const {
    return MODE == kPhase ? (all >> i) & 1u : col(i) < hi;
  }
  MDEV bool has(int i, int j) const { return col(i) + j < hi && (MODE != kPhase || col(i) + j >= lo); }
};

// No aligned word that holds elements of the row at `x` reaches over the matrix.
template <typename T>
MDEV bool row_inside(const T* x, int cols, const Span& s) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x);
  return a - 16 >= s.lo && a + cols * sizeof(T) + 16 <= s.hi;
}

// Per-column vector (weight or bias) into registers; `none` where it is absent.
template <int SPAN, int NV, int E, int MODE, int SHAPE>
MDEV void load_vector(const NormCols<SPAN, NV, E, MODE, SHAPE>& cs, const void* p, int dtype, float none, float* out) {
  if (!p) {
#pragma unroll
    for (int k = 0; k < NV * E; ++k) out[k] = none;
    return;
  }
  if constexpr (MODE == kAligned) {
    if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = cs.some(i) ? cs.col(i) : 0;     // (the columns are a multiple of E)
        if (dtype == METIS_BF16) {
          Unit<__nv_bfloat16, E> u;
          const uint2* q = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + c);
#pragma unroll
          for (int k = 0; k < E / 4; ++k) {
            const uint2 x = q[k];
            u.w[2 * k] = x.x;
            u.w[2 * k + 1] = x.y;
          }
          u.get(out + E * i);
        } else {
          const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + c);
#pragma unroll
          for (int k = 0; k < E / 4; ++k) {
            const float4 x = q[k];
            out[E * i + 4 * k] = x.x;
            out[E * i + 4 * k + 1] = x.y;
            out[E * i + 4 * k + 2] = x.z;
            out[E * i + 4 * k + 3] = x.w;
          }
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < E; ++j) out[E * i + j] = cs.has(i, j) ? load_any(p, dtype, cs.col(i) + j) : 0.f;
}

// kPhase with 32 lanes a row: the elements of a row's first and last unit that are
// partly outside it.  Lanes 0 to E - 1 of the warp that holds the first unit have
// one element of it each, lanes 16 to 16 + E - 1 of the one that holds the last; the
// units themselves read zero.  So a ragged end costs a lane one element a row, and
// no lane a mask.  (Rows of several to a warp are masked element by element.)
template <int SPAN, int MODE>
constexpr bool norm_edges = MODE == kPhase && SPAN == 32;

struct NormEdge {
  bool on;            // this lane has an element
  bool first, last;   // the warp has a part of a unit at the row's begin, at its end
  int first_owner, last_owner, last_unit;   // the lanes that hold them, and the last one's index there
  int unit, owner;    // this lane's element's unit and its lane,
  int elem, col;      // its place in the unit, and its column
  template <int SPAN, int NV, int E, int MODE, int SHAPE>
  MDEV explicit NormEdge(const NormCols<SPAN, NV, E, MODE, SHAPE>& cs) {
    // (rows of 32 lanes are longer than two units: none holds both ends)
    const int lane = threadIdx.x & 31, begin = cs.c0 - lane * E, end = cs.hi - begin;
    first = begin < 0 && -begin % E != 0;
    first_owner = max(-begin, 0) / E;
    last = end > 0 && end < SPAN * NV * E && end % E != 0;
    last_unit = end / (SPAN * E);
    last_owner = end / E % SPAN;
    const bool tail = lane >= 16;
    elem = lane & 15;
    unit = tail ? last_unit : 0;
    owner = tail ? last_owner : first_owner;
    col = begin + (unit * SPAN + owner) * E + elem;
    on = (tail ? last : first) && elem < E && col >= cs.lo && col < cs.hi;
  }
};

// Unit i of an output row of type TY at `p` (its first column's place).
template <typename TY, int SPAN, int NV, int E, int MODE, int SHAPE>
MDEV void store_row_unit(const NormCols<SPAN, NV, E, MODE, SHAPE>& cs, TY* p, const float* v, int i, bool active) {
  if constexpr (MODE == kAny) {
    if (active && cs.whole(i)) {
      if constexpr (sizeof(TY) == 2)
        *p = __float2bfloat16_rn(*v);
      else
        *p = *v;
    }
  } else {
    Unit<TY, E> u;
    u.put(v);
    if (active && cs.whole(i)) {
      u.store(p);
    } else if (MODE == kPhase && !norm_edges<SPAN, MODE> && active && cs.some(i)) {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (cs.has(i, j)) p[j] = u.elem(j);
    }
  }
}

// y: the row's place of column 0.
template <int SPAN, int NV, int E, int MODE, int SHAPE>
MDEV void store_row_unit_any(const NormCols<SPAN, NV, E, MODE, SHAPE>& cs, void* y, int dtype, const float* v, int i,
                             bool active) {
  if (dtype == METIS_BF16)
    store_row_unit(cs, static_cast<__nv_bfloat16*>(y) + cs.col(i), v, i, active);
  else
    store_row_unit(cs, static_cast<float*>(y) + cs.col(i), v, i, active);
}

// s / n for n's rounded reciprocal: one correction of the product (Markstein),
// correctly rounded as long as nothing overflows or underflows.
MDEV float divide(float s, float n, float inv) {
  const float q = s * inv;
  const float r = fmaf(fmaf(-q, n, s), inv, q);
  return fabsf(q) < 3e38f ? r : q;       // keeps infinities and NaN
}

// 1 / sqrt(a), the hardware's approximation and one Newton step.
MDEV float inv_sqrt(float a) {
  const float y = rsqrtf(a);
  const float e = fmaf(-a * y, y, 1.f);
  return fabsf(e) < 0.5f ? fmaf(0.5f * y, e, y) : y;   // a of 0, infinity or NaN: as it is
}

// Sums over a warp of two values at once: in the first step a lane passes on the
// one it does not keep.  Lanes 0 to 15 end with the sum of a, the others with b's.
MDEV float warp_sums2(float a, float b) {
  const bool hi = threadIdx.x & 16;
  float x = (hi ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, hi ? a : b, 16);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
  return x;
}

// Sum over groups of `span` (a power of two) adjacent lanes, in all of them.
template <int kSpan>
MDEV float span_sum(float x) {
#pragma unroll
  for (int off = kSpan / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
  return x;
}

// Sum over a CTA of 1024 threads, in all of them.
MDEV float cta_sum(float x, float* buf) {
  x = span_sum<32>(x);
  __syncthreads();                      // the last call's sums have been read
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  return span_sum<32>(buf[threadIdx.x & 31]);
}

// V floats of every warp of a row's CTA or cluster, exchanged through shared
// memory: put() (lanes that hold one), then sync().  Two buffers in turn: a buffer
// is written again only after every thread has passed the barrier that follows its
// last reading.
template <int V, int SHAPE>
struct Exchange {
  static constexpr int kMost = SHAPE == kCluster ? 64 : 16;    // warps of a row
  static constexpr int kFloats = SHAPE == kLanes ? 1 : 2 * V * kMost;
  float* buf;
  int warps;        // of a row
  int ctas;
  int phase = 0;
  MDEV Exchange(float* b, int n) : buf(b), warps(SHAPE == kCluster ? n * (blockDim.x >> 5) : blockDim.x >> 5), ctas(n) {}
  MDEV int mine() const {
    return static_cast<int>(threadIdx.x >> 5) +
           (SHAPE == kCluster ? static_cast<int>(cluster_rank()) * static_cast<int>(blockDim.x >> 5) : 0);
  }
  MDEV void put(int value, float x) {
    float* b = buf + phase * (V * kMost) + value * kMost + mine();
    if constexpr (SHAPE == kCluster) {
      // into every CTA of the cluster
      const uint32_t at = smem_u32(b);
      for (int r = 0; r < ctas; ++r)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_to_rank(at, static_cast<uint32_t>(r))), "f"(x)
                     : "memory");
    } else {
      *b = x;
    }
  }
  MDEV const float* sync() {
    const float* b = buf + phase * (V * kMost);
    phase ^= 1;
    if constexpr (SHAPE == kCluster)
      cluster_sync_all();
    else
      __syncthreads();
    return b;
  }
};

// CTAs (or clusters) of `rows` groups each, up to `blocks` but so many that the
// groups are a multiple of the rows' period.
inline int64_t norm_blocks(int64_t blocks, int rows, int period) {
  int64_t unit = 1;
  while ((unit * rows) % period) ++unit;
  return imax64(unit, blocks / unit * unit);
}

// What is known of a kernel: the CTAs of W warps that an SM holds, and on which
// devices its limit of dynamic shared memory has been raised (an attribute of the
// kernel on each device).
struct NormHeld {
  std::atomic<uint64_t> devices{0};
  std::atomic<int> per_sm[17]{};
  template <typename K>
  int get(K kernel, int warps, int smem, int most_smem) {
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (!(devices.load(std::memory_order_acquire) & bit)) {
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
      devices.fetch_or(bit, std::memory_order_release);
    }
    int n = per_sm[warps].load(std::memory_order_relaxed);
    if (n == 0) {
      if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, 32 * warps, smem) != cudaSuccess || n < 1) n = 1;
      per_sm[warps].store(n, std::memory_order_relaxed);
    }
    return n;
  }
};

// The launch of one kernel for `cols` columns, `most` warps to a CTA.
struct NormPlan {
  int ctas = 1, warps = kLaneThreads / 32, slice = 0;
  NormPlan(int shape, int cols, int most) {
    if (shape == kLanes) return;
    if (shape == kCluster) {
      ctas = cols <= 2 * most * kWarpCols ? 2 : 4;
      slice = ((cols + ctas - 1) / ctas + 31) / 32 * 32;
    }
    warps = ((shape == kCluster ? slice : cols) + kWarpCols - 1) / kWarpCols;
  }
};

// A matrix of a call, for the choice of the kernels' row mode.
struct RowsOf {
  const void* p;
  int64_t ld;
  int dtype;
};

// The mode for matrices that are read and written together, and for kPhase the
// rows' period and the first row's offset, in units of `width` elements.
inline int norm_mode(const RowsOf* m, int count, int64_t cols, bool phase_ok, int width, int* period, int* offset) {
  bool aligned = cols % 8 == 0, phase = phase_ok && cols + width - 1 <= kNormMaxCols;
  int64_t off0 = 0, ld0 = 0;
  for (int i = 0; i < count; ++i) {
    const int64_t es = m[i].dtype == METIS_BF16 ? 2 : 4;
    const uintptr_t a = reinterpret_cast<uintptr_t>(m[i].p);
    aligned = aligned && a % 16 == 0 && (m[i].ld * es) % 16 == 0;
    const int64_t off = static_cast<int64_t>((a / es) & (width - 1)), ld = m[i].ld & (width - 1);
    if (i == 0) {
      off0 = off;
      ld0 = ld;
    }
    phase = phase && off == off0 && ld == ld0;
  }
  *period = 1;
  *offset = static_cast<int>(off0);
  if (aligned) return kAligned;
  if (!phase) return kAny;
  while ((*period * ld0) & (width - 1)) *period *= 2;
  return kPhase;
}

}  // namespace metis
