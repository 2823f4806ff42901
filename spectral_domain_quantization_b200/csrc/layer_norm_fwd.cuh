// Layer norm, forward: y = (x - mean) rstd w + b over the columns of each row,
// optionally keeping x in 8 bits from the same pass (rows that lie aligned; others
// are copied by act8_save_kernel first: 16384 x 1027 bf16 39.1 us with the copy, of
// which the norm takes 20.4, 8192 x 4001 68.0 and 36.6).
//
// Bound by HBM: every element is read once and written once (and once more as
// 1 + 1/32 bytes with the 8-bit copy).  A warp sums its part of the row, then the
// squares of the deviations from its own mean; behind one barrier the warps' means
// and squares are joined (Chan, Golub and LeVeque's update), relative to the first
// warp's mean m0, so neither the variance nor the mean of a row far from zero is
// a difference of large sums.  The row's mean stays a pair m0 + m1.  The grid is
// no larger than what is resident at once, so a thread loads its columns' weight
// and bias once for all its rows.
//
// Measured, bf16 unless said: 16384 x 4096 44.9 us, 6.0 TB/s (a copy does 6.55); 8192 x
// 4096 24.5 us, float32 49.0 us, with the 8-bit copy 34.7 us (its arithmetic takes the
// issue slots); 65536 x 1024 48.6 us; 4000 x 14336 45 us; rows that start anywhere 65536
// x 1001 46.2 us, 8192 x 4001 36.6 us; matrices that lie differently 8192 x 4096 49.3 us;
// 8192 x 20000 285 us (a barrier of two CTAs a row).  The arithmetic goes two columns an
// instruction (pairs.cuh).
#pragma once

#include "layer_norm.cuh"

namespace metis {

// What the mean m of n float32 values lost, times n, from the sum r of their
// deviations and of the deviations' squares.  Far from zero (|m| over the standard
// deviation) the deviations are nearly exact, and r is the sum's rounding.  Near
// zero they carry a rounding that is the same for all values of a binade, and the
// sum itself is the better of the two.
MDEV float sum_rest(float m, float n, float r, float squares) { return m * m * n > squares ? r : 0.f; }

// The same of bf16 values with sum s: far from zero s is exact (8 bits a value, 24
// in the sum), and what is left is the division's remainder.
MDEV float division_rest(float m, float n, float s) { return fmaf(-m, n, s); }

// What a row ends with.
struct RowStats {
  float m0, off, rstd, mean;    // (x - mean) rstd = (x - m0) rstd + off
  MDEV void set(float first, float rest, float squares, float inv_n, float eps) {
    const float v = squares < 0.f ? 0.f : squares;      // keeps a NaN
    m0 = first;
    rstd = inv_sqrt(fmaf(v, inv_n, eps));
    off = -rest * rstd;
    mean = first + rest;
  }
};

// Warps of a CTA at most.  One element at a time takes more registers than 16 warps
// have, so with kAny those are left to the rows that 12 do not hold (kTall): 8192 x
// 4096 bf16 takes 51.3 us with 12 at most against 61.7 with 16, 4000 x 14336 takes 105
// with 16 against 193 in a cluster.
template <int MODE, int SHAPE>
constexpr int fwd_warps = MODE == kAny && SHAPE != kTall ? 12 : 16;

// CTAs an SM is to hold at least (0: what the compiler makes of it).  One element at a
// time takes 208 registers otherwise: 65536 x 1001 bf16, rows 1002 apart, 84.9 us against
// 105.9.
template <int SPAN, int OWN, int MODE, int SHAPE>
constexpr int fwd_ctas = SHAPE == kLanes && SPAN == 32 && OWN <= 32 && MODE == kAny ? 3 : 0;

// Bytes of a warp's part of a row in the ring.
template <typename T, int SPAN, int NV, int E, int MODE>
struct FwdStage {
  static constexpr int kBytes = NV * UnitSlot<T, E, MODE, 32>::kBytes;
};
template <typename T, int SPAN, int NV>
struct FwdStage<T, SPAN, NV, 1, kAny> {
  static constexpr int kBytes = RowImage<T, SPAN, NV>::kBytes;
};

template <typename T, int SPAN, int NV, int E, int S, int MODE, bool SAVE, int SHAPE>
__global__ void __launch_bounds__(SHAPE == kLanes ? kLaneThreads : 32 * fwd_warps<MODE, SHAPE>,
                                  fwd_ctas<SPAN, NV * E, MODE, SHAPE>)
    norm_fwd_kernel(NormFwdParams p, int ctas) {
  using Cols = NormCols<SPAN, NV, E, MODE, SHAPE>;
  using Slot = UnitSlot<T, E, MODE, 32>;
  using Image = RowImage<T, SPAN, NV>;            // kAny
  constexpr bool kRest = sizeof(T) == 4, CL = Cols::kClustered, kMulti = Cols::kMulti;
  constexpr bool kEdges = norm_edges<SPAN, MODE>;
  constexpr int kOwn = NV * E, G = E == 1 ? 2 : E, kGroups = kOwn / G;   // columns that are worked on together
  constexpr int kSpan = SPAN, kStage = FwdStage<T, SPAN, NV, E, MODE>::kBytes;
  static_assert(!SAVE || MODE == kAligned);
  using Ex = Exchange<kRest ? 3 : 2, SHAPE>;
  constexpr int kMost = Ex::kMost;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float parts[Ex::kFloats];
  const Cols cs(p.cols, p.slice, ctas, p.ldx, p.offset, 8);
  Ex ex(parts, ctas);
  const int lane = threadIdx.x & 31;
  const T* X = static_cast<const T*>(p.X);
  const Span span = span_of<T>(p.X, p.rows, p.cols, p.ldx);
  const uint32_t ring0 = smem_u32(ring) + (threadIdx.x >> 5) * (S * kStage);

  // row `fetch_row` into the stage at `into`
  int64_t fetch_row = cs.row;
  uint32_t into = ring0;
  auto fetch = [&] {
    const bool on = fetch_row < p.rows;
    if (SPAN < 32 || on) {
      const T* x = X + fetch_row * p.ldx;
      const bool inside = MODE == kPhase && on && row_inside(x, p.cols, span);
      if constexpr (MODE == kAny) {
        Image::start(into, lane, x + cs.col(0) - cs.t, on ? cs.left(0) + cs.t : 0, span);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          Slot::start(into + i * Slot::kBytes, lane, x + cs.col(i), on && cs.whole(i), on && cs.some(i), inside, span);
      }
    }
    cp_async_commit();
    fetch_row += cs.step;
    into = into + kStage == ring0 + S * kStage ? ring0 : into + kStage;
  };
  wait_for_previous();
#pragma unroll
  for (int k = 0; k < S - 1; ++k) fetch();
  f32x2 w[kOwn / 2], b[kOwn / 2];
  {
    float v[kOwn];
    load_vector(cs, p.w, p.w_dtype, 1.f, v);
#pragma unroll
    for (int k = 0; k < kOwn / 2; ++k) w[k] = pair(v[2 * k], v[2 * k + 1]);
    load_vector(cs, p.b, p.w_dtype, 0.f, v);
#pragma unroll
    for (int k = 0; k < kOwn / 2; ++k) b[k] = pair(v[2 * k], v[2 * k + 1]);
  }
  // columns of a warp of the row, as the exchange numbers them
  auto columns_of = [&](int warp) {
    if constexpr (!kMulti) return static_cast<float>(p.cols);
    const int per = blockDim.x >> 5;
    const int b0 = (CL ? warp / per * p.slice : 0) - cs.shift, at = b0 + (CL ? warp % per : warp) * kWarpCols;
    return static_cast<float>(max(min(CL ? min(p.cols, b0 + p.slice) : p.cols, at + kWarpCols) - max(at, 0), 0));
  };
  const float n_w = columns_of(kMulti ? ex.mine() : 0);
  const float inv_w = n_w > 0.f ? __fdiv_rn(1.f, n_w) : 0.f;
  const float inv_n = __fdiv_rn(1.f, static_cast<float>(p.cols));
  const float lane_n = kMulti && lane < ex.warps ? columns_of(lane) : 0.f;
  const float inv_lane = lane_n > 0.f ? __fdiv_rn(1.f, lane_n) : 0.f;
  const float n_0 = columns_of(0), inv_0 = __fdiv_rn(1.f, n_0);
  const NormEdge edge(cs);
  const float we = kEdges && edge.on && p.w ? load_any(p.w, p.w_dtype, edge.col) : 1.f;
  const float be = kEdges && edge.on && p.b ? load_any(p.b, p.w_dtype, edge.col) : 0.f;
  float top = 0.f;
  if constexpr (CL) cluster_sync_all();   // every CTA of the cluster runs before its shared memory is written
  uint32_t from = ring0;
  // all threads of a row leave the loop together; with several rows in a warp,
  // all of the warp
  for (int64_t row = cs.row; SPAN == 32 ? row < p.rows : row - (lane / SPAN) < p.rows; row += cs.step) {
    if constexpr (MODE == kAny) __syncwarp();      // every lane has read the stage that is copied to
    fetch();
    const bool active = SPAN == 32 || row < p.rows;
    cp_async_wait<S - 1>();
    f32x2 v[kOwn / 2], part[kGroups];
    float xe = 0.f;                         // this lane's element of the row's ends
    if constexpr (kEdges) {
      __syncwarp();                         // other lanes copied it
      if (edge.on) xe = Slot::elem(from + edge.unit * Slot::kBytes, edge.owner, edge.elem);
      __syncwarp();
      if (edge.first && lane == edge.first_owner) Slot::clear(from, lane);
      if (edge.last && lane == edge.last_owner) Slot::clear(from + edge.last_unit * Slot::kBytes, lane);
    }
    uint32_t at = 0u;
    if constexpr (MODE == kAny) {
      const T* x = X + row * p.ldx + cs.col(0) - cs.t;
      __syncwarp();                         // other lanes copied it
      Image::end(from, lane, x, cs.left(0) + cs.t);
      __syncwarp();
      at = Image::place(from, lane, x);
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      float x[G];
      if constexpr (MODE == kAny) {
        x[0] = Image::elem(at, 2 * i);
        x[1] = Image::elem(at, 2 * i + 1);
      } else {
        Unit<T, E> u = Slot::finish(from + i * Slot::kBytes, lane);
        if (MODE == kPhase && !kEdges && !cs.whole(i)) u.keep(cs.lo - cs.col(i), cs.left(i));
        u.get(x);
      }
#pragma unroll
      for (int k = 0; k < G / 2; ++k) v[G / 2 * i + k] = pair(x[2 * k], x[2 * k + 1]);
      part[i] = tree_pairs<G / 2>(v + G / 2 * i);
    }
    const float sum = span_sum<kSpan>(pair_sum(tree_pairs<kGroups>(part)) + xe);
    const float m = divide(sum, n_w, inv_w);
    const f32x2 minus_m = pair(-m);
    f32x2 squares[2] = {pair(0.f), pair(0.f)}, p1[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      f32x2 e[G / 2];
#pragma unroll
      for (int k = 0; k < G / 2; ++k) {
        e[k] = add2(v[G / 2 * i + k], minus_m);
        if constexpr (MODE == kAny) {
          e[k] = keep_pair(e[k], cs.whole(2 * i), cs.whole(2 * i + 1));
        } else if (MODE == kPhase && !kEdges) {
          if (!cs.whole(i)) e[k] = keep_pair(e[k], cs.has(i, 2 * k), cs.has(i, 2 * k + 1));
        }
      }
      if constexpr (G == 2) {
        squares[i & 1] = fma2(*e, *e, squares[i & 1]);
        if constexpr (kRest) p1[i] = *e;
      } else {
        f32x2 q = mul2(e[0], e[0]);
#pragma unroll
        for (int k = 1; k < G / 2; ++k) q = fma2(e[k], e[k], q);
        if constexpr (kRest) p1[i] = tree_pairs<G / 2>(e);
        if ((MODE == kAligned || kEdges) && !cs.whole(i)) {
          q = pair(0.f);
          if constexpr (kRest) p1[i] = pair(0.f);
        }
        squares[i & 1] = add2(squares[i & 1], q);
      }
    }
    float sq = pair_sum(add2(squares[0], squares[1])), rest = 0.f;
    if constexpr (kRest) rest = pair_sum(tree_pairs<kGroups>(p1));
    if constexpr (kEdges) {
      const float e = edge.on ? xe - m : 0.f;
      sq = fmaf(e, e, sq);
      if constexpr (kRest) rest += e;
    }
    RowStats st;
    if constexpr (!kMulti) {
      sq = span_sum<kSpan>(sq);
      const float r = kRest ? sum_rest(m, n_w, span_sum<kSpan>(rest), sq) : division_rest(m, n_w, sum);
      st.set(m, r * inv_n, fmaf(-r, r * inv_n, sq), inv_n, p.eps);
    } else {
      if constexpr (kRest) {
        const float s = warp_sums2(sq, rest);
        const float s2 = __shfl_sync(0xFFFFFFFFu, s, 0);
        if (lane == 0) {
          ex.put(0, sum);
          ex.put(1, s);
        }
        if (lane == 16) ex.put(2, sum_rest(m, n_w, s, s2));
      } else {
        sq = span_sum<32>(sq);
        if (lane == 0) {
          ex.put(0, sum);
          ex.put(1, sq);
        }
      }
      const float* pt = ex.sync();
      // warp k's mean relative to the first's, what it lost (mr; r times its columns)
      const float first = divide(pt[0], n_0, inv_0);
      auto dev = [&](int k, float cw, float inv, float& r, float& mr) {
        const float mk = divide(pt[k], cw, inv);
        r = kRest ? pt[2 * kMost + k] : division_rest(mk, cw, pt[k]);
        mr = r * inv;
        return (mk - first) + mr;
      };
      float r, mr;
      if constexpr (kMost <= 32) {
        const bool in = lane_n > 0.f;
        const float dm = in ? dev(lane % kMost, lane_n, inv_lane, r, mr) : 0.f;
        const float shift = span_sum<kMost>(lane_n * dm) * inv_n;
        const float e = dm - shift;
        const float x = span_sum<kMost>(in ? fmaf(lane_n * e, e, fmaf(-r, mr, pt[kMost + lane])) : 0.f);
        st.set(first, shift, x, inv_n, p.eps);       // right in the lanes of the row's warps
        st.off = __shfl_sync(0xFFFFFFFFu, st.off, 0);
        st.rstd = __shfl_sync(0xFFFFFFFFu, st.rstd, 0);
      } else {
        const int nw = ex.warps;
        float s = 0.f, x = 0.f;
        for (int k = lane; k < nw; k += 32) {
          const float cw = columns_of(k);
          if (cw > 0.f) s = fmaf(cw, dev(k, cw, __fdiv_rn(1.f, cw), r, mr), s);
        }
        const float shift = span_sum<32>(s) * inv_n;
        for (int k = lane; k < nw; k += 32) {
          const float cw = columns_of(k);
          if (cw > 0.f) {
            const float e = dev(k, cw, __fdiv_rn(1.f, cw), r, mr) - shift;
            x += fmaf(cw * e, e, fmaf(-r, mr, pt[kMost + k]));
          }
        }
        st.set(first, shift, span_sum<32>(x), inv_n, p.eps);
      }
    }
    if (active && cs.t == 0 && (!kMulti || ex.mine() == 0)) {
      if (p.mean) p.mean[row] = st.mean;
      if (p.rstd) p.rstd[row] = st.rstd;
    }
    void* y = static_cast<char*>(p.Y) + row * p.ldy * (p.y_dtype == METIS_BF16 ? 2 : 4);
    const f32x2 minus_m0 = pair(-st.m0), rr = pair(st.rstd), off = pair(st.off);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      float o[G];
#pragma unroll
      for (int k = 0; k < G / 2; ++k) {
        const int j = G / 2 * i + k;
        unpair(fma2(fma2(add2(v[j], minus_m0), rr, off), w[j], b[j]), o[2 * k], o[2 * k + 1]);
      }
      store_row_unit_any(cs, y, p.y_dtype, o, G / E * i, active);
      if constexpr (E == 1) store_row_unit_any(cs, y, p.y_dtype, o + 1, 2 * i + 1, active);
    }
    if constexpr (kEdges) {
      if (edge.on) store_any(y, p.y_dtype, edge.col, fmaf(fmaf(xe - st.m0, st.rstd, st.off), we, be));
    }
    if constexpr (SAVE) {
      float x[NV][E];
      uint32_t codes[NV][E / 4];
#pragma unroll
      for (int i = 0; i < NV; ++i) Slot::finish(from + i * Slot::kBytes, lane).get(x[i]);
      const int pad = CL ? min(static_cast<int>(p.save.ldc), cs.lo + p.slice) : static_cast<int>(p.save.ldc);
      uint8_t* scales = p.save.scales + row * p.save.blocks;
      if constexpr (act8_dealt<E, NV>) {
        const uint32_t sc = p.save.fmt == METIS_MXINT8 ? act8_blocks<METIS_MXINT8, E, NV>(x, codes, top)
                                                       : act8_blocks<METIS_MXFP8, E, NV>(x, codes, top);
        const int c = cs.col(0) + cs.t % (32 / E) * Cols::kStride;     // in the block whose scale this lane has
        if (active && c < pad) scales[c >> 5] = static_cast<uint8_t>(sc);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const uint32_t sc = p.save.fmt == METIS_MXINT8 ? act8_block<METIS_MXINT8, E>(x[i], codes[i], top)
                                                         : act8_block<METIS_MXFP8, E>(x[i], codes[i], top);
          if (active && cs.col(i) < pad && cs.t % (32 / E) == 0) scales[cs.col(i) >> 5] = static_cast<uint8_t>(sc);
        }
      }
      uint8_t* dst = p.save.codes + row * p.save.ldc;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (active && cs.col(i) < pad) {
          if constexpr (E == 8)
            *reinterpret_cast<uint2*>(dst + cs.col(i)) = make_uint2(codes[i][0], codes[i][1]);
          else
            *reinterpret_cast<uint32_t*>(dst + cs.col(i)) = codes[i][0];
        }
      }
    }
    from = from + kStage == ring0 + S * kStage ? ring0 : from + kStage;
  }
  cp_async_wait<0>();
  if constexpr (SAVE) {
    __shared__ float wm[16];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
    if (lane == 0) wm[threadIdx.x >> 5] = top;
    __syncthreads();
    top = 0.f;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) top = fmaxf(top, wm[i]);
    act8_write_amax(p.save.amax,
                    p.save.fmt == METIS_MXINT8 ? act8_held<METIS_MXINT8>(top) : act8_held<METIS_MXFP8>(top));
  }
}

template <typename T, int SPAN, int NV, int E, int MODE, bool SAVE, int SHAPE>
void norm_fwd_go(const NormFwdParams& params, int num_sms, cudaStream_t s) {
  using Cols = NormCols<SPAN, NV, E, MODE, SHAPE>;
  constexpr int S = SHAPE == kLanes ? 3 : 2, kWarp = S * FwdStage<T, SPAN, NV, E, MODE>::kBytes;
  auto* kernel = norm_fwd_kernel<T, SPAN, NV, E, S, MODE, SAVE, SHAPE>;
  static NormHeld held;
  NormFwdParams p = params;
  const NormPlan plan(SHAPE, p.cols + (MODE == kPhase ? 7 : 0), fwd_warps<MODE, SHAPE>);
  p.slice = plan.slice;
  const int smem = plan.warps * kWarp;
  const int per_sm = held.get(kernel, plan.warps, smem, (SHAPE == kLanes ? 4 : fwd_warps<MODE, SHAPE>) * kWarp);
  const int64_t most = imin64(static_cast<int64_t>(num_sms) * per_sm, METIS_ACT8_AMAX) / plan.ctas;
  const int64_t blocks = imin64((p.rows + Cols::kRows - 1) / Cols::kRows, imax64(1, most));
  launch_dependent(kernel, dim3(static_cast<unsigned>(norm_blocks(blocks, Cols::kRows, p.period) * plan.ctas)),
                   32 * plan.warps, static_cast<size_t>(smem), plan.ctas, s, p, plan.ctas);
}

// E columns a unit, 32 a thread (16 where a row has 64 or fewer; 40 or 48 where that
// saves the row's second warp: 16384 x 1027 bf16 takes 21.7 us so against 34.2, 1536
// columns 18.6 against 26.8).
template <typename T, int E, int MODE, bool SAVE>
void norm_fwd_cols(const NormFwdParams& p, int num_sms, cudaStream_t s) {
  constexpr int NV = 32 / E, L = E == 8 ? 4 : 8;      // a block of 32 columns lies in 32 / E lanes
  const int cols = p.cols + (MODE == kPhase ? 7 : 0);
  if (cols <= 64)
    norm_fwd_go<T, L, 64 / (L * E), E, MODE, SAVE, kLanes>(p, num_sms, s);
  else if (cols <= 128)
    norm_fwd_go<T, L, 128 / (L * E), E, MODE, SAVE, kLanes>(p, num_sms, s);
  else if (cols <= 256)
    norm_fwd_go<T, 8, NV, E, MODE, SAVE, kLanes>(p, num_sms, s);
  else if (cols <= 512)
    norm_fwd_go<T, 16, NV, E, MODE, SAVE, kLanes>(p, num_sms, s);
  else if (cols <= 1024)
    norm_fwd_go<T, 32, NV, E, MODE, SAVE, kLanes>(p, num_sms, s);
  else if (cols <= 1280)
    norm_fwd_go<T, 32, 40 / E, E, MODE, SAVE, kLanes>(p, num_sms, s);
  else if (cols <= 1536)
    norm_fwd_go<T, 32, 48 / E, E, MODE, SAVE, kLanes>(p, num_sms, s);
  else if (cols <= fwd_warps<MODE, kCta> * kWarpCols)
    norm_fwd_go<T, 32, NV, E, MODE, SAVE, kCta>(p, num_sms, s);
  else if (MODE == kAny && cols <= fwd_warps<MODE, kTall> * kWarpCols)
    norm_fwd_go<T, 32, NV, E, MODE, SAVE, MODE == kAny ? kTall : kCta>(p, num_sms, s);
  else
    norm_fwd_go<T, 32, NV, E, MODE, SAVE, kCluster>(p, num_sms, s);
}

}  // namespace metis
