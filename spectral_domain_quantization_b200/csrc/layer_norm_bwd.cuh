// Layer norm, backward, for rows held in registers.
//
//   xh = (x - mean) rstd, g = dy w
//   dx = rstd (g - sum(g)/n - xh sum(g xh)/n),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Bound by HBM: dy and x (2 or 4 bytes, or 1 + 1/32 from the 8-bit copy) are
// read once and dx written once.  A thread owns the same columns in every row it
// sees, so dw and db are running sums in its registers; a CTA's rows end as one
// row of partial sums, and a second kernel adds those in a fixed order.
//
// Measured, bf16 unless said: 16384 x 4096 76.4 us, 5.3 TB/s (a copy does 6.55), float32
// 127 us (6.3 TB/s), from 8 bits with a float32 gradient 99.7 us (6.1 TB/s); 8192 x 4096
// 46.0 us, from 8 bits 42.8 us; 65536 x 1024 72.4 us; 4000 x 14336 89.1 us, float32 115 us;
// rows that start anywhere 65536 x 1001 86.3 us, 8192 x 4001 58.1 us, 16384 x 1027 34.3
// us; matrices that lie differently 8192 x 4096 65.9 us.  The arithmetic goes two columns
// an instruction (pairs.cuh); what is left short of the copy's rate waits for rows with
// 12 to 16 warps an SM, since the sums of 32 columns a thread take 64 registers and the
// weights 32 (kTall keeps the weights in shared memory; the other shapes were not tried
// so).
#pragma once

#include "layer_norm.cuh"

namespace metis {

struct Act8Tag {};

// Bytes of a unit of x in the ring, of a warp: dense, or E codes of the 8-bit copy.
template <typename TX, int E, int MODE>
struct XBytes {
  static constexpr int value = UnitSlot<TX, E, MODE, 32>::kBytes;
};
template <int E, int MODE>
struct XBytes<Act8Tag, E, MODE> {
  static constexpr int value = E * 32;
};

// x of one unit.
template <typename TX, int E>
struct XUnit {
  Unit<TX, E> u;
  // x - mean, for the negative mean twice
  MDEV void centered(int, f32x2 minus, f32x2* d) const {
    float x[E];
    u.get(x);
#pragma unroll
    for (int k = 0; k < E / 2; ++k) d[k] = add2(pair(x[2 * k], x[2 * k + 1]), minus);
  }
};
// 8 bits: an element is a small integer (or E4M3) times the block's power of two,
// so that x - mean takes one fma.
template <int E>
struct XUnit<Act8Tag, E> {
  uint32_t w[E / 4];
  uint32_t sc;      // scale code
  MDEV void centered(int fmt, f32x2 minus, f32x2* d) const {
    float f, x[E];
    if (fmt == METIS_MXINT8) {
      f = act8_factor<METIS_MXINT8>(sc);
#pragma unroll
      for (int k = 0; k < E / 4; ++k) act8_elems4<METIS_MXINT8>(w[k], x + 4 * k);
    } else {
      f = act8_factor<METIS_MXFP8>(sc);
#pragma unroll
      for (int k = 0; k < E / 4; ++k) act8_elems4<METIS_MXFP8>(w[k], x + 4 * k);
    }
#pragma unroll
    for (int k = 0; k < E / 2; ++k) d[k] = fma2(pair(x[2 * k], x[2 * k + 1]), pair(f), minus);
  }
};

template <typename TX>
struct DenseType {
  using type = TX;
};
template <>
struct DenseType<Act8Tag> {
  using type = float;   // not used
};

template <typename TX, typename TG, int SPAN, int NV, int E, int MODE>
struct BwdStage {
  static constexpr int kG = UnitSlot<TG, E, MODE, 32>::kBytes;
  static constexpr int kOne = kG + XBytes<TX, E, MODE>::value;
  static constexpr int kBytes = NV * kOne;      // of a warp
};
template <typename TX, typename TG, int SPAN, int NV>
struct BwdStage<TX, TG, SPAN, NV, 1, kAny> {
  static constexpr int kG = RowImage<TG, SPAN, NV>::kBytes;
  static constexpr int kOne = kG, kBytes = kG + RowImage<TX, SPAN, NV>::kBytes;
};
template <typename TG, int SPAN, int NV>
struct BwdStage<Act8Tag, TG, SPAN, NV, 1, kAny> {
  static constexpr int kG = RowImage<TG, SPAN, NV>::kBytes;
  static constexpr int kOne = kG, kBytes = kG + 32 * NV;
};

constexpr int kBwdWarps = 8;       // of a CTA
constexpr int kTallWarps = 16;

// CTAs of 8 warps an SM is to hold at least (0: what the compiler makes of it), so 128
// registers a thread, in dense rows that lie aligned.  With and without, us: rows of one
// CTA in bf16 4096 x 8192 47.4 and 64.2, 16384 x 4096 76.3 and 83.1; clusters 4000 x 14336
// bf16 89.6 and 131.8, from float32 with a bf16 gradient 96.8 and 136.0, the other way
// round 107.9 and 144.3.  Not where both are float32: the shared memory of the stages is
// what an SM runs out of (clusters 4000 x 14336 119.1 and 115.9, 4000 x 9000 101.4 and
// 97.5), nor in rows of one CTA with a float32 matrix (16384 x 2048 70.9 and 70.8).
template <typename TX, typename TG, int E, int MODE, int SHAPE>
constexpr int bwd_ctas = MODE == kAligned && !std::is_same_v<TX, Act8Tag> &&
                                 ((SHAPE == kCluster && !(std::is_same_v<TX, float> && std::is_same_v<TG, float>)) ||
                                  (SHAPE == kCta && E == 8))
                             ? 2
                             : 0;

template <typename TX, typename TG, int SPAN, int NV, int E, int S, int MODE, int SHAPE>
__global__ void __launch_bounds__(SHAPE == kLanes ? kLaneThreads : (SHAPE == kTall ? 512 : 256),
                                  bwd_ctas<TX, TG, E, MODE, SHAPE>)
    norm_bwd_kernel(NormBwdParams p, int ctas) {
  using Cols = NormCols<SPAN, NV, E, MODE, SHAPE>;
  using Stage = BwdStage<TX, TG, SPAN, NV, E, MODE>;
  using GS = UnitSlot<TG, E, MODE, 32>;
  using DX = typename DenseType<TX>::type;
  using XS = UnitSlot<DX, E, MODE, 32>;            // dense x
  using GI = RowImage<TG, SPAN, NV>;               // kAny
  using XI = RowImage<DX, SPAN, NV>;
  using Ex = Exchange<2, SHAPE>;
  constexpr bool kDense = !std::is_same_v<TX, Act8Tag>, kMulti = Cols::kMulti, CL = Cols::kClustered;
  constexpr bool kEdges = norm_edges<SPAN, MODE>;
  constexpr int kSpan = SPAN, kMost = Ex::kMost, kOwn = NV * E, kStage = Stage::kBytes;
  constexpr int G = E == 1 ? 2 : E;              // columns that are worked on together: a unit, or two of one column
  static_assert(kDense || MODE != kPhase, "the 8-bit blocks are columns of the matrix: no shift");
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float parts[Ex::kFloats];
  const Cols cs(p.cols, p.slice, ctas, p.ldg, p.offset, 8);
  Ex ex(parts, ctas);
  const int tid = threadIdx.x, lane = tid & 31;
  const TG* dY = static_cast<const TG*>(p.dY);
  const DX* X = static_cast<const DX*>(p.X);
  const Span gspan = span_of<TG>(p.dY, p.rows, p.cols, p.ldg);
  const Span xspan = span_of<DX>(p.X, p.rows, p.cols, p.ldx);
  const uint32_t ring0 = smem_u32(ring) + (tid >> 5) * (S * kStage);
  // kAny, 8 bits: where a warp's elements wait as float32
  const uint32_t d_at = smem_u32(ring) + (blockDim.x >> 5) * (S * kStage) + (tid >> 5) * (128 * NV);

  // row `fetch_row` into the stage at `into`; what a row needs besides, its mean
  // and rstd and the scale codes of its 8-bit blocks, goes into registers one row
  // ahead
  // (kDerived: the loop sets both, for want of registers.  Clusters so and with both
  // carried, us: 4000 x 14336 float32 115.9 and 160.8, bf16 89.8 and 91.5, 4000 x 9000 from
  // 8 bits with a float32 gradient 88.7 and 144.9; 8-bit rows of lanes 100000 x 512 60.2
  // and 63.0.  Rows of a CTA take longer so: 16384 x 4096 bf16 81.7 and 76.4.)
  constexpr bool kDerived = CL || (!kDense && !kMulti);
  int64_t fetch_row = cs.row;
  uint32_t into = ring0;
  auto fetch = [&] {
    const bool on = fetch_row < p.rows;
    if (SPAN < 32 || on) {
      const TG* g = dY + fetch_row * p.ldg;
      const bool inside = MODE == kPhase && on && row_inside(g, p.cols, gspan) &&
                          (!kDense || row_inside(X + fetch_row * p.ldx, p.cols, xspan));
      if constexpr (MODE == kAny) {
        const int n = on ? cs.left(0) + cs.t : 0, c = cs.col(0) - cs.t;
        GI::start(into, lane, g + c, n, gspan);
        if constexpr (kDense) {
          XI::start(into + Stage::kG, lane, X + fetch_row * p.ldx + c, n, xspan);
        } else {
          // SPAN * NV codes, 16 at a time (c is a multiple of 32, and the codes' rows
          // are padded to one)
          const uint8_t* q = p.saved.codes + fetch_row * p.saved.ldc + c;
#pragma unroll
          for (int k = 0; k < (NV + 15) / 16; ++k) {
            const int at = 16 * (cs.t + SPAN * k);
            if (at < SPAN * NV) cp_async16(into + Stage::kG + lane / SPAN * (SPAN * NV) + at, q + at, at < n ? 16 : 0);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const uint32_t at = into + i * Stage::kOne;
          GS::start(at, lane, g + cs.col(i), on && cs.whole(i), on && cs.some(i), inside, gspan);
          if constexpr (kDense)
            XS::start(at + GS::kBytes, lane, X + fetch_row * p.ldx + cs.col(i), on && cs.whole(i), on && cs.some(i),
                      inside, xspan);
          else
            cp_async<E>(at + GS::kBytes + E * lane, p.saved.codes + fetch_row * p.saved.ldc + cs.col(i),
                        on && cs.left(i) > 0);
        }
      }
    }
    cp_async_commit();
    if constexpr (!kDerived) {
      fetch_row += cs.step;
      into = into + kStage == ring0 + S * kStage ? ring0 : into + kStage;
    }
  };
  float next_mean = 0.f, next_rstd = 0.f;
  // kAny: lane t has the scale code of the t-th 8-bit block of its row's lanes
  constexpr int kScales = kDense || MODE == kAny ? 1 : NV;
  uint32_t next_sc[kScales];
  auto fetch_stats = [&](int64_t row) {
    const bool on = row < p.rows;
    next_mean = on ? p.mean[row] : 0.f;
    next_rstd = on ? p.rstd[row] : 0.f;
    if constexpr (!kDense && MODE == kAny) {
      const int c = cs.col(0) - cs.t + 32 * cs.t;
      next_sc[0] = on && 32 * cs.t < SPAN * NV && c < cs.hi ? p.saved.scales[row * p.saved.blocks + (c >> 5)] : 0u;
    } else if constexpr (!kDense) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        next_sc[i] = on && cs.left(i) > 0 ? p.saved.scales[row * p.saved.blocks + (cs.col(i) >> 5)] : 0u;
    }
  };
  wait_for_previous();
#pragma unroll
  for (int k = 0; k < S - 1; ++k) fetch();
  fetch_stats(cs.row);
  f32x2 w[kOwn / 2], aw[kOwn / 2], ab[kOwn / 2];
  {
    float v[kOwn];
    load_vector(cs, p.w, p.w_dtype, 1.f, v);
#pragma unroll
    for (int k = 0; k < kOwn / 2; ++k) w[k] = pair(v[2 * k], v[2 * k + 1]);
  }
  // kTall: 128 registers a thread have no room for the weights; each thread keeps
  // its own behind the ring
  constexpr bool kStaged = SHAPE == kTall;
  const uint32_t w_at = smem_u32(ring) + (blockDim.x >> 5) * (S * kStage) + 16 * tid;
  if constexpr (kStaged) {
#pragma unroll
    for (int k = 0; k < kOwn / 4; ++k)
      asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(w_at + 16 * k * blockDim.x), "l"(w[2 * k]), "l"(w[2 * k + 1])
                   : "memory");
  }
  auto w_group = [&](int i, f32x2* o) {
    if constexpr (kStaged) {
#pragma unroll
      for (int k = 0; k < G / 4; ++k)
        asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                     : "=l"(o[2 * k]), "=l"(o[2 * k + 1])
                     : "r"(w_at + 16 * (i * (G / 4) + k) * blockDim.x)
                     : "memory");
    } else {
#pragma unroll
      for (int j = 0; j < G / 2; ++j) o[j] = w[G / 2 * i + j];
    }
  };
#pragma unroll
  for (int k = 0; k < kOwn / 2; ++k) aw[k] = ab[k] = pair(0.f);
  const NormEdge edge(cs);
  const float we = kEdges && edge.on && p.w ? load_any(p.w, p.w_dtype, edge.col) : 1.f;
  float awe = 0.f, abe = 0.f;             // dw and db of that element's column
  if constexpr (CL) cluster_sync_all();   // every CTA of the cluster runs before its shared memory is written
  uint32_t from = ring0;
  // all threads of a row leave the loop together; with several rows in a warp,
  // all of the warp
  for (int64_t row = cs.row; SPAN == 32 ? row < p.rows : row - (lane / SPAN) < p.rows; row += cs.step) {
    if constexpr (MODE == kAny) __syncwarp();      // every lane has read the stage that is copied to
    if constexpr (kDerived) {
      static_assert(S == 2);
      fetch_row = row + cs.step;
      into = 2 * ring0 + kStage - from;
    }
    fetch();
    const bool active = SPAN == 32 || row < p.rows;
    const float mean = next_mean, rstd = next_rstd;
    uint32_t sc[kScales];
#pragma unroll
    for (int i = 0; i < kScales; ++i) sc[i] = kDense ? 0u : next_sc[i];
    fetch_stats(row + cs.step);
    cp_async_wait<S - 1>();
    uint32_t g_at = 0u, x_at = 0u;
    if constexpr (MODE == kAny) {
      const int c = cs.col(0) - cs.t, n = cs.left(0) + cs.t;
      __syncwarp();                         // other lanes copied it
      GI::end(from, lane, dY + row * p.ldg + c, n);
      if constexpr (kDense) XI::end(from + Stage::kG, lane, X + row * p.ldx + c, n);
      __syncwarp();
      g_at = GI::place(from, lane, dY + row * p.ldg + c);
      if constexpr (kDense) {
        x_at = XI::place(from + Stage::kG, lane, X + row * p.ldx + c);
      } else {
        // x - mean as float32 behind the ring, four codes of a block at a time
        const uint32_t codes = from + Stage::kG + lane / SPAN * (SPAN * NV), wide = d_at + lane / SPAN * (4 * SPAN * NV);
        const uint32_t factor = __float_as_uint(p.saved.fmt == METIS_MXINT8 ? act8_factor<METIS_MXINT8>(sc[0])
                                                                            : act8_factor<METIS_MXFP8>(sc[0]));
        auto decode = [&](auto fmt) {
#pragma unroll
          for (int j = 0; j < NV / 4; ++j) {
            const int k = cs.t + SPAN * j;
            const float f = __uint_as_float(__shfl_sync(0xFFFFFFFFu, factor, lane - cs.t + (k >> 3)));
            uint32_t w;
            lds<1>(codes + 4 * k, &w);
            float v[4];
            act8_elems4<decltype(fmt)::value>(w, v);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = fmaf(v[q], f, -mean);
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(wide + 16 * k), "f"(v[0]), "f"(v[1]),
                         "f"(v[2]), "f"(v[3])
                         : "memory");
          }
        };
        if (p.saved.fmt == METIS_MXINT8)
          decode(std::integral_constant<int, METIS_MXINT8>{});
        else
          decode(std::integral_constant<int, METIS_MXFP8>{});
        __syncwarp();
        x_at = wide + 4 * cs.t;
      }
    }
    // dy and x - mean of group i
    const f32x2 minus = pair(-mean);
    auto g_group = [&](int i, f32x2* dy) {
      float v[G];
      if constexpr (MODE == kAny) {
        v[0] = GI::elem(g_at, 2 * i);
        v[1] = GI::elem(g_at, 2 * i + 1);
      } else {
        Unit<TG, E> u = GS::finish(from + i * Stage::kOne, lane);
        if (MODE == kPhase && !kEdges && !cs.whole(i)) u.keep(cs.lo - cs.col(i), cs.left(i));
        u.get(v);
      }
#pragma unroll
      for (int k = 0; k < G / 2; ++k) dy[k] = pair(v[2 * k], v[2 * k + 1]);
    };
    auto x_group = [&](int i, f32x2* d) {
      if constexpr (MODE == kAny) {
        if constexpr (kDense)
          *d = add2(pair(XI::elem(x_at, 2 * i), XI::elem(x_at, 2 * i + 1)), minus);
        else
          *d = pair(lds_elem<float>(x_at + 8 * SPAN * i), lds_elem<float>(x_at + 8 * SPAN * i + 4 * SPAN));
      } else {
        XUnit<TX, E> x;
        if constexpr (!kDense) {
          lds<E / 4>(from + i * Stage::kOne + GS::kBytes + E * lane, x.w);
          x.sc = sc[i];
        } else {
          x.u = XS::finish(from + i * Stage::kOne + GS::kBytes, lane);
          if (MODE == kPhase && !kEdges && !cs.whole(i)) x.u.keep(cs.lo - cs.col(i), cs.left(i));
        }
        x.centered(p.saved.fmt, minus, d);
      }
    };
    // sums of g xh and of g rstd.  rstd goes to dy, not to x - mean: a column that is
    // not the row's has x = 0 and dy = 0, and dy (0 - mean) is 0 for any mean, where
    // (0 - mean) rstd may be past float32 and 0 times it NaN
    float s1 = 0.f, s2 = 0.f;
    float xe = 0.f, ge = 0.f;               // this lane's element of the row's ends: x - mean, and dy
    if constexpr (kEdges) {
      __syncwarp();                         // other lanes copied it
      if (edge.on) {
        const uint32_t at = from + edge.unit * Stage::kOne;
        ge = GS::elem(at, edge.owner, edge.elem);
        xe = XS::elem(at + GS::kBytes, edge.owner, edge.elem) - mean;
      }
      __syncwarp();
      if (edge.first && lane == edge.first_owner) {
        GS::clear(from, lane);
        XS::clear(from + GS::kBytes, lane);
      }
      if (edge.last && lane == edge.last_owner) {
        GS::clear(from + edge.last_unit * Stage::kOne, lane);
        XS::clear(from + edge.last_unit * Stage::kOne + GS::kBytes, lane);
      }
      const float r = ge * rstd, gr = r * we;
      s1 = gr * xe;
      s2 = gr;
      awe = fmaf(r, xe, awe);
      abe += ge;
    }
    f32x2 t1 = pair(s1, 0.f), t2 = pair(s2, 0.f);
    const f32x2 rr = pair(rstd);
#pragma unroll
    for (int i = 0; i < kOwn / G; ++i) {
      f32x2 d[G / 2], dy[G / 2], wu[G / 2];
      w_group(i, wu);
      x_group(i, d);
      g_group(i, dy);
#pragma unroll
      for (int j = 0; j < G / 2; ++j) {
        const int k = G / 2 * i + j;
        const f32x2 r = mul2(dy[j], rr), gr = mul2(r, wu[j]);
        t1 = fma2(gr, d[j], t1);
        t2 = add2(t2, gr);
        aw[k] = fma2(r, d[j], aw[k]);
        ab[k] = add2(ab[k], dy[j]);
      }
    }
    s1 = pair_sum(t1);
    s2 = pair_sum(t2);
    if (p.dX) {
      float c1, c2;
      if constexpr (!kMulti) {
        c1 = span_sum<kSpan>(s1);
        c2 = span_sum<kSpan>(s2);
      } else {
        const float s = warp_sums2(s1, s2);
        if ((lane & 15) == 0) ex.put(lane >> 4, s);
        const float* pt = ex.sync();
        if constexpr (kMost == 16) {
          // lanes 0 to 15 have the warps' first sums, 16 to 31 their second
          const float t = span_sum<16>((lane & 15) < ex.warps ? pt[lane] : 0.f);
          c1 = __shfl_sync(0xFFFFFFFFu, t, 0);
          c2 = __shfl_sync(0xFFFFFFFFu, t, 16);
        } else {
          float a = 0.f, b = 0.f;
          for (int k = lane; k < ex.warps; k += 32) {
            a += pt[k];
            b += pt[kMost + k];
          }
          c1 = span_sum<32>(a);
          c2 = span_sum<32>(b);
        }
      }
      // dx = rstd g + (x - mean) kd + k0
      const float kd = -rstd * (rstd * (c1 * p.inv_n)), k0 = -(c2 * p.inv_n);
      void* out = static_cast<char*>(p.dX) + row * p.ldd * (p.dx_dtype == METIS_BF16 ? 2 : 4);
      const f32x2 kd2 = pair(kd), k02 = pair(k0);
#pragma unroll
      for (int i = 0; i < kOwn / G; ++i) {
        f32x2 d[G / 2], dy[G / 2], wu[G / 2];
        float o[G];
        w_group(i, wu);
        x_group(i, d);
        g_group(i, dy);
#pragma unroll
        for (int j = 0; j < G / 2; ++j)
          unpair(fma2(mul2(dy[j], rr), wu[j], fma2(d[j], kd2, k02)), o[2 * j], o[2 * j + 1]);
        store_row_unit_any(cs, out, p.dx_dtype, o, G / E * i, active);
        if constexpr (E == 1) store_row_unit_any(cs, out, p.dx_dtype, o + 1, 2 * i + 1, active);
      }
      if constexpr (kEdges) {
        if (edge.on) store_any(out, p.dx_dtype, edge.col, fmaf(ge * we, rstd, fmaf(xe, kd, k0)));
      }
    }
    if constexpr (kDerived)
      from = into;
    else
      from = from + kStage == ring0 + S * kStage ? ring0 : from + kStage;
  }
  cp_async_wait<0>();
  launch_next();   // the kernel that adds the partial sums waits for this one's end
  // this CTA's partial sums; the ring's memory is free
  float* gather = reinterpret_cast<float*>(ring);
  const int64_t blk = CL ? blockIdx.x / ctas : blockIdx.x;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* part = which == 0 ? p.part_w : p.part_b;
    if (!part) continue;
    part += blk * p.part_ld;
    float a[kOwn];
#pragma unroll
    for (int k = 0; k < kOwn / 2; ++k) unpair(which == 0 ? aw[k] : ab[k], a[2 * k], a[2 * k + 1]);
    if constexpr (Cols::kRows > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (kEdges ? cs.whole(i) : cs.has(i, j)) gather[(tid / SPAN) * (SPAN * kOwn) + cs.col(i) + j] = a[E * i + j];
      if (kEdges && edge.on) gather[(tid / SPAN) * (SPAN * kOwn) + edge.col] = which == 0 ? awe : abe;
      __syncthreads();
      for (int c = tid; c < p.cols; c += kLaneThreads) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < Cols::kRows; ++k) s += gather[k * (SPAN * kOwn) + c];
        part[c] = s;
      }
    } else {
      const bool wide = MODE == kAligned && (reinterpret_cast<uintptr_t>(part) & 15u) == 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (wide && cs.left(i) >= E) {
#pragma unroll
          for (int k = 0; k < E / 4; ++k)
            reinterpret_cast<float4*>(part + cs.col(i))[k] =
                make_float4(a[E * i + 4 * k], a[E * i + 4 * k + 1], a[E * i + 4 * k + 2], a[E * i + 4 * k + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < E; ++j)
            if (kEdges ? cs.whole(i) : cs.has(i, j)) part[cs.col(i) + j] = a[E * i + j];
        }
      }
      if (kEdges && edge.on) part[edge.col] = which == 0 ? awe : abe;
    }
  }
}

// Launches, or (occupancy) returns how many CTAs or clusters run at once.
template <typename TX, typename TG, int SPAN, int NV, int E, int MODE, int SHAPE>
int norm_bwd_go(const NormBwdParams& params, int parts, bool occupancy, int num_sms, cudaStream_t s) {
  using Cols = NormCols<SPAN, NV, E, MODE, SHAPE>;
  constexpr int kStage = BwdStage<TX, TG, SPAN, NV, E, MODE>::kBytes;
  constexpr int kGather = SHAPE == kLanes && Cols::kRows > 1 ? 32 * NV * E * 4 : 0;   // of a warp, when the ring is done
  // two stages and the CTAs that then fit an SM: three stages take 77.2 us against
  // 76.3 on 16384 x 4096 bf16, and 144 against 127 in float32
  constexpr int S = 2;
  // the weights, or the elements of an 8-bit row that lies anywhere
  constexpr int kStaged = SHAPE == kTall ? 4 * kWarpCols : (MODE == kAny && std::is_same_v<TX, Act8Tag> ? 128 * NV : 0);
  constexpr int kMostWarps = SHAPE == kTall ? kTallWarps : kBwdWarps;
  constexpr int kWarp = (S * kStage > kGather ? S * kStage : kGather) + kStaged;
  auto* kernel = norm_bwd_kernel<TX, TG, SPAN, NV, E, S, MODE, SHAPE>;
  static NormHeld held;
  NormBwdParams p = params;
  const NormPlan plan(SHAPE, p.cols + (MODE == kPhase ? 7 : 0), kMostWarps);
  p.slice = plan.slice;
  const int smem = plan.warps * kWarp;
  const int per_sm = held.get(kernel, plan.warps, smem, (SHAPE == kLanes ? 4 : kMostWarps) * kWarp);
  if (occupancy) {
    const int64_t most = imax64(1, static_cast<int64_t>(num_sms) * per_sm / plan.ctas);
    return static_cast<int>(
        norm_blocks(imin64((p.rows + Cols::kRows - 1) / Cols::kRows, most), Cols::kRows, p.period));
  }
  launch_dependent(kernel, dim3(static_cast<unsigned>(parts * plan.ctas)), 32 * plan.warps, static_cast<size_t>(smem),
                   plan.ctas, s, p, plan.ctas);
  return 0;
}

// E columns a unit, 32 a thread (16 where a row has 64 or fewer; 40 where that saves
// the row's second warp and its sums still fit the registers: 16384 x 1280 bf16 takes
// 29.6 us so against 40.7, 16384 x 1027 34.3 against 50.3).
template <typename TX, typename TG, int E, int MODE>
int norm_bwd_cols(const NormBwdParams& p, int parts, bool occ, int num_sms, cudaStream_t s) {
  constexpr int NV = 32 / E, L = E == 8 ? 4 : 8;
  const int cols = p.cols + (MODE == kPhase ? 7 : 0);
  if (cols <= 64) return norm_bwd_go<TX, TG, L, 64 / (L * E), E, MODE, kLanes>(p, parts, occ, num_sms, s);
  if (cols <= 128) return norm_bwd_go<TX, TG, L, 128 / (L * E), E, MODE, kLanes>(p, parts, occ, num_sms, s);
  if (cols <= 256) return norm_bwd_go<TX, TG, 8, NV, E, MODE, kLanes>(p, parts, occ, num_sms, s);
  if (cols <= 512) return norm_bwd_go<TX, TG, 16, NV, E, MODE, kLanes>(p, parts, occ, num_sms, s);
  if (cols <= 1024) return norm_bwd_go<TX, TG, 32, NV, E, MODE, kLanes>(p, parts, occ, num_sms, s);
  if constexpr (E == 8) {
    if (cols <= 1280) return norm_bwd_go<TX, TG, 32, 40 / E, E, MODE, kLanes>(p, parts, occ, num_sms, s);
  }
  if (cols <= kBwdWarps * kWarpCols) return norm_bwd_go<TX, TG, 32, NV, E, MODE, kCta>(p, parts, occ, num_sms, s);
  // One CTA of up to 16 warps in place of a cluster of two, for long rows (4000 of them
  // unless said; one CTA against a cluster, us).  Shifted bf16 rows: from 10 warps on,
  // since shorter ones gain little and lose where the rows are few (8449 columns 83.2 and
  // 86.5, 9001 85.6 and 88.2, 333 rows of 9001 25.0 and 22.7; 10239 88.1 and 93.5, 12279
  // 102.1 and 102.0, 14335 108.0 and 153.8).  From 8 bits: where a cluster's CTAs have more
  // than 6 warps, so that an SM holds one of them (bf16 gradient: 9000 columns 78.9 and
  // 74.8, 10240 76.6 and 76.0, 12288 86.7 and 80.2, 12320 86.8 and 118.7, 14336 88.4 and
  // 120.4; float32 gradient: 9000 98.2 and 88.5, 12288 105 and 95.0, 14336 109 and 148).
  // Dense rows that lie aligned have clusters of two CTAs to an SM (bwd_ctas); the stages
  // of the other shifted rows and the weights do not fit an SM's shared memory.
  constexpr bool kKept = std::is_same_v<TX, Act8Tag>;
  if constexpr ((kKept && E != 1) || (E == 8 && MODE == kPhase)) {
    if (cols > (kKept ? 12 : 10) * kWarpCols && cols <= kTallWarps * kWarpCols)
      return norm_bwd_go<TX, TG, 32, NV, E, MODE, kTall>(p, parts, occ, num_sms, s);
  }
  return norm_bwd_go<TX, TG, 32, NV, E, MODE, kCluster>(p, parts, occ, num_sms, s);
}

template <typename TX>
int norm_bwd_kind(const NormBwdParams& p, int mode, bool narrow, int parts, bool occ, int num_sms, cudaStream_t s) {
  using H = __nv_bfloat16;
  constexpr bool kDense = !std::is_same_v<TX, Act8Tag>, kF32 = std::is_same_v<TX, float>;
  const bool g16 = p.g_dtype == METIS_BF16;
  if (mode == kAny)
    return g16 ? norm_bwd_cols<TX, H, 1, kAny>(p, parts, occ, num_sms, s)
               : norm_bwd_cols<TX, float, 1, kAny>(p, parts, occ, num_sms, s);
  if constexpr (kDense) {
    if (mode == kPhase) {
      if constexpr (!kF32)
        if (narrow) return norm_bwd_cols<TX, H, 8, kPhase>(p, parts, occ, num_sms, s);
      return g16 ? norm_bwd_cols<TX, H, 4, kPhase>(p, parts, occ, num_sms, s)
                 : norm_bwd_cols<TX, float, 4, kPhase>(p, parts, occ, num_sms, s);
    }
  }
  if constexpr (!kF32)
    if (narrow) return norm_bwd_cols<TX, H, 8, kAligned>(p, parts, occ, num_sms, s);
  return g16 ? norm_bwd_cols<TX, H, 4, kAligned>(p, parts, occ, num_sms, s)
             : norm_bwd_cols<TX, float, 4, kAligned>(p, parts, occ, num_sms, s);
}

}  // namespace metis
