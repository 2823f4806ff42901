// Activations kept in 8 bits between the forward and the backward pass: the
// 8-bit copy of a matrix, its way back to bf16 / f32, and the FP4 operand of
// dW = X^T dY made from it in one pass.
//
// All three kernels are bound by HBM: a copy moves 2 (bf16) or 4 bytes in and
// 1 + 1/32 out per element, or the reverse; the FP4 pass reads 1 + 1/32 and
// writes 1/2 + 1/16 (NVFP4) or 1/2 + 1/32.
#include "abi_common.h"
#include "act8.cuh"
#include "act8.h"
#include "dependent.cuh"
#include "fp4_block.cuh"
#include "rows.cuh"

namespace metis {

namespace {

constexpr int kThreads = 256;

// Where unit u of 8 (or E) columns lies.  The codes of all rows form one sequence of
// units, 4 to a block; a row's first and last element need its row and place: a
// multiplication by a rounded-up reciprocal for fewer than 2^31 units (Granlund and
// Montgomery's division by an invariant: with s = ceil(log2 d) and m = floor(2^32
// (2^s - d) / d) + 1, n / d is (mulhi(n, m) + n) >> s), a 64-bit division otherwise.
struct UnitMap {
  int64_t total;
  int64_t per_row;
  uint32_t m, s;
  bool narrow;
  MDEV void split(int64_t u, int64_t& row, int& k) const {
    if (narrow) {
      const uint32_t n = static_cast<uint32_t>(u);
      const uint32_t r = (__umulhi(n, m) + n) >> s;
      row = r;
      k = static_cast<int>(n - r * static_cast<uint32_t>(per_row));
    } else {
      row = u / per_row;
      k = static_cast<int>(u - row * per_row);
    }
  }
};

UnitMap unit_map(int64_t rows, int64_t per_row) {
  UnitMap m{};
  m.per_row = per_row;
  m.total = rows * per_row;
  m.narrow = m.total < (int64_t{1} << 31);
  while ((int64_t{1} << m.s) < per_row) ++m.s;
  m.m = static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{1} << m.s) - per_row)) / per_row + 1);
  return m;
}

// How a dense matrix lies against the units.
enum UnitShape {
  kFlat = 0,      // rows of whole blocks, one behind the other: unit u is elements 8 u to 8 u + 7
  kRowsAligned,   // rows on 16-byte boundaries
  kRowsAny
};

// Columns of a unit of the way back.
template <typename T>
constexpr int restore_width(int shape) {
  return sizeof(T) == 4 && shape != kRowsAny ? 4 : 8;
}

MDEV float cta_max(float m) {
  __shared__ float wm[kThreads / 32];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  if ((threadIdx.x & 31) == 0) wm[threadIdx.x >> 5] = m;
  __syncthreads();
  m = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, wm[i]);
  return m;
}

// 8 elements a thread, a block in 4 adjacent lanes, the units dealt to the lanes in
// order.  16384 x 14336 bf16 110.6 us (6.4 TB/s; a copy does 6.55), 16384 x 4096 float32
// 53.9 us (6.3 TB/s); 8192 x 4096 bf16 18.3 us.
template <int FMT, typename T, int SHAPE>
__global__ void __launch_bounds__(kThreads) act8_save_kernel(const T* X, int64_t rows, int64_t cols, int64_t ld,
                                                             Act8View out, UnitMap map) {
  constexpr bool AL = SHAPE != kRowsAny;
  constexpr int kU = 4;                           // units in flight per thread
  const int lane = threadIdx.x & 31;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  const Span span = span_of<T>(X, rows, cols, ld);
  float top = 0.f;
  wait_for_previous();
  // the loop's bound is the same for a warp
  for (int64_t u0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; u0 - lane < map.total;
       u0 += kU * stride) {
    UnitLoad<T, AL> in[kU];
    int left[kU];
    bool last[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int64_t u = u0 + i * stride;
      const T* src = X + 8 * u;
      left[i] = 8;
      last[i] = true;
      if constexpr (SHAPE != kFlat) {
        int64_t row;
        int k;
        map.split(u < map.total ? u : 0, row, k);
        left[i] = static_cast<int>(cols) - 8 * k;
        last[i] = lane == 31 || k + 1 == map.per_row;
        src = X + row * ld + 8 * k;
      }
      if (u >= map.total) left[i] = -16;
      in[i].start(src, left[i], last[i], span);
    }
    float v[kU][8];
    uint32_t codes[kU][2];
#pragma unroll
    for (int i = 0; i < kU; ++i) in[i].finish(left[i], last[i]).get(v[i]);
    const uint32_t sc = act8_blocks<FMT, 8, kU>(v, codes, top);
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int64_t u = u0 + i * stride;
      if (u < map.total) *reinterpret_cast<uint2*>(out.codes + 8 * u) = make_uint2(codes[i][0], codes[i][1]);
    }
    const int64_t mine = u0 + (lane & 3) * stride;     // in the block whose scale this lane has
    if (mine < map.total) out.scales[mine >> 2] = static_cast<uint8_t>(sc);
  }
  act8_write_amax(out.amax, act8_held<FMT>(cta_max(top)));
}

// E elements a thread (8, and 4 of an aligned float32 matrix, so that the warp's
// stores are contiguous); a row's units stop at its last column.  16384 x 14336 to bf16
// 127 us (5.6 TB/s: twice as much written as read), 16384 x 4096 to float32 63.3 us (5.3
// TB/s).
template <int FMT, typename T, int SHAPE>
__global__ void __launch_bounds__(kThreads) act8_restore_kernel(Act8View in, int64_t cols, T* Y, int64_t ld,
                                                                UnitMap map) {
  constexpr int E = restore_width<T>(SHAPE);
  constexpr int kU = 32 / E;
  const int lane = threadIdx.x & 31;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  wait_for_previous();
  for (int64_t u0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; u0 - lane < map.total;
       u0 += kU * stride) {
    uint32_t raw[kU][E / 4];
    uint32_t sc[kU];
    T* dst[kU];
    int k[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int64_t u = u0 + i * stride;
      k[i] = 0;
      sc[i] = 0u;
#pragma unroll
      for (int w = 0; w < E / 4; ++w) raw[i][w] = 0u;
      dst[i] = Y + E * u;
      if (u < map.total) {
        int64_t c = u;                        // the unit's place among the codes'
        if constexpr (SHAPE != kFlat) {
          int64_t row;
          map.split(u, row, k[i]);
          c = row * (in.ldc / E) + k[i];
          dst[i] = Y + row * ld + E * k[i];
        }
        if constexpr (E == 8) {
          const uint2 q = *reinterpret_cast<const uint2*>(in.codes + 8 * c);
          raw[i][0] = q.x;
          raw[i][E / 4 - 1] = q.y;
        } else {
          raw[i][0] = *reinterpret_cast<const uint32_t*>(in.codes + 4 * c);
        }
        sc[i] = in.scales[c / (32 / E)];
      }
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const float f = act8_factor<FMT>(sc[i]);
      float v[E];
#pragma unroll
      for (int w = 0; w < E / 4; ++w) act8_elems4<FMT>(raw[i][w], v + 4 * w);
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] *= f;
      Unit<T, E> y;
      y.put(v);
      const bool on = u0 + i * stride < map.total;
      if constexpr (SHAPE == kRowsAny) {
        store_unit(dst[i], y, on ? static_cast<int>(cols) - 8 * k[i] : 0, lane == 0 || k[i] == 0,
                             lane == 31 || k[i] + 1 == map.per_row);
      } else if (on) {
        const int left = static_cast<int>(cols) - E * k[i];
        if (SHAPE == kFlat || left >= E) {
          y.store(dst[i]);
        } else {
#pragma unroll
          for (int j = 0; j < E; ++j)
            if (j < left) dst[i][j] = y.elem(j);
        }
      }
    }
  }
}

int occupancy(const void* kernel, size_t smem = 0) {
  int per_sm = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, smem) != cudaSuccess || per_sm < 1)
    per_sm = 1;
  return per_sm;
}

// no more CTAs than are resident at once (the loops are grid-strided), and than the
// maximum has slots.  Only the copy writes those, but the way back gains nothing from the
// 160 more that would fit: 16384 x 14336 bf16 130.4 us with them against 127.5.
int grid_for(int per_sm, int64_t ctas, int num_sms) {
  const int64_t most = imin64(static_cast<int64_t>(num_sms) * per_sm, METIS_ACT8_AMAX);
  return static_cast<int>(imax64(1, imin64(ctas, most)));
}

template <typename T>
UnitShape unit_shape(const T* p, int64_t cols, int64_t ld) {
  if ((reinterpret_cast<uintptr_t>(p) & 15u) || (ld * static_cast<int64_t>(sizeof(T))) % 16) return kRowsAny;
  return cols % 32 == 0 && ld == cols ? kFlat : kRowsAligned;
}

template <int FMT, typename T, int SHAPE>
void save_shape(const T* X, int64_t rows, int64_t cols, int64_t ld, const Act8View& out, int num_sms, cudaStream_t s) {
  const UnitMap map = unit_map(rows, 4 * out.blocks);
  auto* kernel = act8_save_kernel<FMT, T, SHAPE>;
  static const int per_sm = occupancy(reinterpret_cast<const void*>(kernel));
  const int grid = grid_for(per_sm, (map.total + kThreads - 1) / kThreads, num_sms);
  launch_dependent(kernel, dim3(static_cast<unsigned>(grid)), kThreads, 0, 1, s, X, rows, cols, ld, out, map);
}

template <int FMT, typename T, int SHAPE>
void restore_shape(const Act8View& in, int64_t rows, int64_t cols, T* Y, int64_t ld, int num_sms, cudaStream_t s) {
  constexpr int E = restore_width<T>(SHAPE);
  const UnitMap map = unit_map(rows, (cols + E - 1) / E);
  auto* kernel = act8_restore_kernel<FMT, T, SHAPE>;
  static const int per_sm = occupancy(reinterpret_cast<const void*>(kernel));
  const int grid = grid_for(per_sm, (map.total + kThreads - 1) / kThreads, num_sms);
  launch_dependent(kernel, dim3(static_cast<unsigned>(grid)), kThreads, 0, 1, s, in, cols, Y, ld, map);
}

template <int FMT, typename T>
void save_t(const T* X, int64_t rows, int64_t cols, int64_t ld, const Act8View& out, int num_sms, cudaStream_t s) {
  switch (unit_shape(X, cols, ld)) {
    case kFlat: return save_shape<FMT, T, kFlat>(X, rows, cols, ld, out, num_sms, s);
    case kRowsAligned: return save_shape<FMT, T, kRowsAligned>(X, rows, cols, ld, out, num_sms, s);
    default: return save_shape<FMT, T, kRowsAny>(X, rows, cols, ld, out, num_sms, s);
  }
}

template <int FMT, typename T>
void restore_t(const Act8View& in, int64_t rows, int64_t cols, T* Y, int64_t ld, int num_sms, cudaStream_t s) {
  switch (unit_shape(Y, cols, ld)) {
    case kFlat: return restore_shape<FMT, T, kFlat>(in, rows, cols, Y, ld, num_sms, s);
    case kRowsAligned: return restore_shape<FMT, T, kRowsAligned>(in, rows, cols, Y, ld, num_sms, s);
    default: return restore_shape<FMT, T, kRowsAny>(in, rows, cols, Y, ld, num_sms, s);
  }
}

// ---------------------------------------------------------------------------
// 8 bits -> FP4
// ---------------------------------------------------------------------------

struct Act8QuantParams {
  Act8View in;
  int64_t rows, cols;
  int64_t outer, inner;
  int64_t scale_cols;        // padded scale columns of the tensor-core layout
  uint8_t* codes;
  uint8_t* scales;
  uint8_t* scales_linear;    // optional
  float* tensor_scale;
  int otiles, itiles;        // tiles over the padded outer and inner indices
  int step_o, step_i;        // gridDim.x as outer and inner tiles
};

// a / b, correctly rounded, from b's correctly rounded reciprocal: the first
// correction leaves a quotient within a unit in the last place, the second rounds it
// (Markstein).  b within 2^-90 .. 2^90; a quotient under 2^-9 may be off (its scale
// code is 0 either way).
MDEV float divide_exact(float a, float b, float inv) {
  float q = a * inv;
  q = fmaf(fmaf(-q, b, a), inv, q);
  return fmaf(fmaf(-q, b, a), inv, q);
}

// The scale of an NVFP4 tensor, for its blocks.
struct NvScale {
  float s_t, inv;
  bool plain;       // s_t is out of divide_exact's range
  MDEV explicit NvScale(float s) {
    s_t = s;
    inv = __fdiv_rn(1.f, s);
    plain = !(s > 0x1p-90f && s < 0x1p90f);
  }
  // quant_block_nv_tab's scale code of a block with maximum a
  MDEV uint32_t code(float a) const {
    if (plain) return e4m3_code(__fdiv_rn(__fdiv_rn(a, s_t), 6.f));
    return e4m3_code(divide_exact(divide_exact(a, s_t, inv), 6.f, 1.f / 6.f));
  }
};

// One FP4 block's codes (8 a word) and scale code; the bytes of quant_block_nv_tab
// and quant_block_mx.
template <int FMT4>
MDEV uint32_t fp4_block(const float* v, const NvScale& nv, const float* enc_tab, uint32_t* w) {
  constexpr int kBlk = FMT4 == METIS_NVFP4 ? 16 : 32;
  float a = 0.f;
#pragma unroll
  for (int j = 0; j < kBlk; ++j) a = fmaxf(a, fabsf(v[j]));
  uint32_t code;
  float enc;
  if (FMT4 == METIS_NVFP4) {
    code = nv.code(a);
    enc = enc_tab[code];
  } else {
    int se = a == 0.f ? 0 : floor_log2(a) - 2;
    se = se < -127 ? -127 : se;
    code = a == 0.f ? 0u : static_cast<uint32_t>(se + 127);
    enc = pow2f(-se);
  }
  const bool none = FMT4 == METIS_NVFP4 ? code == 0u : a == 0.f;
#pragma unroll
  for (int k = 0; k < kBlk / 8; ++k) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __fmul_rn(v[8 * k + j], enc);
    w[k] = e2m1_pack8(q);
    if (none) w[k] = 0u;
  }
  return code;
}

// The tiles of a CTA: blockIdx.x, blockIdx.x + gridDim.x, ... of otiles rows of
// itiles, without a division a tile.
struct Tile {
  int o, i;           // outer and inner tile
  MDEV explicit Tile(const Act8QuantParams& p) {
    o = static_cast<int>(blockIdx.x) / p.itiles;
    i = static_cast<int>(blockIdx.x) - o * p.itiles;
  }
  MDEV void next(const Act8QuantParams& p) {
    o += p.step_o;
    i += p.step_i;
    if (i >= p.itiles) {
      i -= p.itiles;
      ++o;
    }
  }
};

// A CTA takes tiles of 128 outer indices x 8 blocks (axis 0) or 128 inner
// indices (axis 1).  The scales of such a tile are whole 512-byte chunks of the
// tensor-core layout: they are gathered in shared memory, padding included, and
// written as contiguous 16-byte words, so the call needs no clearing pass over
// them.  NVFP4's tensor maximum comes with the 8-bit copy, so there is no pass
// for it either.
//  * axis 1 (blocks along the columns): a thread takes 32 columns of a row.
//  * axis 0 (blocks along the rows): a warp takes one block of rows of 128
//    columns and reads 4 columns a lane, 128 bytes a row.  A row's 4 block
//    scales (the 8-bit blocks run along the columns) come as one byte a lane
//    for 8 rows, by shuffle.  The codes of a column are put together in shared
//    memory and leave as contiguous 64 (NVFP4) or 128 bytes a column.
// 16384 x 14336: MXINT8 to NVFP4 115 us along the rows, 107 along the columns (3.3 and
// 3.5 TB/s); MXFP8 to MXFP4 92 and 92 us (4.0 TB/s); 8192 x 4096 to NVFP4 21.0 and 20.1.
// Neither HBM nor the issue slots are full (57 to 62 % of those, by 16 warps an SM): the
// conversion, scaling, maximum and encoding of an element are scalar instructions that
// depend on one another, and a warp has few of them in flight.  24 warps an SM take
// longer, since 80 registers a thread spill (NVFP4 123 us along the rows, MXFP4 130).
template <int FMT8, int FMT4, int AXIS>
__global__ void __launch_bounds__(kThreads, 2) act8_quantize_kernel(Act8QuantParams p) {
  constexpr int kBlk = FMT4 == METIS_NVFP4 ? 16 : 32;
  constexpr int kTi = AXIS == 0 ? 8 * kBlk : 128;  // inner indices of a tile
  constexpr int kNb = kTi / kBlk;                  // FP4 blocks along a tile
  constexpr int kLdc = kTi / 2 + 8;                // bytes between columns of code_tile: 8-byte stores of 16 lanes
                                                   // then fall on different banks
  __shared__ float enc_tab[128];
  __shared__ __align__(16) uint8_t sc_tile[128 * kNb];
  __shared__ __align__(16) uint8_t code_tile[AXIS == 0 ? 128 * kLdc : 16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  wait_for_previous();
  float s_t = 1.f;
  if (FMT4 == METIS_NVFP4) {
    float m = 0.f;
    for (int i = tid; i < METIS_ACT8_AMAX; i += kThreads) m = fmaxf(m, p.in.amax[i]);
    s_t = nv_tensor_scale(cta_max(m));
    nv_enc_table(s_t, enc_tab);
    if (blockIdx.x == 0 && tid == 0) *p.tensor_scale = s_t;
    __syncthreads();
  }
  const NvScale nv(s_t);
  Tile tile(p);
  // axis 0: a warp's block of kBlk rows x 128 bytes of the next tile is on its way
  // (cp.async into the warp's own half of a two-stage ring) while it works on the
  // current one; its scale codes (row 8 j + lane / 4, 8-bit block lane & 3) wait in
  // registers
  constexpr int kRows = AXIS == 0 ? kBlk : 8;
  extern __shared__ __align__(16) uint8_t ring[];
  const uint32_t mine = smem_u32(ring) + warp * (2 * 128 * kRows);
  uint32_t sb[kRows / 8], next_sb[kRows / 8];
  auto fetch = [&](const Tile& t, int stage) {
    const int64_t r0 = static_cast<int64_t>(t.i) * kTi + warp * kBlk;
    const bool rows = t.o < p.otiles && r0 < p.inner;     // whole blocks: inner is a multiple of 32
    const int64_t c = static_cast<int64_t>(t.o) * 128 + 16 * (lane & 7), blk = static_cast<int64_t>(t.o) * 4 + (lane & 3);
    const uint8_t* src = p.in.codes + (r0 + (lane >> 3)) * p.in.ldc + c;
    const uint32_t dst = mine + stage * (128 * kRows) + 16 * lane;
#pragma unroll
    for (int j = 0; j < kRows / 4; ++j) {
      cp_async16(dst + 512 * j, src, rows && c < p.in.ldc ? 16 : 0);
      src += 4 * p.in.ldc;
    }
    cp_async_commit();
    const uint8_t* sp = p.in.scales + (r0 + (lane >> 2)) * p.in.blocks + blk;
#pragma unroll
    for (int j = 0; j < kRows / 8; ++j) next_sb[j] = rows && blk < p.in.blocks ? sp[8 * j * p.in.blocks] : 0u;
  };
  if constexpr (AXIS == 0) fetch(tile, 0);
  int stage = 0;
  for (; tile.o < p.otiles; tile.next(p)) {
    const int64_t o0 = static_cast<int64_t>(tile.o) * 128, i0 = static_cast<int64_t>(tile.i) * kTi;
    if constexpr (AXIS == 0) {
#pragma unroll
      for (int j = 0; j < kRows / 8; ++j) sb[j] = next_sb[j];
      // the other stage was read before the last tile's barriers
      Tile after = tile;
      after.next(p);
      fetch(after, stage ^ 1);
      cp_async_wait<1>();
      __syncwarp();                       // the warp's lanes read what the others copied
    }
    if (AXIS == 1) {
      // 512 units of 32 columns: a row's 4 units in adjacent lanes
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e = tid + kThreads * h, r = e >> 2, u = e & 3;
        const int64_t o = o0 + r, c = i0 + 32 * u;
        uint32_t sc4[2] = {0, 0};
        if (o < p.outer && c < p.inner) {
          const uint4* src = reinterpret_cast<const uint4*>(p.in.codes + o * p.in.ldc + c);
          const uint4 a = src[0], b = src[1];
          const float f = act8_factor<FMT8>(p.in.scales[o * p.in.blocks + (c >> 5)]);
          float v[32];
          const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) act8_elems4<FMT8>(w[j], v + 4 * j);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __fmul_rn(v[j], f);
          uint32_t pk[4];
#pragma unroll
          for (int b2 = 0; b2 < 32 / kBlk; ++b2)
            sc4[b2] = fp4_block<FMT4>(v + kBlk * b2, nv, enc_tab, pk + (kBlk / 8) * b2);
          *reinterpret_cast<uint4*>(p.codes + o * (p.inner / 2) + c / 2) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          if (p.scales_linear) {
#pragma unroll
            for (int b2 = 0; b2 < 32 / kBlk; ++b2)
              p.scales_linear[o * (p.inner / kBlk) + c / kBlk + b2] = static_cast<uint8_t>(sc4[b2]);
          }
        }
#pragma unroll
        for (int b2 = 0; b2 < 32 / kBlk; ++b2)
          sc_tile[tc_scale_offset(r, u * (32 / kBlk) + b2, kNb)] = static_cast<uint8_t>(sc4[b2]);
      }
    } else {
      // outer = columns of X, inner = its rows; a warp a block of rows
      constexpr int kQ = FMT4 == METIS_NVFP4 ? 4 : 2;    // columns whose values are held at once
      const int64_t c = o0 + 4 * lane;                   // this lane's 4 columns
      const int64_t r0 = i0 + warp * kBlk;
      uint32_t sc4 = 0;                                  // the 4 columns' scale codes
      uint32_t pk[4][kBlk / 8] = {};
      if (r0 < p.inner) {                                // whole blocks: inner is a multiple of 32
        float f[kBlk / 8];
#pragma unroll
        for (int j = 0; j < kBlk / 8; ++j) f[j] = act8_factor<FMT8>(sb[j]);
        const uint32_t at = mine + stage * (128 * kBlk) + 4 * lane;
#pragma unroll
        for (int q0 = 0; q0 < 4; q0 += kQ) {
          float v[kQ][kBlk];
#pragma unroll
          for (int j = 0; j < kBlk; ++j) {
            uint32_t raw;                                // 4 columns of row j
            lds<1>(at + 128 * j, &raw);
            const float fj = __shfl_sync(0xFFFFFFFFu, f[j >> 3], 4 * (j & 7) + (lane >> 3));
#pragma unroll
            for (int q = 0; q < kQ; ++q) v[q][j] = __fmul_rn(act8_elem_at<FMT8>(raw, q0 + q), fj);
          }
#pragma unroll
          for (int q = 0; q < kQ; ++q) {
            uint32_t code = fp4_block<FMT4>(v[q], nv, enc_tab, pk[q0 + q]);
            const int64_t cq = c + q0 + q;
            if (cq >= p.outer) code = 0u;                // padding columns: scale 0
            sc4 |= code << (8 * (q0 + q));
            if (p.scales_linear && cq < p.outer)
              p.scales_linear[cq * (p.inner / kBlk) + r0 / kBlk] = static_cast<uint8_t>(code);
          }
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        sc_tile[tc_scale_offset(4 * lane + q, warp, kNb)] = static_cast<uint8_t>(sc4 >> (8 * q));
        uint8_t* dst = code_tile + (32 * q + lane) * kLdc + warp * (kBlk / 2);   // column 4 lane + q
#pragma unroll
        for (int w = 0; w < kBlk / 8; w += 2) *reinterpret_cast<uint2*>(dst + 4 * w) = make_uint2(pk[q][w], pk[q][w + 1]);
      }
    }
    __syncthreads();
    if (AXIS == 0) {
      constexpr int kW = kTi / 32;                       // 16-byte words a column (32 rows each)
#pragma unroll
      for (int h = 0; h < 128 * kW / kThreads; ++h) {
        const int e = tid + kThreads * h, cc = e / kW, w = e % kW;
        const int64_t o = o0 + cc, r = i0 + 32 * w;
        if (o < p.outer && r < p.inner) {
          const uint2* q = reinterpret_cast<const uint2*>(code_tile + (32 * (cc & 3) + (cc >> 2)) * kLdc + 16 * w);
          *reinterpret_cast<uint4*>(p.codes + o * (p.inner / 2) + r / 2) = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
        }
      }
    }
    if (tid < 8 * kNb)   // 128 kNb bytes of scales: contiguous chunks of the layout
      *reinterpret_cast<uint4*>(p.scales + tc_scale_offset(o0, i0 / kBlk, p.scale_cols) + 16 * tid) =
          *reinterpret_cast<const uint4*>(sc_tile + 16 * tid);
    __syncthreads();
    stage ^= 1;
  }
  if constexpr (AXIS == 0) cp_async_wait<0>();
}

template <int FMT8, int FMT4, int AXIS>
void quantize_axis(const Act8QuantParams& params, int num_sms, cudaStream_t s) {
  Act8QuantParams p = params;
  constexpr int kSmem = AXIS == 0 ? 8 * 2 * 128 * (FMT4 == METIS_NVFP4 ? 16 : 32) : 0;   // the warps' rings
  auto* kernel = act8_quantize_kernel<FMT8, FMT4, AXIS>;
  if (AXIS == 0) ensure_smem(reinterpret_cast<const void*>(kernel), kSmem);
  static const int per_sm = occupancy(reinterpret_cast<const void*>(kernel), kSmem);
  const int grid = grid_for(per_sm, static_cast<int64_t>(p.otiles) * p.itiles, num_sms);
  p.step_o = grid / p.itiles;
  p.step_i = grid % p.itiles;
  launch_dependent(kernel, dim3(static_cast<unsigned>(grid)), kThreads, kSmem, 1, s, p);
}

template <int FMT8, int FMT4>
void quantize_t(const Act8QuantParams& p, int axis, int num_sms, cudaStream_t s) {
  axis == 1 ? quantize_axis<FMT8, FMT4, 1>(p, num_sms, s) : quantize_axis<FMT8, FMT4, 0>(p, num_sms, s);
}

}  // namespace

void launch_act8_save(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld, const Act8View& out,
                      int num_sms, cudaStream_t s) {
  const bool i8 = out.fmt == METIS_MXINT8;
  if (dtype == METIS_BF16) {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(X);
    i8 ? save_t<METIS_MXINT8>(x, rows, cols, ld, out, num_sms, s)
       : save_t<METIS_MXFP8>(x, rows, cols, ld, out, num_sms, s);
  } else {
    const float* x = static_cast<const float*>(X);
    i8 ? save_t<METIS_MXINT8>(x, rows, cols, ld, out, num_sms, s)
       : save_t<METIS_MXFP8>(x, rows, cols, ld, out, num_sms, s);
  }
}

void launch_act8_restore(const Act8View& in, int64_t rows, int64_t cols, void* Y, int dtype, int64_t ld, int num_sms,
                         cudaStream_t s) {
  const bool i8 = in.fmt == METIS_MXINT8;
  if (dtype == METIS_BF16) {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(Y);
    i8 ? restore_t<METIS_MXINT8>(in, rows, cols, y, ld, num_sms, s)
       : restore_t<METIS_MXFP8>(in, rows, cols, y, ld, num_sms, s);
  } else {
    float* y = static_cast<float*>(Y);
    i8 ? restore_t<METIS_MXINT8>(in, rows, cols, y, ld, num_sms, s)
       : restore_t<METIS_MXFP8>(in, rows, cols, y, ld, num_sms, s);
  }
}

void launch_act8_quantize(const Act8View& in, int64_t rows, int64_t cols, int axis, const metis_fp4_tensor* out,
                          int num_sms, cudaStream_t s) {
  Act8QuantParams p{};
  p.in = in;
  p.rows = rows;
  p.cols = cols;
  p.outer = out->outer;
  p.inner = out->inner;
  p.scale_cols = tc_scale_cols(out->fmt, out->inner);
  p.codes = out->codes;
  p.scales = out->scales;
  p.scales_linear = out->scales_linear;
  p.tensor_scale = out->tensor_scale;
  p.otiles = static_cast<int>(tc_scale_rows(p.outer) / 128);     // (outer < 2^37: checked by the entry point)
  const int blk = out->fmt == METIS_NVFP4 ? 16 : 32;
  p.itiles = static_cast<int>(p.scale_cols * blk / (axis == 0 ? 8 * blk : 128));   // the padded scale columns too
  const bool i8 = in.fmt == METIS_MXINT8, nv = out->fmt == METIS_NVFP4;
  if (i8)
    nv ? quantize_t<METIS_MXINT8, METIS_NVFP4>(p, axis, num_sms, s)
       : quantize_t<METIS_MXINT8, METIS_MXFP4>(p, axis, num_sms, s);
  else
    nv ? quantize_t<METIS_MXFP8, METIS_NVFP4>(p, axis, num_sms, s)
       : quantize_t<METIS_MXFP8, METIS_MXFP4>(p, axis, num_sms, s);
}

}  // namespace metis
