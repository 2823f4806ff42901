// One block of an activation kept in 8 bits: 32 consecutive columns under one
// E8M0 scale (OCP MX v1.0 element types).
//
//   a = max |x| of the block.
//   a not finite: scale code 255, codes 0 (every value of the block reads NaN)
//   a == 0:       scale code 0, codes 0
//   MXINT8: se = clamp(floor(log2 a), -120, 127);
//           code = rne(x 2^(6 - se)) clamped to +-127, value = code 2^(se - 6)
//   MXFP8:  se = clamp(floor(log2 a) - 8, -126, 127);
//           code = E4M3 rne(x 2^-se) saturating at 448, value = e4m3 2^se
//   scale code = se + 127.
// Every scaling is by a normal power of two, so the one rounding is the
// element's.  (A lower clamp than the E8M0 range's, so that no factor is
// subnormal: blocks whose maximum is under 2^-120 keep an absolute step.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace metis {

// max that returns NaN if either operand is NaN
MDEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Scale code of a block with maximum a >= 0 (or NaN), and 2^(6 - se) or 2^-se.
template <int FMT>
MDEV uint32_t act8_scale(float a, float& enc) {
  const int e = static_cast<int>(__float_as_uint(a) >> 23) - 127;  // floor(log2 a), -127 for subnormals and 0
  const int se = FMT == METIS_MXINT8 ? max(e, -120) : max(e - 8, -126);
  enc = __uint_as_float(static_cast<uint32_t>(FMT == METIS_MXINT8 ? 133 - se : 127 - se) << 23);
  if (e == 128) return 255u;  // infinity or NaN
  return a == 0.f ? 0u : static_cast<uint32_t>(se + 127);
}

// 4 scaled values (x enc) -> 4 code bytes, element i in byte i.  `clamp`: the
// block's maximum rounds to 128 (MXINT8); without it no value does.
template <int FMT>
MDEV uint32_t act8_pack4(const float* q, bool clamp) {
  if (FMT == METIS_MXINT8) {
    // 1.5 2^23 + q rounds q to the nearest integer, ties to even, and leaves
    // its two's complement in the low byte
    uint32_t b[4];
    if (clamp) {
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(fminf(fmaxf(q[i], -127.f), 127.f) + 12582912.f);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(q[i] + 12582912.f);
    }
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
  uint16_t h[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(q[2 * i + 1]), "f"(q[2 * i]));
  return static_cast<uint32_t>(h[0]) | (static_cast<uint32_t>(h[1]) << 16);
}

// NV units of E columns a thread, each unit's block of 32 columns in 32 / E
// adjacent lanes (by whole warps): the units' code words, and the scale code of a
// block.  `top` follows the largest finite maximum; what 8 bits hold of it is the
// tensor's largest magnitude, since the rounding of a block's maximum grows with the
// maximum.
//
// With as many units as lanes (NV == 32 / E) the maxima are reduced while they are
// dealt out: lane t of the group ends with unit t's block, makes its scale alone and
// hands the factor round, so the per-block work is done once, not in every lane.
// Returns the scale code of the block of unit t, t the lane in the group.
template <int E, int NV>
constexpr bool act8_dealt = NV == 32 / E;

template <int FMT, int E, int NV>
MDEV uint32_t act8_blocks(const float (*v)[E], uint32_t (*codes)[E / 4], float& top) {
  constexpr int kL = 32 / E;
  static_assert(act8_dealt<E, NV>);
  const int t = threadIdx.x & (kL - 1);
  float a[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    a[i] = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) a[i] = max_nan(a[i], fabsf(v[i][j]));
  }
  // step s: a lane keeps the units whose bit s is its own, and gets their other half
#pragma unroll
  for (int n = NV / 2; n > 0; n >>= 1) {
    const bool up = t & n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? a[i + n] : a[i], give = up ? a[i] : a[i + n];
      a[i] = max_nan(keep, __shfl_xor_sync(0xFFFFFFFFu, give, n));
    }
  }
  float enc;
  const uint32_t sc = act8_scale<FMT>(a[0], enc);
  if (sc != 255u) top = fmaxf(top, a[0]);
  // a block that rounds to 128 (MXINT8) or is not finite takes the careful way
  const bool odd = sc == 255u || (FMT == METIS_MXINT8 && a[0] * enc > 127.f);
  const bool careful = __any_sync(0xFFFFFFFFu, odd);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int from = (threadIdx.x & 31 & ~(kL - 1)) + i;
    const float f = __shfl_sync(0xFFFFFFFFu, enc, from);
    float q[E];
#pragma unroll
    for (int j = 0; j < E; ++j) q[j] = v[i][j] * f;
    if (careful) {
      const bool none = __shfl_sync(0xFFFFFFFFu, sc, from) == 255u;
#pragma unroll
      for (int k = 0; k < E / 4; ++k) codes[i][k] = none ? 0u : act8_pack4<FMT>(q + 4 * k, true);
    } else {
#pragma unroll
      for (int k = 0; k < E / 4; ++k) codes[i][k] = act8_pack4<FMT>(q + 4 * k, false);
    }
  }
  return sc;
}

// One unit, its block in 32 / E adjacent lanes (by whole warps); every lane gets the
// scale code.
template <int FMT, int E>
MDEV uint32_t act8_block(const float* v, uint32_t* codes, float& top) {
  float a = 0.f;
#pragma unroll
  for (int j = 0; j < E; ++j) a = max_nan(a, fabsf(v[j]));
#pragma unroll
  for (int off = 1; off < 32 / E; off <<= 1) a = max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, off));
  float enc, q[E];
  const uint32_t sc = act8_scale<FMT>(a, enc);
#pragma unroll
  for (int j = 0; j < E; ++j) q[j] = v[j] * enc;
  const bool clamp = a * enc > 127.f;
#pragma unroll
  for (int k = 0; k < E / 4; ++k) codes[k] = sc == 255u ? 0u : act8_pack4<FMT>(q + 4 * k, clamp);
  if (sc != 255u) top = fmaxf(top, a);
  return sc;
}

// One scaled value -> its code byte.
template <int FMT>
MDEV uint32_t act8_code(float q) {
  if (FMT == METIS_MXINT8) return __float_as_uint(fminf(fmaxf(q, -127.f), 127.f) + 12582912.f) & 0xFFu;
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.f), "f"(q));
  return h & 0xFFu;
}

// The factor of a block's elements: 2^(se - 6) or 2^se; NaN for code 255.
// (A scale code below the codec's smallest has elements 0 only.)
template <int FMT>
MDEV float act8_factor(uint32_t sc) {
  const uint32_t bits = FMT == METIS_MXINT8 ? (max(sc, 7u) - 6u) << 23 : sc << 23;
  return __uint_as_float(sc == 255u ? 0x7FC00000u : bits);
}

// Element values (not yet scaled) of the 4 code bytes in w.
template <int FMT>
MDEV void act8_elems4(uint32_t w, float* v) {
  if (FMT == METIS_MXINT8) {
    // 2^23 + (code + 128) as a float, minus 2^23 + 128
    const uint32_t u = w ^ 0x80808080u;
    v[0] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7650)) - 8388736.f;
    v[1] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7651)) - 8388736.f;
    v[2] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7652)) - 8388736.f;
    v[3] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7653)) - 8388736.f;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h2;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(w >> (16 * i))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

// Element value (not yet scaled) of byte q of a word.
template <int FMT>
MDEV float act8_elem_at(uint32_t w, int q) {
  if (FMT == METIS_MXINT8)
    return __uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4B000000u, 0x7650u + q)) - 8388736.f;
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(w >> (8 * (q & 2)))));
  const __half2 h = *reinterpret_cast<const __half2*>(&h2);
  return (q & 1) ? __high2float(h) : __low2float(h);
}

template <int FMT>
MDEV float act8_elem(uint32_t byte) {
  if (FMT == METIS_MXINT8) return static_cast<float>(static_cast<int8_t>(byte));
  float v[4];
  act8_elems4<FMT>(byte, v);
  return v[0];
}

// The largest magnitude held of blocks whose largest finite maximum is a.
template <int FMT>
MDEV float act8_held(float a) {
  float enc;
  const uint32_t sc = act8_scale<FMT>(a, enc);
  return act8_elem<FMT>(act8_code<FMT>(a * enc)) * act8_factor<FMT>(sc);
}

// The calling CTA's maximum m (0 or more, valid in thread 0) into its slots of
// the tensor's maximum: CTA b owns slots b, b + gridDim.x, ...; all but the
// first hold 0.  gridDim.x <= METIS_ACT8_AMAX.
MDEV void act8_write_amax(float* amax, float m) {
  if (threadIdx.x != 0) return;
  for (int i = blockIdx.x; i < METIS_ACT8_AMAX; i += gridDim.x) {
    amax[i] = m;
    m = 0.f;
  }
}

}  // namespace metis
