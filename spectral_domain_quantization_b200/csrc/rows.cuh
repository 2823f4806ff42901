// Consecutive elements of a matrix row ("units") in registers, for rows that start
// anywhere.  Nothing outside the matrix is touched: what reaches over its first or
// last byte is read by element.
//
// In registers (UnitLoad, store_unit): a warp's lanes hold consecutive units of 8.
// Where every row starts on a 16-byte boundary a unit is one (bf16) or two (f32)
// 16-byte words.  Where it does not, the lane still loads the aligned 16-byte chunks
// from the one its first element lies in: the bytes behind its own chunks are the next
// lane's first chunk (a shuffle; the last lane of a row's lanes loads that chunk
// itself), and the unit is cut out of the two by a byte shift.  A store goes the other
// way round: a lane writes the aligned chunk made of its predecessor's last bytes and
// its own first; only the two ends of the lanes' run are written by element.  8192 x
// 4096 bf16 with rows 4097 apart go into 8 bits in 35 us so and come back in 39 (18.3
// and 17.9 with rows 4096 apart): the shuffles and shifts are what is left.
//
// In shared memory (UnitSlot, RowImage): rows on their way in, copied asynchronously.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace metis {

// E elements as stored.
template <typename T, int E = 8>
struct Unit {
  static constexpr int kWords = E * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
  MDEV void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  MDEV void get(float* v) const {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) v[i] = __uint_as_float(w[i]);
    }
  }
  MDEV void put(const float* v) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = __float_as_uint(v[i]);
    }
  }
  // element j as stored
  MDEV T elem(int j) const {
    if constexpr (sizeof(T) == 2)
      return __ushort_as_bfloat16(static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1))));
    else
      return __uint_as_float(w[j]);
  }
  // elements before `from` and from `to` on to zero
  MDEV void keep(int from, int to) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 2) {
        if (2 * i < from || 2 * i >= to) w[i] &= 0xFFFF0000u;
        if (2 * i + 1 < from || 2 * i + 1 >= to) w[i] &= 0xFFFFu;
      } else {
        if (i < from || i >= to) w[i] = 0u;
      }
    }
  }
  // as one word at an address aligned to it
  MDEV void store(T* p) const {
    if constexpr (kWords == 2) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
};

// The bytes of a matrix.
struct Span {
  uintptr_t lo, hi;
};

template <typename T>
MDEV Span span_of(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  Span s;
  s.lo = reinterpret_cast<uintptr_t>(p);
  s.hi = s.lo + static_cast<uintptr_t>((rows - 1) * ld + cols) * sizeof(T);
  return s;
}

template <typename T>
MDEV uint32_t bits_of(T v) {
  if constexpr (sizeof(T) == 2)
    return __bfloat16_as_ushort(v);
  else
    return __float_as_uint(v);
}

// The aligned chunk at `a`; what lies outside the matrix reads 0.
template <typename T>
MDEV void load_chunk(uintptr_t a, const Span& s, uint32_t* w) {
  if (a >= s.lo && a + 16 <= s.hi) {
    const uint4 q = *reinterpret_cast<const uint4*>(a);
    w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = 0u;
#pragma unroll
      for (int h = 0; h < 4 / static_cast<int>(sizeof(T)); ++h) {
        const uintptr_t e = a + 4 * i + h * sizeof(T);
        if (e >= s.lo && e < s.hi) w[i] |= bits_of(*reinterpret_cast<const T*>(e)) << (16 * h);
      }
    }
  }
}

// in[0 .. N + 3] -> out[0 .. N - 1], from byte `sh` (0 .. 15, a multiple of
// sizeof(T)) of in.
template <typename T, int N>
MDEV void cut(const uint32_t* in, int sh, uint32_t* out) {
  uint32_t a[N + 2], b[N + 1];
#pragma unroll
  for (int i = 0; i < N + 2; ++i) a[i] = (sh & 8) ? in[i + 2] : in[i];
#pragma unroll
  for (int i = 0; i < N + 1; ++i) b[i] = (sh & 4) ? a[i + 1] : a[i];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (sizeof(T) == 2)
      out[i] = (sh & 2) ? __byte_perm(b[i], b[i + 1], 0x5432) : b[i];
    else
      out[i] = b[i];
  }
}

// A unit on its way in.  start() issues the loads, finish() (by whole warps)
// gives the unit; `n`: elements left in the row from the unit's first (8 or more:
// whole; 0 or less: none), `last`: no lane behind this one holds the row's next
// unit.
template <typename T, bool AL>
struct UnitLoad;

template <typename T>
struct UnitLoad<T, true> {
  Unit<T> u;
  MDEV void start(const T* p, int n, bool, const Span&) {
    if (n >= 8) {
#pragma unroll
      for (int i = 0; i < Unit<T>::kWords / 4; ++i) {
        const uint4 q = reinterpret_cast<const uint4*>(p)[i];
        u.w[4 * i] = q.x; u.w[4 * i + 1] = q.y; u.w[4 * i + 2] = q.z; u.w[4 * i + 3] = q.w;
      }
    } else {
      u.zero();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) {
          if constexpr (sizeof(T) == 2)
            u.w[j >> 1] |= bits_of(p[j]) << (16 * (j & 1));
          else
            u.w[j] = bits_of(p[j]);
        }
    }
  }
  MDEV Unit<T> finish(int, bool) const { return u; }
};

template <typename T>
struct UnitLoad<T, false> {
  static constexpr int kN = Unit<T>::kWords;
  uint32_t c[kN], x[4];
  int sh;
  MDEV void start(const T* p, int n, bool last, const Span& s) {
    const uintptr_t addr = reinterpret_cast<uintptr_t>(p);
    sh = static_cast<int>(addr & 15u);
    const int se = sh / static_cast<int>(sizeof(T));
    constexpr int kE = 16 / static_cast<int>(sizeof(T));
#pragma unroll
    for (int i = 0; i < kN; ++i) c[i] = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = 0u;
#pragma unroll
    for (int k = 0; k < kN / 4; ++k)
      if (n + se > k * kE) load_chunk<T>(addr - sh + 16 * k, s, c + 4 * k);
    if (last && sh != 0 && n + se > 8) load_chunk<T>(addr - sh + 4 * kN, s, x);
  }
  MDEV Unit<T> finish(int n, bool last) const {
    uint32_t in[kN + 4];
#pragma unroll
    for (int i = 0; i < kN; ++i) in[i] = c[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, c[i], 1);
      in[kN + i] = last ? x[i] : next;
    }
    Unit<T> u;
    cut<T, kN>(in, sh, u.w);
    if (n < 8) u.keep(0, n);
    return u;
  }
};

// A unit on its way out, by whole warps.  `first`: no lane before this one holds
// the row's previous unit.
template <typename T>
MDEV void store_unit(T* p, const Unit<T>& u, int n, bool first, bool last) {
  constexpr int kN = Unit<T>::kWords;
  constexpr int kE = 16 / static_cast<int>(sizeof(T));
  const uintptr_t addr = reinterpret_cast<uintptr_t>(p);
  const int sh = static_cast<int>(addr & 15u), se = sh / static_cast<int>(sizeof(T));
  uint32_t in[kN + 4], out[kN];
#pragma unroll
  for (int i = 0; i < 4; ++i) in[i] = __shfl_up_sync(0xFFFFFFFFu, u.w[kN - 4 + i], 1);
#pragma unroll
  for (int i = 0; i < kN; ++i) in[4 + i] = u.w[i];
  // byte 0 of the chunks is byte 16 - sh of `in` (all 16 of the predecessor's
  // bytes are behind it when sh == 0)
  if (sh == 0) {
#pragma unroll
    for (int i = 0; i < kN; ++i) out[i] = u.w[i];
  } else {
    cut<T, kN>(in, 16 - sh, out);
  }
  bool whole[kN / 4];                     // chunk k is written as one word
#pragma unroll
  for (int k = 0; k < kN / 4; ++k) {
    whole[k] = n >= (k + 1) * kE - se && (k > 0 || sh == 0 || !first);
    if (whole[k])
      *reinterpret_cast<uint4*>(addr - sh + 16 * k) =
          make_uint4(out[4 * k], out[4 * k + 1], out[4 * k + 2], out[4 * k + 3]);
  }
  const bool next_whole = !last && n - 8 >= kE - se;   // the next lane writes this one's last elements
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int k = (j + se) / kE;          // the chunk of element j
    bool done = next_whole;
#pragma unroll
    for (int q = 0; q < kN / 4; ++q)
      if (k == q) done = whole[q];
    if (j < n && !done) p[j] = u.elem(j);
  }
}

MDEV float load_any(const void* p, int dtype, int64_t i) { return load_elem(p, dtype, i); }

MDEV void store_any(void* p, int dtype, int64_t i, float v) {
  if (dtype == METIS_BF16)
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<float*>(p)[i] = v;
}

// ---------------------------------------------------------------------------
// units that wait in shared memory
// ---------------------------------------------------------------------------

MDEV void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
MDEV void cp_async8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
MDEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
MDEV void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
MDEV void lds16(uint32_t a, uint32_t* w) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(a)
               : "memory");
}

MDEV void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// B bytes (4, 8 or 16), zeros instead where `on` is false (the address is then not followed).
template <int B>
MDEV void cp_async(uint32_t dst, const void* src, bool on) {
  if constexpr (B == 16)
    cp_async16(dst, src, on ? 16 : 0);
  else if constexpr (B == 8)
    cp_async8(dst, src, on ? 8 : 0);
  else
    cp_async4(dst, src, on ? 4 : 0);
}
template <int W>
MDEV void lds(uint32_t a, uint32_t* w) {
  if constexpr (W == 4) {
    lds16(a, w);
  } else if constexpr (W == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
  } else {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(a) : "memory");
  }
}

template <typename T>
MDEV float lds_elem(uint32_t a) {
  if constexpr (sizeof(T) == 2) {
    uint16_t h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(a) : "memory");
    return __bfloat162float(__ushort_as_bfloat16(h));
  } else {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(a) : "memory");
    return f;
  }
}

// How the rows of a matrix lie.
enum RowMode {
  kAligned = 0,  // every unit of a row is one aligned word, and there is no part of a unit
  kPhase = 1,    // rows start anywhere, but all matrices of the call at the same element of a 16-byte (bf16: 8
                 // elements) period: a thread's columns are shifted so that its units are aligned words, a group
                 // of threads takes rows of one shift only, and only a row's first and last unit are in part outside
  kAny = 2       // rows start anywhere: a warp's lanes take neighbouring elements, one at a time (RowImage)
};

// A unit's place in a stage of a ring: a thread copies what it will read itself
// (cp.async), so the ring needs no barrier, and as many rows are on their way as
// it has stages, whatever the registers hold.  One word of a thread, kThreads of
// them in a row.
template <typename T, int E, int MODE, int kThreads>
struct UnitSlot {
  static constexpr int kWord = E * static_cast<int>(sizeof(T));
  static constexpr int kBytes = kWord * kThreads;
  // `p`: the unit's first element; it has `whole` columns of the row, or `some`.
  // `inside`: no word of the row reaches over the matrix
  static MDEV void start(uint32_t base, int tid, const T* p, bool whole, bool some, bool inside, const Span& s) {
    const uint32_t dst = base + kWord * tid;
    if (MODE == kAligned || inside) {
      cp_async<kWord>(dst, p, some);
    } else {
      const uintptr_t a = reinterpret_cast<uintptr_t>(p);
      if (whole || !some || (a >= s.lo && a + kWord <= s.hi)) {
        cp_async<kWord>(dst, some ? p : reinterpret_cast<const T*>(s.lo & ~uintptr_t{15}), some);
      } else {                               // over the matrix's first or last byte
#pragma unroll
        for (int i = 0; i < kWord / 4; ++i) {
          uint32_t w = 0u;
#pragma unroll
          for (int h = 0; h < 4 / static_cast<int>(sizeof(T)); ++h) {
            const uintptr_t e = a + 4 * i + h * sizeof(T);
            if (e >= s.lo && e < s.hi) w |= bits_of(*reinterpret_cast<const T*>(e)) << (16 * h);
          }
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + 4 * i), "r"(w) : "memory");
        }
      }
    }
  }
  static MDEV Unit<T, E> finish(uint32_t base, int tid) {
    Unit<T, E> u;
    lds<Unit<T, E>::kWords>(base + kWord * tid, u.w);
    return u;
  }
  // element j of thread tid's unit, and zeros in the place of the unit
  static MDEV float elem(uint32_t base, int tid, int j) {
    return lds_elem<T>(base + kWord * tid + static_cast<uint32_t>(sizeof(T)) * j);
  }
  static MDEV void clear(uint32_t base, int tid) {
#pragma unroll
    for (int i = 0; i < kWord / 8; ++i)
      asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(base + kWord * tid + 8 * i), "r"(0u) : "memory");
  }
};

// kAny: the SPAN * NV elements of a row that SPAN lanes share, as they lie in memory
// from the 16-byte chunk with the first of them on.  Lane t reads the elements
// t, t + SPAN, ...: neighbouring lanes neighbouring elements, whatever the row's
// alignment.  By whole warps; what one lane copied another reads, so a __syncwarp
// goes before end(), between end() and elem(), and before the stage is copied to again.
template <typename T, int SPAN, int NV>
struct RowImage {
  static constexpr int kE = 16 / static_cast<int>(sizeof(T));
  static constexpr int kChunks = NV / kE;                          // of a lane; one more for the last element
  static constexpr int kOne = 16 * (SPAN * kChunks + 1);
  static constexpr int kBytes = kOne * (32 / SPAN);                // of a warp
  static_assert(NV % kE == 0 && SPAN >= kE - 1);
  // `p`: the first element; `n` of them (0 or less: none) are the row's
  static MDEV void start(uint32_t base, int lane, const T* p, int n, const Span& s) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p) & ~uintptr_t{15};
    const uintptr_t end = n > 0 ? reinterpret_cast<uintptr_t>(p + n) : 0;
    const int t = lane % SPAN;
    base += kOne * (lane / SPAN);
#pragma unroll
    for (int k = 0; k < kChunks; ++k) chunk(base, a, t + SPAN * k, end, s);
    if (t == 0) chunk(base, a, SPAN * kChunks, end, s);
  }
  // zeros from element n on, as far as the chunk with it reaches
  static MDEV void end(uint32_t base, int lane, const T* p, int n) {
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) + n * static_cast<int>(sizeof(T));
    const int at = off + lane % SPAN * static_cast<int>(sizeof(T));
    if (n > 0 && n < SPAN * NV && at < (off + 15) / 16 * 16) put(base + kOne * (lane / SPAN) + at);
  }
  // the address of lane t's first element; the next ones are SPAN elements apart
  static MDEV uint32_t place(uint32_t base, int lane, const T* p) {
    return base + kOne * (lane / SPAN) + static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u) +
           static_cast<uint32_t>(sizeof(T)) * (lane % SPAN);
  }
  static MDEV float elem(uint32_t place, int i) {
    return lds_elem<T>(place + static_cast<uint32_t>(sizeof(T)) * SPAN * i);
  }

 private:
  // the aligned chunk k from `a` on, zeros where it is not wanted or lies outside
  static MDEV void chunk(uint32_t base, uintptr_t a, int k, uintptr_t end, const Span& s) {
    a += 16 * k;
    const uint32_t dst = base + 16 * k;
    if (a < end && a < s.lo) {              // the matrix's first chunk: by element
      uint32_t w[4];
      load_chunk<T>(a, s, w);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                   : "memory");
    } else {
      const bool want = a < end;
      const int bytes = want ? (s.hi - a < 16 ? static_cast<int>(s.hi - a) : 16) : 0;
      cp_async16(dst, reinterpret_cast<const void*>(want ? a : s.lo & ~uintptr_t{15}), bytes);
    }
  }
  static MDEV void put(uint32_t a) {
    if constexpr (sizeof(T) == 2)
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(static_cast<uint16_t>(0)) : "memory");
    else
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(0u) : "memory");
  }
};

}  // namespace metis
