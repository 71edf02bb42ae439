// pieces.hpp -- rows of floats of any length and element alignment, read and written in
// pieces of P consecutive elements a lane.  A whole piece is one wide access (the device
// takes them at any element's address).  The last piece of a row that is no multiple of P begins
// earlier, over elements of the piece before it; only a row shorter than a piece goes element by
// element.
#pragma once
#include "common.hpp"
#include "rows.hpp"

namespace iq4 {

inline int type_bytes(int t) { return t == kF32 ? 4 : 2; }

// Rows of more bytes than this are read and written past the L2 (non-temporal): each is used once, and
// they would only push each other out of it and of the memory-side cache behind it.
constexpr int64_t kStreamBytes = 64 << 20;

// Division of n < 2^31 by a fixed number d, the pieces of a row (1 .. 2^30): with 2^l >= d and m = floor(2^(31 + l) / d) + 1
// (below 2^32), m d - 2^(31 + l) is at most 2^l, so that floor(n m / 2^(31 + l)) is n / d.
struct Pieces {
  uint32_t n, m, l;
  explicit Pieces(uint32_t d) : n(d), l(0) {
    while (((uint64_t)1 << l) < d) ++l;
    m = (uint32_t)(((uint64_t)1 << (31 + l)) / d) + 1;
  }
#ifdef __HIPCC__
  __device__ __forceinline__ uint32_t row(uint32_t i) const { return __umulhi(i << 1, m) >> l; }
#endif
};
// Rows of a launch: below 2^31 threads, those of the last workgroup included.
inline int64_t rows_a_launch(const Pieces& p) { return (((int64_t)1 << 31) - 256) / p.n; }

#ifdef __HIPCC__
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

// (Not templates over the vector: a type passed as a template argument loses its alignment.)
template <bool STREAM>
__device__ __forceinline__ u32x4 get16(const void* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const u32x4_any*>(p));
  return *static_cast<const u32x4_any*>(p);
}
template <bool STREAM>
__device__ __forceinline__ u32x2 get8(const void* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const u32x2_any*>(p));
  return *static_cast<const u32x2_any*>(p);
}
template <bool STREAM>
__device__ __forceinline__ void put16(void* p, u32x4 v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<u32x4_any*>(p));
  else *static_cast<u32x4_any*>(p) = v;
}
template <bool STREAM>
__device__ __forceinline__ void put8(void* p, u32x2 v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<u32x2_any*>(p));
  else *static_cast<u32x2_any*>(p) = v;
}

// Piece q of a row of n elements: the first element, how many there are (P unless the row is shorter), and
// how many of them are the piece's before it too.
struct Piece {
  int at, left, twice;
};
template <int P>
__device__ __forceinline__ Piece piece_of(uint32_t q, int64_t n) {  // n <= 2^20
  const int at = (int)q * P, end = at + P - (int)n, over = end > 0 ? end : 0;
  return over == 0 || n < P ? Piece{at, P - over, 0} : Piece{at - over, P, over};
}

// Elements at .. at + P - 1 of a row, `left` of which exist (the others are zero), as binary32.
template <int TYPE, int P, bool STREAM = false>
__device__ __forceinline__ void load_piece(const void* row, int at, int left, float (&v)[P]) {
  if constexpr (TYPE == kF32) {
    const float* p = static_cast<const float*>(row) + at;
    if (left >= P) {
#pragma unroll
      for (int q = 0; q < P / 4; ++q) {
        const u32x4 w = get16<STREAM>(p + 4 * q);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * q + i] = __uint_as_float(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = i < left ? p[i] : 0.f;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(row) + at;
    uint32_t w[P / 2];
    if (left >= P) {
      if constexpr (P == 8) {
        const u32x4 x = get16<STREAM>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = x[i];
      } else {
        const u32x2 x = get8<STREAM>(p);
        w[0] = x[0], w[1] = x[1];
      }
    } else {
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        w[i] = 2 * i < left ? p[2 * i] : 0u;
        if (2 * i + 1 < left) w[i] |= (uint32_t)p[2 * i + 1] << 16;
      }
    }
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      if constexpr (TYPE == kF16) {
        v[2 * i] = h2f((uint16_t)(w[i] & 0xFFFFu));
        v[2 * i + 1] = h2f((uint16_t)(w[i] >> 16));
      } else {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
}

// The same elements rounded (once, to nearest even) to TYPE and written.
template <int TYPE, int P, bool STREAM = false>
__device__ __forceinline__ void store_piece(void* row, int at, int left, const float (&v)[P]) {
  if constexpr (TYPE == kF32) {
    float* p = static_cast<float*>(row) + at;
    if (left >= P) {
#pragma unroll
      for (int q = 0; q < P / 4; ++q) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[4 * q + i]);
        put16<STREAM>(p + 4 * q, w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (i < left) p[i] = v[i];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(row) + at;
    uint32_t w[P / 2];
#pragma unroll
    for (int i = 0; i < P / 2; ++i) w[i] = pack2<TYPE>(v[2 * i], v[2 * i + 1]);
    if (left >= P) {
      if constexpr (P == 8) put16<STREAM>(p, u32x4{w[0], w[1], w[2], w[3]});
      else put8<STREAM>(p, u32x2{w[0], w[1]});
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (i < left) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
  }
}
#endif  // __HIPCC__

}  // namespace iq4
