// rows.hpp -- rows of activations held in 8 or 4 bits with a scale per 32 elements: the
// formats' arithmetic (shared by the quantiser and the norm, rows.hip) and the launchers'
// arguments.
//
// MXFP4 / MXFP8 (OCP microscaling): a block's scale is the power of two 2^(s - 127),
// s = max(E - emax, 0) with E the biased binary32 exponent of the block's largest
// magnitude and emax = 2 (E2M1, largest value 6) or 8 (E4M3, largest value 448); an
// element is x * 2^(127 - s), exact, rounded to nearest even and clamped to the largest
// value.  A block that holds an infinity or a NaN gets s = 255 (NaN) and zero codes.
// Q8_1: as iq4_quantize_q8_1 (qmv.hip); such a block gets d = NaN and zero codes.
#pragma once
#include "common.hpp"

namespace iq4 {

enum RowFormat { kRowsMxfp4 = 0, kRowsMxfp8 = 1, kRowsQ8_1 = 2 };
enum ElemType { kF32 = 0, kF16 = 1, kBF16 = 2 };

// Bytes of one row's codes and scales.  MX rows are padded with zero codes (and zero
// scale bytes) to the product kernel's steps: 128 elements of codes, 512 of scales.
inline int64_t rows_code_bytes(int fmt, int64_t k) {
  const int64_t kp = (k + 127) / 128 * 128;
  return fmt == kRowsMxfp4 ? kp / 2 : fmt == kRowsMxfp8 ? kp : k;
}
inline int64_t rows_scale_bytes(int fmt, int64_t k) { return fmt == kRowsQ8_1 ? k / 16 : (k + 511) / 512 * 16; }

struct RowsOut {  // codes and scales of quantised rows (strides in bytes)
  uint8_t* codes;
  int64_t ldq;
  uint8_t* scales;
  int64_t lds;
};

struct RowsIn {
  const uint8_t* codes;
  int64_t ldq;
  const uint8_t* scales;
  int64_t lds;
};

int launch_quantize_rows(const void* x, int x_type, int64_t m, int64_t k, int64_t ldx, int fmt, RowsOut o,
                         hipStream_t s);
int launch_dequant_rows(RowsIn in, int fmt, int64_t m, int64_t k, int out_type, void* out, int64_t ldo,
                        hipStream_t s);

struct NormArgs {
  const void* x;
  const void* res;    // or null
  int64_t ldx, ldr;
  const float* gain;  // or null
  float eps;
  void* h;            // x + res as stored, or null (may be x or res itself)
  int64_t ldh;
  void* y;            // the normed row, or null
  int y_type;
  int64_t ldy;
  int fmt;            // RowFormat, or -1: no quantised output
  RowsOut o;
  int64_t m, k;
};
int launch_rmsnorm(const NormArgs& a, int type, hipStream_t s);

#ifdef __HIPCC__
// ---- eight consecutive elements -------------------------------------------------------

// STREAM: past the L2 (a non-temporal load).
template <bool STREAM, typename V>
__device__ __forceinline__ V load_vec(const void* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const V*>(p));
  return *static_cast<const V*>(p);
}

template <int TYPE, bool STREAM = false>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  if constexpr (TYPE == kF32) {
    const f32x4 a = load_vec<STREAM, f32x4>(static_cast<const float*>(p) + at);
    const f32x4 b = load_vec<STREAM, f32x4>(static_cast<const float*>(p) + at + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
    const u32x4 w = load_vec<STREAM, u32x4>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
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

// Two values rounded to nearest even in a 16-bit type, packed (v0 in the low half).
template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float v0, float v1) {
  if constexpr (TYPE == kF16) {
    const f16x2 h = {(_Float16)v0, (_Float16)v1};
    return __builtin_bit_cast(uint32_t, h);
  } else {
    const bf16x2 h = {(__bf16)v0, (__bf16)v1};
    return __builtin_bit_cast(uint32_t, h);
  }
}

template <int TYPE>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&v)[8]) {
  if constexpr (TYPE == kF32) {
    f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(p) + at);
    o[0] = f32x4{v[0], v[1], v[2], v[3]};
    o[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + at) =
        u32x4{pack2<TYPE>(v[0], v[1]), pack2<TYPE>(v[2], v[3]), pack2<TYPE>(v[4], v[5]), pack2<TYPE>(v[6], v[7])};
  }
}
__device__ __forceinline__ void store8(int type, void* p, int64_t at, const float (&v)[8]) {
  if (type == kF32) store8<kF32>(p, at, v);
  else if (type == kF16) store8<kF16>(p, at, v);
  else store8<kBF16>(p, at, v);
}

// 2^(e - 127) for a biased exponent 0 .. 254 (0: the subnormal 2^-127).
__device__ __forceinline__ float pow2_biased(uint32_t e) {
  return __uint_as_float(e ? e << 23 : 0x00400000u);
}

// Another lane's value inside a row of 16 lanes, by a DPP control (without LDS).
template <int CTRL>
__device__ __forceinline__ int lane_move(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}

// ---- one block of 32 by four neighbouring lanes, eight elements each ---------------------
// All four lanes of a block call this together (the maxima cross lanes); `live` lanes
// write.  `oct` is the index of the eight elements in the row, `r` the row.
__device__ __forceinline__ void store_rows8(const RowsOut& o, int fmt, int64_t r, int oct, const float (&v)[8],
                                            bool live) {
  uint32_t top = 0;  // the largest magnitude by its bits: a NaN is above infinity, and that above all else
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  top = max(top, (uint32_t)lane_move<0xB1>((int)top));  // lane ^ 1
  top = max(top, (uint32_t)lane_move<0x4E>((int)top));  // lane ^ 2
  const bool bad = top >= 0x7F800000u;
  uint8_t* codes = o.codes + r * o.ldq;
  uint8_t* scales = o.scales + r * o.lds;
  if (fmt == kRowsQ8_1) {
    const float d = __uint_as_float(top) / 127.0f;
    uint16_t d16 = __half_as_ushort(__float2half_rn(d));
    const float rd = (d16 != 0 && !bad) ? 1.0f / d : 0.0f;
    if (bad) d16 = 0x7E00u;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = bad ? 0.0f : v[i] * rd;
      const float tr = truncf(p);
      float c = tr + ((fabsf(p - tr) >= 0.5f) ? copysignf(1.0f, p) : 0.0f);  // halves away from zero
      c = fminf(fmaxf(c, -127.0f), 127.0f);
      w[i >> 2] |= ((uint32_t)(int)c & 0xFFu) << (8 * (i & 3));
    }
    if (live) {
      *reinterpret_cast<u32x2*>(codes + 8 * oct) = u32x2{w[0], w[1]};
      if ((oct & 3) == 0) *reinterpret_cast<uint16_t*>(scales + oct / 2) = d16;
    }
    return;
  }
  const uint32_t e = top >> 23;
  const uint32_t emax = (fmt == kRowsMxfp4) ? 2u : 8u;
  const uint32_t s = bad ? 255u : (e > emax ? e - emax : 0u);
  const float inv = bad ? 0.0f : pow2_biased(254u - s);
  if (fmt == kRowsMxfp4) {
    uint32_t w = 0;
    if (!bad) {  // v * inv is exact; the conversion rounds to nearest even and saturates at 6
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * inv, v[1] * inv, 1.0f, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * inv, v[3] * inv, 1.0f, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * inv, v[5] * inv, 1.0f, 2);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * inv, v[7] * inv, 1.0f, 3);
    }
    if (live) *reinterpret_cast<uint32_t*>(codes + 4 * oct) = w;
  } else {
    uint32_t w[2] = {0u, 0u};
    if (!bad) {  // clamped first: the conversion itself makes a NaN of what is above 464
      float c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = fminf(fmaxf(v[i] * inv, -448.0f), 448.0f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i], c[4 * i + 1], 0, false);
        w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i + 2], c[4 * i + 3], p, true);
      }
    }
    if (live) *reinterpret_cast<u32x2*>(codes + 8 * oct) = u32x2{w[0], w[1]};
  }
  if (live && (oct & 3) == 0) scales[oct >> 2] = (uint8_t)s;
}
#endif  // __HIPCC__

}  // namespace iq4
