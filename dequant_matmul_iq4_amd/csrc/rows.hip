// rows.hip -- rows of activations in 8 or 4 bits (rows.hpp gives the formats): the
// quantiser, the decoder, and the RMS norm that quantises its rows as it makes them.
// All three only move memory: a few operations per element, each element read and
// written once.  A lane holds eight consecutive elements and four lanes a block of 32.
#include "common.hpp"
#include "rows.hpp"

namespace iq4 {

// Float rows larger than this are read and written past the L2: they would only push each other
// out of it and of the memory-side cache behind it (norm of 13056 x 4096 bf16 with its decode
// 125 -> 118 us reading so, 112 -> 109 writing so; 3256 x 14336 f16 rows 72 -> 66 and 65 -> 63).
// Smaller ones were often just written, or are read next, and are still there (norm of 3256 x 2048:
// 22.4 us, 24.9 reading past it).
constexpr int64_t kStreamBytes = 64 << 20;
static inline bool streams(int type, int64_t m, int64_t k) { return m * k * (type == kF32 ? 4 : 2) > kStreamBytes; }

// ---- quantise -------------------------------------------------------------------------
// Lanes walk the rows' groups of eight, the zero padding of MX rows included (fewer than 2^32
// groups); the scale bytes past the padded codes belong to no group and are zeroed by the
// row's last lane.  Four lanes agree on a block's scale inside the wave, and every wave reads and
// writes one run of memory.  Bound by memory: 3256 x 14336 f16 to MXFP8 27.1 us, 5.2 TB/s;
// 13056 x 4096 f32 to Q8_1 47-52 us, 271 MB, 5.2-5.8 TB/s; 4 x 4096 2.5 us, of which an empty launch is 1.7.
template <int TYPE, bool STREAM>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const void* __restrict__ x, uint32_t m, int k,
                                                            int64_t ldx, int fmt, uint32_t octs, int scale_bytes,
                                                            RowsOut o) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  const uint32_t r = i / octs;
  const int oct = (int)(i - r * octs);
  const bool live = r < m;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live && 8 * oct < k) load8<TYPE, STREAM>(x, r * ldx + 8 * oct, v);
  store_rows8(o, fmt, r, oct, v, live);
  if (live && fmt != kRowsQ8_1 && oct == (int)octs - 1)
    for (int b = octs / 4; b < scale_bytes; ++b) o.scales[r * o.lds + b] = 0;
}

int launch_quantize_rows(const void* x, int x_type, int64_t m, int64_t k, int64_t ldx, int fmt, RowsOut o,
                         hipStream_t s) {
  const int octs = (int)((fmt == kRowsQ8_1 ? k : (k + 127) / 128 * 128) / 8);
  const int64_t grid = (m * octs + 255) / 256;
  const int sb = (int)rows_scale_bytes(fmt, k);
  const bool st = streams(x_type, m, k);
#define IQ4_QUANT(T, S)                                                                                             \
  hipLaunchKernelGGL((quantize_rows_kernel<T, S>), dim3((unsigned)grid), dim3(256), 0, s, x, (uint32_t)m, (int)k, ldx, \
                     fmt, (uint32_t)octs, sb, o)
  if (x_type == kF32) { if (st) IQ4_QUANT(kF32, true); else IQ4_QUANT(kF32, false); }
  else if (x_type == kF16) { if (st) IQ4_QUANT(kF16, true); else IQ4_QUANT(kF16, false); }
  else { if (st) IQ4_QUANT(kBF16, true); else IQ4_QUANT(kBF16, false); }
#undef IQ4_QUANT
  return check_launch("quantize_rows_kernel");
}

// ---- decode ---------------------------------------------------------------------------
// The value code * scale is exact in binary32 (at most four significant bits, or the
// eight of a Q8_1 code times the eleven of its scale), then rounded once to the output's
// type.  A lane stores 16 bytes (four binary32 values, eight of 16 bits), so that a wave
// writes a kilobyte in one piece.  Bound by the writes: 3256 x 14336 MXFP8 to f32 33.5 us, 7.0 TB/s
// (the last of them still on their way through the memory-side cache); 13056 x 4096 MXFP4 34.7.
template <int FMT, int PER>
__device__ __forceinline__ void decode(const uint8_t* codes, const uint8_t* scales, int at, float (&v)[PER]) {
  if constexpr (FMT == kRowsQ8_1) {
    const float d = h2f(*reinterpret_cast<const uint16_t*>(scales + 2 * (at >> 5)));
    uint32_t w[PER / 4];
#pragma unroll
    for (int j = 0; j < PER / 4; ++j) w[j] = *reinterpret_cast<const uint32_t*>(codes + at + 4 * j);
#pragma unroll
    for (int j = 0; j < PER; ++j) v[j] = (float)(int8_t)((w[j >> 2] >> (8 * (j & 3))) & 0xFFu) * d;
  } else {
    const uint32_t s = scales[at >> 5];
    const float d = (s == 255u) ? __uint_as_float(0x7FC00000u) : pow2_biased(s);
    if constexpr (FMT == kRowsMxfp4) {
      uint32_t w;
      if constexpr (PER == 8) w = *reinterpret_cast<const uint32_t*>(codes + at / 2);
      else w = *reinterpret_cast<const uint16_t*>(codes + at / 2);
#define IQ4_TWO(B)                                                       \
  if constexpr (2 * B < PER) {                                           \
    const auto p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, B); \
    v[2 * B] = p[0] * d;                                                 \
    v[2 * B + 1] = p[1] * d;                                             \
  }
      IQ4_TWO(0) IQ4_TWO(1) IQ4_TWO(2) IQ4_TWO(3)
#undef IQ4_TWO
    } else {
#pragma unroll
      for (int j = 0; j < PER / 4; ++j) {
        const int w = *reinterpret_cast<const int*>(codes + at + 4 * j);
        const auto p = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), q = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
        v[4 * j] = p[0] * d;
        v[4 * j + 1] = p[1] * d;
        v[4 * j + 2] = q[0] * d;
        v[4 * j + 3] = q[1] * d;
      }
    }
  }
}

template <int FMT, int TYPE, bool STREAM>
__global__ void __launch_bounds__(256) dequant_rows_kernel(RowsIn in, uint32_t m, uint32_t pieces,
                                                           void* __restrict__ out, int64_t ldo) {
  constexpr int kPer = TYPE == kF32 ? 4 : 8;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  const uint32_t r = i / pieces;
  const int at = kPer * (int)(i - r * pieces);
  if (r >= m) return;
  float v[kPer];
  decode<FMT, kPer>(in.codes + r * in.ldq, in.scales + r * in.lds, at, v);
  if constexpr (TYPE == kF32) {
    f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(out) + r * ldo + at);
    const f32x4 w = {v[0], v[1], v[2], v[3]};
    if constexpr (STREAM) __builtin_nontemporal_store(w, o);
    else *o = w;
  } else {
    u32x4* o = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + r * ldo + at);
    const u32x4 w = {pack2<TYPE>(v[0], v[1]), pack2<TYPE>(v[2], v[3]), pack2<TYPE>(v[4], v[5]), pack2<TYPE>(v[6], v[7])};
    if constexpr (STREAM) __builtin_nontemporal_store(w, o);
    else *o = w;
  }
}

template <int FMT>
static int launch_dequant_fmt(RowsIn in, int64_t m, int64_t k, int out_type, void* out, int64_t ldo, hipStream_t s) {
  const uint32_t pieces = (uint32_t)(k / (out_type == kF32 ? 4 : 8));
  // a launch has fewer than 2^32 threads: the largest binary32 results (2^34 values) are made in two
  if (m * pieces > ((int64_t)1 << 32) - 256) {
    const int64_t half = m / 2;
    if (int e = launch_dequant_fmt<FMT>(in, half, k, out_type, out, ldo, s)) return e;
    in.codes += half * in.ldq;
    in.scales += half * in.lds;
    return launch_dequant_fmt<FMT>(in, m - half, k, out_type, static_cast<float*>(out) + half * ldo, ldo, s);
  }
  const dim3 grid((unsigned)((m * pieces + 255) / 256));
  const bool st = streams(out_type, m, k);
#define IQ4_DEQ(T)                                                                                                       \
  {                                                                                                                      \
    if (st) hipLaunchKernelGGL((dequant_rows_kernel<FMT, T, true>), grid, dim3(256), 0, s, in, (uint32_t)m, pieces, out, ldo); \
    else hipLaunchKernelGGL((dequant_rows_kernel<FMT, T, false>), grid, dim3(256), 0, s, in, (uint32_t)m, pieces, out, ldo);   \
  }
  if (out_type == kF32) IQ4_DEQ(kF32)
  else if (out_type == kF16) IQ4_DEQ(kF16)
  else IQ4_DEQ(kBF16)
#undef IQ4_DEQ
  return check_launch("dequant_rows_kernel");
}

int launch_dequant_rows(RowsIn in, int fmt, int64_t m, int64_t k, int out_type, void* out, int64_t ldo,
                        hipStream_t s) {
  if (fmt == kRowsMxfp4) return launch_dequant_fmt<kRowsMxfp4>(in, m, k, out_type, out, ldo, s);
  if (fmt == kRowsMxfp8) return launch_dequant_fmt<kRowsMxfp8>(in, m, k, out_type, out, ldo, s);
  return launch_dequant_fmt<kRowsQ8_1>(in, m, k, out_type, out, ldo, s);
}

// ---- RMS norm ---------------------------------------------------------------------------
//   h = x + res, rounded to the rows' type (what is stored is what is normed);
//   u = f32(1 / sqrt(mean(h^2) + eps));   y = f32(f32(h * u) * gain).
// The mean is held in 64 bits: its rounding error then stays some 2^-29 of a binary32
// step, so u, y and with them every rounding decision of the quantised row are a function
// of the row alone, whatever the order of the sum.  The extra cost (one conversion and one
// fused multiply-add per element) hides under the row's loads.
// Bound by memory: 13056 x 4096 bf16 with a residual to MXFP4 60 us, 349 MB, 5.8 TB/s; for one
// row of 4096 by latency: 3.0 us, of which an empty launch is 1.7.
// One workgroup per row; a lane keeps its groups of eight in registers (V of them) between
// the sum and the second use.
template <int TYPE, bool STREAM>
__device__ __forceinline__ void norm_load(const NormArgs& a, int64_t r, int oct, float (&v)[8]) {
  load8<TYPE, STREAM>(a.x, r * a.ldx + 8 * oct, v);
  if (a.res) {
    float t[8];
    load8<TYPE, STREAM>(a.res, r * a.ldr + 8 * oct, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // the binary32 sum of two 16-bit floats rounds to them as the exact sum does
      v[i] = v[i] + t[i];
      if constexpr (TYPE == kF16) v[i] = (float)(_Float16)v[i];
      if constexpr (TYPE == kBF16) v[i] = (float)(__bf16)v[i];
    }
  }
}

template <int TYPE>
__device__ __forceinline__ void norm_store(const NormArgs& a, int64_t r, int oct, float u, float (&v)[8], bool live) {
  if (live) {
    float g[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (a.gain) load8<kF32>(a.gain, 8 * oct, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (v[i] * u) * g[i];
    if (a.y) store8(a.y_type, a.y, r * a.ldy + 8 * oct, v);
  }
}

// The wave's sum in every lane: within 16 lanes by DPP, across them by two exchanges (all by
// exchanges through LDS: one row of 4096 with its decode 4.93 us for 4.83, 13056 rows 104.5 for 101.7).
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)(uint32_t)lane_move<CTRL>((int)u) |
                                          (uint64_t)(uint32_t)lane_move<CTRL>((int)(u >> 32)) << 32));
}
__device__ __forceinline__ double wave_sum(double v) {
  v += moved<0xB1>(v);   // lane ^ 1
  v += moved<0x4E>(v);   // lane ^ 2
  v += moved<0x141>(v);  // half rows mirrored: the other four of eight
  v += moved<0x140>(v);  // rows mirrored: the other eight of sixteen
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

template <int TYPE, int NT, int V, bool STREAM>
__global__ void __launch_bounds__(NT) rmsnorm_kernel(NormArgs a, int octs_k, int octs, int scale_bytes) {
  __shared__ double part[NT / 64];
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  float v[V][8];
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int oct = tid + j * NT;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
    if (oct < octs_k) {
      norm_load<TYPE, STREAM>(a, r, oct, v[j]);
      if (a.h) store8<TYPE>(a.h, r * a.ldh + 8 * oct, v[j]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fma((double)v[j][i], (double)v[j][i], sum);
  }
  sum = wave_sum(sum);
  if constexpr (NT > 64) {
    if ((tid & 63) == 0) part[tid >> 6] = sum;
    __syncthreads();
    sum = part[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) sum += part[w];
  }
  // a row with an infinity or a NaN is all NaN
  float u = (float)(1.0 / sqrt(sum / (double)a.k + (double)a.eps));
  if (!(sum < __builtin_inf())) u = __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int oct = tid + j * NT;
    norm_store<TYPE>(a, r, oct, u, v[j], oct < octs_k);
    if (a.fmt >= 0) store_rows8(a.o, a.fmt, r, oct, v[j], oct < octs);
  }
  if (a.fmt >= 0 && a.fmt != kRowsQ8_1)
    for (int b = octs / 4 + tid; b < scale_bytes; b += NT) a.o.scales[r * a.o.lds + b] = 0;
}

// Rows too long for registers: the sum in a first pass, which stores h if it is wanted, and
// the row read again in a second (h if stored: x or res may be the same memory as h).  3256 x 32768
// bf16 with a residual to MXFP8 166 us: 750 MB and the second reading, 964 MB, 5.8 TB/s (rows of 16384, in
// registers, 68 us, 375 MB); one such row 8.3 us.
template <int TYPE>
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(NormArgs a, int octs_k, int octs, int scale_bytes) {
  __shared__ double part[16];
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  double sum = 0.0;
  for (int oct = tid; oct < octs_k; oct += 1024) {
    float v[8];
    norm_load<TYPE, false>(a, r, oct, v);
    if (a.h) store8<TYPE>(a.h, r * a.ldh + 8 * oct, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fma((double)v[i], (double)v[i], sum);
  }
  sum = wave_sum(sum);
  if ((tid & 63) == 0) part[tid >> 6] = sum;
  __syncthreads();
  sum = part[0];
  for (int w = 1; w < 16; ++w) sum += part[w];
  float u = (float)(1.0 / sqrt(sum / (double)a.k + (double)a.eps));
  if (!(sum < __builtin_inf())) u = __uint_as_float(0x7FC00000u);
  for (int base = 0; base < octs; base += 1024) {
    const int oct = base + tid;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (oct < octs_k) {
      if (a.h) load8<TYPE>(a.h, r * a.ldh + 8 * oct, v);
      else norm_load<TYPE, false>(a, r, oct, v);
    }
    norm_store<TYPE>(a, r, oct, u, v, oct < octs_k);
    if (a.fmt >= 0) store_rows8(a.o, a.fmt, r, oct, v, oct < octs);
  }
  if (a.fmt >= 0 && a.fmt != kRowsQ8_1)
    for (int b = octs / 4 + tid; b < scale_bytes; b += 1024) a.o.scales[r * a.o.lds + b] = 0;
}

template <int TYPE>
static int launch_norm_t(const NormArgs& a, hipStream_t s) {
  const int octs_k = (int)(a.k / 8);
  const bool mx = a.fmt == kRowsMxfp4 || a.fmt == kRowsMxfp8;
  const int octs = mx ? (int)((a.k + 127) / 128 * 16) : octs_k;
  const int sb = mx ? (int)rows_scale_bytes(a.fmt, a.k) : 0;
  const dim3 grid((unsigned)a.m);
  const bool st = streams(TYPE, a.m, a.k);
#define IQ4_NORM(NT, V)                                                                                              \
  {                                                                                                                  \
    if (st) hipLaunchKernelGGL((rmsnorm_kernel<TYPE, NT, V, true>), grid, dim3(NT), 0, s, a, octs_k, octs, sb);       \
    else hipLaunchKernelGGL((rmsnorm_kernel<TYPE, NT, V, false>), grid, dim3(NT), 0, s, a, octs_k, octs, sb);         \
  }
  // a lane per group of eight as far as a workgroup goes (one row of 4096 with its decode: 0.7 us
  // less than with two groups a lane)
  if (octs <= 64) IQ4_NORM(64, 1)
  else if (octs <= 256) IQ4_NORM(256, 1)
  else if (octs <= 512) IQ4_NORM(512, 1)
  else if (octs <= 1024) IQ4_NORM(1024, 1)
  else if (octs <= 2048) IQ4_NORM(1024, 2)
  else hipLaunchKernelGGL(rmsnorm_long_kernel<TYPE>, grid, dim3(1024), 0, s, a, octs_k, octs, sb);
#undef IQ4_NORM
  return check_launch("rmsnorm_kernel");
}

int launch_rmsnorm(const NormArgs& a, int type, hipStream_t s) {
  if (type == kF32) return launch_norm_t<kF32>(a, s);
  if (type == kF16) return launch_norm_t<kF16>(a, s);
  return launch_norm_t<kBF16>(a, s);
}

}  // namespace iq4
