// swiglu.hip -- h = silu(g) * u between an expert's (or a dense layer's) two products,
// quantised for the second one in the same pass, and its gradient.  With
// s = 1 / (1 + e^-g):
//   h = g s u;   du = dh g s,   dg = dh u s (1 + g (1 - s)).
#include "pieces.hpp"
#include "swiglu.hpp"

namespace iq4 {

// Below this e^-g comes near the end of binary32, while g e^g u may be a normal number (-91.8 for u = 1, -180 for
// the largest): such elements are made again in 64 bits, behind a branch that a lane without one skips.
constexpr float kDeep = -80.f;

// e^-g in binary32 for g >= kDeep: 2^-(g log2 e) with the product's rounding error carried along (its relative
// weight in the result grows with |g|); above 88 the power leaves binary32.
__device__ __forceinline__ float power(float g) {
  const float x = fminf(fmaxf(-g, -88.f), 88.f);
  const float hi = x * 1.44269502f;
  const float lo = fmaf(x, 1.92596303e-8f, fmaf(x, 1.44269502f, -hi));
  const float e = __builtin_amdgcn_exp2f(hi);
  return fmaf(e, lo * 0.693147182f, e);
}
// e^g for g < kDeep, where it is the sigmoid too (1 + e^g rounds to 1): a binary32 fraction of the same way, and the
// power of two that only 64 bits hold.
__device__ __forceinline__ double deep_power(float g) {
  const float x = fmaxf(g, -1000.f);  // (2^-1443: zero)
  const float hi = x * 1.44269502f;
  const float lo = fmaf(x, 1.92596303e-8f, fmaf(x, 1.44269502f, -hi));
  const float n = rintf(hi), e = __builtin_amdgcn_exp2f(hi - n);
  return __builtin_amdgcn_ldexp((double)fmaf(e, lo * 0.693147182f, e), (int)n);
}
// 1 / (1 + e^-g) in binary32 for g >= kDeep.
__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + power(g)); }
// g / (1 + e^-g) * u for g >= kDeep, all roundings but the last and the power's carried along: a row that is
// quantised next makes a whole step of every error next to a border.  Its errors' root mean square is 0.42 of a last
// place; with the sum, the reciprocal and both products rounded it was 0.68, and of the formula's operations
// one by one, each rounded right, it is 0.57.
__device__ __forceinline__ float gated(float g, float u) {
  const float e = power(g);
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  const float t = fmaf(-e, r, 1.0f - r);  // what r misses, relative to it
  const float a = g * r, h = a * u;
  const float rest = fmaf(fmaf(a, t, fmaf(g, r, -a)), u, fmaf(a, u, -h));
  return fabsf(h) < __builtin_inff() ? h + rest : h;
}
__device__ __forceinline__ float deep_gated(float g, float u) { return (float)(deep_power(g) * g * u); }

// Eight elements a lane, whatever row they belong to.  Memory bounds it: 26048 rows of 768 in binary16
// 23 us with y alone (5.2 TB/s), 3 of the few rows of a step.  Past the caches it is no faster.
template <int T>
__global__ void __launch_bounds__(256) swiglu_kernel(SwigluArgs a, Pieces octs) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  const uint32_t r = octs.row(i);
  const int oct = (int)(i - r * octs.n);
  const bool live = r < a.m;
  // (a row that is quantised has whole pieces; behind them, up to its padding, there are none)
  const Piece c = piece_of<8>(oct, a.k);
  const bool here = live && 8 * (int64_t)oct < a.k;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (here) {
    float g[8], u[8];
    load_piece<T, 8>(static_cast<const char*>(a.g) + r * a.ldg * (T == kF32 ? 4 : 2), c.at, c.left, g);
    load_piece<T, 8>(static_cast<const char*>(a.u) + r * a.ldu * (T == kF32 ? 4 : 2), c.at, c.left, u);
    bool deep = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = gated(g[e], u[e]), deep |= g[e] < kDeep;
    if (__builtin_expect(deep, 0)) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (g[e] < kDeep) v[e] = deep_gated(g[e], u[e]);
    }
    if (a.y) {
      char* y = static_cast<char*>(a.y) + r * a.ldy * (a.y_type == kF32 ? 4 : 2);
      if (a.y_type == kF32) store_piece<kF32, 8>(y, c.at, c.left, v);
      else if (a.y_type == kF16) store_piece<kF16, 8>(y, c.at, c.left, v);
      else store_piece<kBF16, 8>(y, c.at, c.left, v);
    }
  }
  if (a.fmt < 0) return;
  store_rows8(a.o, a.fmt, r, oct, v, live);
  if (live && a.fmt != kRowsQ8_1 && oct == (int)octs.n - 1)
    for (int b = octs.n / 4; b < (int)((a.k + 511) / 512 * 16); ++b) a.o.scales[r * a.o.lds + b] = 0;
}

// Rows go in as many launches as they take.
int launch_swiglu(const SwigluArgs& a0, int type, hipStream_t s) {
  SwigluArgs a = a0;
  const bool mx = a.fmt == kRowsMxfp4 || a.fmt == kRowsMxfp8;
  const Pieces octs((uint32_t)((mx ? (a.k + 127) / 128 * 128 : a.k + 7) / 8));
  const int64_t most = rows_a_launch(octs);
  for (int64_t left = a0.m; left > 0; left -= a.m) {
    a.m = left < most ? left : most;
    const dim3 grid((unsigned)((a.m * octs.n + 255) / 256));
    if (type == kF32) hipLaunchKernelGGL(swiglu_kernel<kF32>, grid, dim3(256), 0, s, a, octs);
    else if (type == kF16) hipLaunchKernelGGL(swiglu_kernel<kF16>, grid, dim3(256), 0, s, a, octs);
    else hipLaunchKernelGGL(swiglu_kernel<kBF16>, grid, dim3(256), 0, s, a, octs);
    if (int e = check_launch("swiglu_kernel")) return e;
    a.g = static_cast<const char*>(a.g) + a.m * a.ldg * type_bytes(type);
    a.u = static_cast<const char*>(a.u) + a.m * a.ldu * type_bytes(type);
    if (a.y) a.y = static_cast<char*>(a.y) + a.m * a.ldy * type_bytes(a.y_type);
    if (a.fmt >= 0) a.o.codes += a.m * a.o.ldq, a.o.scales += a.m * a.o.lds;
  }
  return 0;
}

// 16 bytes of the wider type a lane; five rows of memory a row, which bound it: 3256 rows of 14336 in
// bfloat16 74 us (6.3 TB/s), 500 rows 12.
template <int TD, int T, bool STREAM>
__global__ void __launch_bounds__(256) swiglu_grad_kernel(SwigluGradArgs a, Pieces pieces) {
  constexpr int P = (TD == kF32 || T == kF32) ? 4 : 8, kSize = T == kF32 ? 4 : 2;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  const uint32_t r = pieces.row(i);
  if (r >= a.m) return;
  const Piece c = piece_of<P>(i - r * pieces.n, a.k);  // (what two pieces have is written twice, the same)
  float d[P], g[P], u[P], x[P], z[P];
  bool deep = false;
  load_piece<TD, P, STREAM>(static_cast<const char*>(a.dh) + r * a.lddh * (TD == kF32 ? 4 : 2), c.at, c.left, d);
  load_piece<T, P, STREAM>(static_cast<const char*>(a.g) + r * a.ldg * kSize, c.at, c.left, g);
  load_piece<T, P, STREAM>(static_cast<const char*>(a.u) + r * a.ldu * kSize, c.at, c.left, u);
#pragma unroll
  for (int e = 0; e < P; ++e) {
    const float s = sigmoid(g[e]);
    z[e] = d[e] * (g[e] * s);
    x[e] = (d[e] * u[e]) * (s * fmaf(g[e], 1.0f - s, 1.0f));
    deep |= g[e] < kDeep;
  }
  if (__builtin_expect(deep, 0)) {
#pragma unroll
    for (int e = 0; e < P; ++e) {
      if (!(g[e] < kDeep)) continue;
      const double s = deep_power(g[e]) * d[e];
      z[e] = (float)(s * g[e]), x[e] = (float)(s * (1.0 + g[e]) * u[e]);
    }
  }
  store_piece<T, P, STREAM>(static_cast<char*>(a.dg) + r * a.lddg * kSize, c.at, c.left, x);
  store_piece<T, P, STREAM>(static_cast<char*>(a.du) + r * a.lddu * kSize, c.at, c.left, z);
}

int launch_swiglu_grad(const SwigluGradArgs& a0, int dh_type, int type, hipStream_t s) {
  SwigluGradArgs a = a0;
  const int p = (dh_type == kF32 || type == kF32) ? 4 : 8;
  const Pieces pieces((uint32_t)((a.k + p - 1) / p));
  const int64_t most = rows_a_launch(pieces);
  // (3256 rows of 14336 in bfloat16 74 us for 82; written rows off 16 bytes would leave in parts)
  const bool st = a.m * a.k * type_bytes(type) > kStreamBytes && aligned(a.dg, 16) && aligned(a.du, 16) &&
                  ((a.lddg | a.lddu) * type_bytes(type)) % 16 == 0;
  for (int64_t left = a0.m; left > 0; left -= a.m) {
    a.m = left < most ? left : most;
    const dim3 grid((unsigned)((a.m * pieces.n + 255) / 256));
#define IQ4_GRAD2(TD, T)                                                                                        \
  {                                                                                                             \
    if (st) hipLaunchKernelGGL((swiglu_grad_kernel<TD, T, true>), grid, dim3(256), 0, s, a, pieces);            \
    else hipLaunchKernelGGL((swiglu_grad_kernel<TD, T, false>), grid, dim3(256), 0, s, a, pieces);              \
  }
#define IQ4_GRAD(TD)                                 \
  {                                                  \
    if (type == kF32) IQ4_GRAD2(TD, kF32)            \
    else if (type == kF16) IQ4_GRAD2(TD, kF16)       \
    else IQ4_GRAD2(TD, kBF16)                        \
  }
    if (dh_type == kF32) IQ4_GRAD(kF32)
    else if (dh_type == kF16) IQ4_GRAD(kF16)
    else IQ4_GRAD(kBF16)
#undef IQ4_GRAD
#undef IQ4_GRAD2
    if (int e = check_launch("swiglu_grad_kernel")) return e;
    a.dh = static_cast<const char*>(a.dh) + a.m * a.lddh * type_bytes(dh_type);
    a.g = static_cast<const char*>(a.g) + a.m * a.ldg * type_bytes(type);
    a.u = static_cast<const char*>(a.u) + a.m * a.ldu * type_bytes(type);
    a.dg = static_cast<char*>(a.dg) + a.m * a.lddg * type_bytes(type);
    a.du = static_cast<char*>(a.du) + a.m * a.lddu * type_bytes(type);
  }
  return 0;
}

}  // namespace iq4
