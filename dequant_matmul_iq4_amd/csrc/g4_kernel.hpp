// g4_kernel.hpp -- the product of few rows with group-scaled 4-bit weights (g4.hpp): the kernel and
// its launch, compiled once per group size (g4_32.hip, g4_64.hip, g4_128.hip).
//
// Mathematics.  With d = sum of (q - z) x over a group's k, a row's result is the sum of s d over
// its groups.  A code tile's products run on the matrix cores, whose products are exact here and
// whose sums are binary32; each group's d is scaled by one fused multiply-add.  No weight is rounded.
//
//   binary16 X  q - z as a binary16 number, (1024 + q) - (1024 + z): the codes are or-ed into the
//               bits of 1024, two at a time.  11 operations for eight weights.
//   bfloat16 X  no packed instruction makes q - z a bfloat16 number (19 operations from a dot
//               product with (1, 0) and (0, 1)), so the weight is 16 + q, or-ed into the bits of 16, and
//               the group's sums of X, made once for all rows of W, are multiplied by -(16 + z) and begin
//               d: 8 operations.  The sums are then some five times those of q - z, and so
//               are their roundings, 2^-24 of them each.  An infinity leaves a NaN (infinity
//               minus infinity): a result that is not finite is made again without this, in 64 bits, by a wave.
//   binary32 X  two binary16 numbers, the value rounded to eleven bits and what is left, rounded
//               likewise; a wave has a slice of k, and there a row's values are multiplied by the power
//               of two that brings the largest to 2^14 .. 2^15 (what is left by 2^11 more), and its sums divided by it.
//               Within 2^-23 of the value (a tie of what is left), or 2^-50 of the slice's largest (half a step of the
//               smallest).  Each of the two is a row of the operand; their sums are divided and joined.  (Without the 2^11
//               a value below 2^-16 of the largest loses bits, 2^-39 of that one, and 4 rows of 2560 x 6144 take 8.0 us
//               for 8.1; three parts lose nothing, but an operand then has five rows for eight.)
//               An infinity's rest is a NaN, and scales near the largest number may take the multiplied sums past
//               it: again a result that is not finite is made again.
//
// Operands of v_mfma_f32_16x16x32 (lane l = 16 g + c): the activations are the first one, rows by c;
// the weights the second, 16 rows of W by c, so that a lane's scale is that of the row whose codes
// it holds; the lane receives D[4g + i][c], four rows of X times row c of W.
#pragma once
#include "experts.hpp"
#include "g4.hpp"
#include "pieces.hpp"

#include <math.h>

#include <type_traits>

namespace iq4 {

// An instruction takes one constant from a scalar register, the other has to come from a vector one.
struct G4Consts {
  uint32_t lo, hi, top;
};
template <bool BRAIN>
__device__ __forceinline__ G4Consts g4_consts() {
  G4Consts k = {BRAIN ? 0x00780078u : 0x000F000Fu, 0x00F000F0u, BRAIN ? 0x41804180u : 0x64006400u};
  asm("" : "+s"(k.lo), "+s"(k.hi), "+v"(k.top));  // opaque: not literals
  return k;
}
// Eight weights of a word: q - z in binary16 (bias 1024 + z twice; the second pair is 16 q in the bits of
// 1024, brought down by a multiply-add with bias16, -(64 + z) twice).
// (SHIFT: brought down by a shift instead, where bias16 would serve for eight weights only.)
template <bool SHIFT>
__device__ __forceinline__ u32x4 g4_half(const G4Consts& k, uint32_t w, f16x2 bias, f16x2 bias16) {
  const f16x2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
  u32x4 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t v = h ? w >> 8 : w;
    const f16x2 a = __builtin_bit_cast(f16x2, (v & k.lo) | k.top) - bias;
    f16x2 b;
    if constexpr (SHIFT) b = __builtin_bit_cast(f16x2, ((w >> (8 * h + 4)) & k.lo) | k.top) - bias;
    else b = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, (v & k.hi) | k.top), sixteenth, bias16);
    r[2 * h] = __builtin_bit_cast(uint32_t, a);
    r[2 * h + 1] = __builtin_bit_cast(uint32_t, b);
  }
  return r;
}
// 16 + q in bfloat16.
__device__ __forceinline__ u32x4 g4_brain(const G4Consts& k, uint32_t w) {
  return u32x4{((w << 3) & k.lo) | k.top, ((w >> 1) & k.lo) | k.top, ((w >> 5) & k.lo) | k.top, ((w >> 9) & k.lo) | k.top};
}

// Largest value over the 16 lanes of a row.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, (uint32_t)lane_move<0xB1>((int)v));   // lane ^ 1
  v = max(v, (uint32_t)lane_move<0x4E>((int)v));   // lane ^ 2
  v = max(v, (uint32_t)lane_move<0x141>((int)v));  // half rows mirrored
  return max(v, (uint32_t)lane_move<0x140>((int)v));  // rows mirrored
}
// x less the binary16 number in the low or high half of h, exact: one mixed instruction each.
__device__ __forceinline__ float less_lo(float x, uint32_t h) {
  float r;
  asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(r) : "v"(h), "v"(x));
  return r;
}
__device__ __forceinline__ float less_hi(float x, uint32_t h) {
  float r;
  asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(r) : "v"(h), "v"(x));
  return r;
}
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The largest magnitude, by its bits, of eight elements from k on of a row of X: an infinity is above all numbers, and a
// NaN above that.
template <int XT>
__device__ __forceinline__ uint32_t g4_top(const char* row, int k, int K) {
  float v[8];
  load_piece<XT, 8>(row, min(k, K - 8), 8, v);
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  return k < K ? top : 0u;
}
// The results of one row of X in a row tile, from the definition: in 64 bits, in a fixed order, column c in the lanes
// (g, c).  infinite: the row holds an infinity, so that only the code tiles where it has one count.
template <int XT, int G>
__device__ float g4_again(const G4Args& a, const uint8_t* W, int64_t x_row, int64_t rt, bool infinite, int lane) {
  const int g = lane >> 4, c = lane & 15, K = (int)a.k;
  constexpr int kSets = 128 / G;
  const int kt_n = g4_k_tiles(a.k);
  const uint8_t* ss = W + g4_code_plane(a.n, a.k);
  const uint8_t* zs = ss + g4_scale_plane(a.n, a.k, G);
  const char* row = static_cast<const char*>(a.x) + x_row * a.ldx * (XT == kF32 ? 4 : 2);
  double sum = 0.0;
  auto add = [&](int kt) {
    const int64_t tile = rt * kt_n + kt;
#pragma unroll 2
    for (int b = 0; b < 4; ++b) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(W + tile * kG4TileBytes + 16 * lane + 4 * b);
      const int k = 128 * kt + 32 * b + 8 * g;
      const int64_t at = (tile * 16 + c) * kSets + 32 * b / G;
      const uint16_t h = reinterpret_cast<const uint16_t*>(ss)[at];
      const double s = a.scale_type == kF16 ? h2f(h) : __uint_as_float((uint32_t)h << 16);
      const int z = a.zeros ? zs[at] : 8;
      float x[8];
      load_piece<XT, 8>(row, min(k, K - 8), 8, x);
      double d = 0.0;
#pragma unroll
      for (int e = 0; e < 8; ++e) d = fma((double)((int)(w >> (16 * (e & 1) + 4 * (e >> 1)) & 15u) - z), (double)x[e], d);
      sum = k < K ? fma(s, d, sum) : sum;
    }
  };
#pragma nounroll
  for (int kt = 0; kt < kt_n; kt += 4) {
    // (16 lanes have a code tile's elements)
    const uint64_t who = infinite ? __ballot(g4_top<XT>(row, 128 * kt + 8 * lane, K) >= 0x7F800000u) : ~0ull;
#pragma nounroll
    for (int h = 0; h < 4; ++h)
      if (kt + h < kt_n && (who >> (16 * h) & 0xFFFF)) add(kt + h);
  }
  sum += __shfl_xor(sum, 16);
  return (float)(sum + __shfl_xor(sum, 32));
}

// How a call's work is dealt out (set by the launcher).
struct G4Plan {
  int cols;    // tiles of rows of X
  int y;       // those along the grid's y (the rest along z)
  int ks;      // waves a workgroup
  int kt_n, rt_n;  // code tiles along k, row tiles
  int per;     // row tiles of W a workgroup
  int rb;      // row tiles between two joins of the waves' sums: all, or a multiple of those that a wave loads ahead
               // (four at most; one where k goes in slices)
  int chunks;  // slices of k one after another (the activations of one are in registers)
};
constexpr int kG4StageRow = 128 * 2 + 16;  // a row of 128 binary16 numbers; 16 bytes on, so that rows begin in different banks
// A wave's LDS before its sums: the way of its operands; binary32, the powers of two; bfloat16, the groups'
// sums of X.
constexpr int g4_x_lds(int xt, int nv, int sx, int group) {
  return 16 * kG4StageRow + (xt == kF32 ? nv * 64 : xt == kBF16 ? sx * (128 / group) * nv * 64 : 0);
}

// A workgroup of KS waves: `per` row tiles of W against one tile of rows of X (NV operands of 16
// rows; a binary32 row is two of them), k dealt out to the waves in slices of SX code tiles.  A wave
// keeps its slice of X as operands in registers and runs over the row tiles, whose codes go from
// memory straight into registers, a row tile ahead.  The waves' sums are joined through LDS in
// the waves' order.
// Measured, weights from memory: one binary16 row of 4096 x 4096 5.3 us (1.6 TB/s: the start and one pass of latency),
// of 14336 x 4096 10.1 (3.0 TB/s); 47 bfloat16 rows of it 22 (X, 262 KB into each CU; vector operations for 9 of them, the
// matrix pipe 18 %, waves wait 40 % of their time); 32 binary32 rows of 28 experts of 1536 x 2048 16.6 (2.1 TB/s: offsets, pair
// ids and rows come before the weights' products); 488 rows of 128 experts of 2048 x 768 23 (3.3 TB/s; waves wait 56 %).
template <int XT, int NV, int SX, int G, bool CHUNKS>
__global__ void __launch_bounds__(512) g4_kernel(G4Args a, G4Plan plan) {
  // all arguments at once: loaded where they are used, one would wait for memory after the other
  asm volatile("" ::"s"(a.W), "s"(a.n), "s"(a.k), "s"(a.scale_type), "s"(a.zeros), "s"(a.x), "s"(a.ldx), "s"(a.m));
  asm volatile("" ::"s"(a.y), "s"(a.y_type), "s"(a.ldy), "s"(a.offsets), "s"(plan.cols), "s"(plan.y), "s"(plan.ks));
  asm volatile("" ::"s"(plan.kt_n), "s"(plan.rt_n), "s"(plan.per), "s"(plan.rb), "s"(plan.chunks));
  constexpr bool f32 = XT == kF32;
  constexpr int kBM = f32 ? 8 * NV : 16 * NV;
  constexpr int kSets = 128 / G, kSteps = G / 32;  // groups of a code tile, steps of a group
  constexpr int kFours = f32 ? 2 : 4;              // groups of four rows of X in an operand
  constexpr int kXLds = g4_x_lds(XT, NV, SX, G);
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int slice = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), KS = plan.ks;
  const int col = (int)blockIdx.z * plan.y + (int)blockIdx.y;
  if (col >= plan.cols || (int)blockIdx.x * plan.per >= plan.rt_n) return;
  const uint8_t* W = a.W;
  int row0 = col * kBM, rows = min(kBM, (int)a.m - row0);
  if (__builtin_expect(a.offsets != nullptr, 0)) {
    int e;
    if (!expert_tile(a.offsets, a.n_expert, (int)a.m, kBM, col, e, row0, rows)) return;
    W += e * a.w_stride;
  }
  const int kt_n = plan.kt_n, rt_n = plan.rt_n, K = (int)a.k;
  const int first = (int)blockIdx.x * plan.per, last = min(first + plan.per, rt_n);
  const int wave_lds = kXLds + plan.rb * NV * 1024;
  uint8_t* mine = lds + slice * wave_lds;
  int* exps = reinterpret_cast<int*>(mine + 16 * kG4StageRow);  // binary32
  uint8_t* sums = mine + 16 * kG4StageRow;                       // bfloat16
  f32x4* part = reinterpret_cast<f32x4*>(mine + kXLds);

  // ---- codes, scales and zero points of a row tile's slice ------------------------------------------
  struct WTile {
    u32x4 q;
    uint32_t s[G == 32 ? 2 : 1], z;
  };
  const int64_t tiles_n = (int64_t)rt_n * kt_n;
  const uint8_t* S = W + tiles_n * kG4TileBytes;
  // (without zero points bytes of the scales are loaded, and not looked at: a branch around the load would
  // make every wait one for all loads)
  const uint8_t* Z = a.zeros ? S + tiles_n * (16 * kSets * 2) : S;
  auto load_w = [&](int64_t tile, WTile& o) {  // tile: rt * kt_n + kt, the same in all lanes
    o.q = *reinterpret_cast<const u32x4*>(W + tile * kG4TileBytes + (uint32_t)(lane * 16));
    const uint8_t* s = S + tile * (16 * kSets * 2) + (uint32_t)(c * kSets * 2);
    if constexpr (G == 32) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(s);
      o.s[0] = v[0], o.s[1] = v[1];
    } else if constexpr (G == 64) {
      o.s[0] = *reinterpret_cast<const uint32_t*>(s);
    } else {
      o.s[0] = *reinterpret_cast<const uint16_t*>(s);
    }
    const uint8_t* z = Z + tile * (16 * kSets) + (uint32_t)(c * kSets);
    if constexpr (G == 32) o.z = *reinterpret_cast<const uint32_t*>(z);
    else if constexpr (G == 64) o.z = *reinterpret_cast<const uint16_t*>(z);
    else o.z = *z;
  };
  // A slice's code tiles [base, base + SX).  Where the slice would pass the last code tile it begins
  // earlier, and the tiles that are not its own (below `own`) get activations of zero.
  auto slice_of = [&](int chunk, int& base, int& own) {
    own = (chunk * KS + slice) * SX;
    base = min(own, kt_n - SX);
  };
  int base, own;
  slice_of(0, base, own);

  // ---- the activations of a slice, as operands in registers ------------------------------------------
  // First as in memory, whole rows of a code tile: lane (g, c) has elements 8 c .. 8 c + 7 of row 4 p + g in
  // word p, binary32 in words 2 p and 2 p + 1.  (As the instruction takes them, neighbouring lanes would
  // load of different rows, 64 cache lines an instruction, which takes four times as long: 16 rows of
  // 14336 x 4096 so 14.1 us, and 4.2 of them until the loads are under way.)  Then through LDS.
  u32x4 xf[SX][NV][4];
  auto x_row = [&](int i) {  // row i of the tile (one past the last repeats that, and is not stored)
    int r = row0 + min(i, rows - 1);
    if (__builtin_expect(a.offsets != nullptr, 0)) {
      if (a.pairs) r = a.pairs[r] / a.top_k;
      r = min(max(r, 0), (int)a.n_rows - 1);
    }
    return (int64_t)r;
  };
  auto load_x = [&](int chunk) {
    int base, own;
    slice_of(chunk, base, own);
    const bool whole = base == own && (base + SX) * 128 <= K;  // the same in all lanes
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int p = 0; p < kFours; ++p) {
        if (4 * (kFours * v + p) >= rows) continue;  // (no result comes of what LDS then holds)
        const int i = 4 * (kFours * v + p) + g;
        const bool here = i < rows;
        const char* x = static_cast<const char*>(a.x) + (x_row(i) * a.ldx + 128 * (int64_t)base + 8 * c) * (f32 ? 4 : 2);
#pragma unroll
        for (int t = 0; t < SX; ++t) {
          u32x4 lo = {0u, 0u, 0u, 0u}, hi = {0u, 0u, 0u, 0u};
          if (here && (whole || (base + t >= own && 128 * (base + t) + 8 * c < K))) {
            lo = get16<false>(x + 128 * t * (f32 ? 4 : 2));
            if constexpr (f32) hi = get16<false>(x + 128 * t * 4 + 16);
          }
          if constexpr (f32) xf[t][v][2 * p] = lo, xf[t][v][2 * p + 1] = hi;
          else xf[t][v][p] = lo;
        }
      }
  };
  // The same where the slice is whole and all four loads of each operand have rows: without a branch, the code tiles one
  // after another, so that the first one's way through LDS begins while the others are under way (20.5
  // us to 19.7 for 47 rows of 14336 x 4096).  (Rows past the last are that one again.)
  auto load_whole = [&]() {
    const char* x[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int p = 0; p < 4; ++p)
        x[v][p] = static_cast<const char*>(a.x) + (x_row(16 * v + 4 * p + g) * a.ldx + 128 * (int64_t)base + 8 * c) * 2;
#pragma unroll
    for (int t = 0; t < SX; ++t)
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int p = 0; p < 4; ++p) xf[t][v][p] = get16<false>(x[v][p] + 256 * t);
  };
  auto make_operands = [&](auto all) {
    if constexpr (!f32) {
#pragma unroll
      for (int t = 0; t < SX; ++t)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
          for (int p = 0; p < 4; ++p)
            if (all || 16 * v + 4 * p < rows) *reinterpret_cast<u32x4*>(mine + (4 * p + g) * kG4StageRow + 16 * c) = xf[t][v][p];
          wave_fence();
#pragma unroll
          for (int s = 0; s < 4; ++s) xf[t][v][s] = *reinterpret_cast<const u32x4*>(mine + c * kG4StageRow + 64 * s + 16 * g);
          wave_fence();
        }
    }
    if constexpr (XT == kBF16) {  // the groups' sums of each row
      const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
      for (int t = 0; t < SX; ++t)
#pragma unroll
        for (int b = 0; b < kSets; ++b)
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < kSteps; ++s) d = mfma_bf16(xf[t][v][b * kSteps + s], ones, d);
            if (c == 0) *reinterpret_cast<f32x4*>(sums + ((t * kSets + b) * NV + v) * 64 + 16 * g) = d;
          }
      wave_fence();
    }
    if constexpr (f32) {
      uint32_t scale[NV][2];  // bits of the power of two
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          if (8 * v + 4 * p >= rows) continue;
          float top = 0.f;  // (a NaN is passed over: it makes its own results NaN whatever the scale is)
#pragma unroll
          for (int t = 0; t < SX; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              top = fmaxf(fmaxf(top, fabsf(__uint_as_float(xf[t][v][2 * p][i]))), fabsf(__uint_as_float(xf[t][v][2 * p + 1][i])));
          // 2^(141 - E) for a largest value of exponent field E, at most 2^126
          const uint32_t f = min(268u - (row_max(__float_as_uint(top)) >> 23), 253u);
          scale[v][p] = f << 23;
          if (c < 2) exps[16 * v + 8 * c + 4 * p + g] = 127 - 11 * c - (int)f;  // (of the rest, 11 less)
        }
#pragma unroll
      for (int t = 0; t < SX; ++t)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            if (8 * v + 4 * p >= rows) continue;
            const float s = __uint_as_float(scale[v][p]);
            float x[8], rest[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[i] = __uint_as_float(xf[t][v][2 * p][i]) * s;
              x[4 + i] = __uint_as_float(xf[t][v][2 * p + 1][i]) * s;
            }
            u32x4 h, m;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              asm("" : "+v"(x[2 * i]), "+v"(x[2 * i + 1]));  // (one packed conversion, not two mixed products)
              h[i] = pack2<kF16>(x[2 * i], x[2 * i + 1]);
              rest[2 * i] = less_lo(x[2 * i], h[i]);
              rest[2 * i + 1] = less_hi(x[2 * i + 1], h[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = pack2<kF16>(rest[2 * i] * 0x1p11f, rest[2 * i + 1] * 0x1p11f);
            uint8_t* to = mine + (4 * p + g) * kG4StageRow + 16 * c;
            *reinterpret_cast<u32x4*>(to) = h;
            *reinterpret_cast<u32x4*>(to + 8 * kG4StageRow) = m;
          }
          wave_fence();
#pragma unroll
          for (int s = 0; s < 4; ++s) xf[t][v][s] = *reinterpret_cast<const u32x4*>(mine + c * kG4StageRow + 64 * s + 16 * g);
          wave_fence();
        }
    }
  };

  // ---- products ---------------------------------------------------------------------------------------
  const G4Consts consts = g4_consts<XT == kBF16>();
  const bool scale_f16 = a.scale_type == kF16;
  f32x4 acc[NV];
  auto multiply = [&](int t, const WTile& w) {
    const uint32_t zeros = a.zeros ? w.z : 0x08080808u;
    float sc[kSets];
    if (scale_f16) {
#pragma unroll
      for (int b = 0; b < kSets; ++b) sc[b] = h2f((uint16_t)(w.s[b >> 1] >> (16 * (b & 1))));
    } else {
#pragma unroll
      for (int b = 0; b < kSets; ++b) sc[b] = __uint_as_float((b & 1) ? w.s[b >> 1] & 0xFFFF0000u : w.s[b >> 1] << 16);
    }
#pragma unroll
    for (int b = 0; b < kSets; ++b) {
      f32x4 d[NV];
      if constexpr (XT == kBF16) {
        const float corr = -16.0f - (float)((zeros >> (8 * b)) & 0xFFu);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const f32x4 sum = *reinterpret_cast<const f32x4*>(sums + ((t * kSets + b) * NV + v) * 64 + 16 * g);
#pragma unroll
          for (int e = 0; e < 4; ++e) d[v][e] = corr * sum[e];
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const u32x4 wf = g4_brain(consts, w.q[b * kSteps + s]);
#pragma unroll
          for (int v = 0; v < NV; ++v) d[v] = mfma_bf16(xf[t][v][b * kSteps + s], wf, d[v]);
        }
      } else {
        // 1024 + z twice: the zero point's byte under the byte 0x64
        const uint32_t bias = __builtin_amdgcn_perm(0x64646464u, zeros, 0x04000400u + 0x00010001u * b);
        const uint32_t bias16 = ((bias << 4) & 0x00F000F0u) | 0xD400D400u;  // -(64 + z) twice
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const u32x4 wf = g4_half<G == 32>(consts, w.q[b * kSteps + s], __builtin_bit_cast(f16x2, bias), __builtin_bit_cast(f16x2, bias16));
#pragma unroll
          for (int v = 0; v < NV; ++v) d[v] = mfma_f16(xf[t][v][b * kSteps + s], wf, s ? d[v] : f32x4{0.f, 0.f, 0.f, 0.f});
        }
      }
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[v][e] = fmaf(d[v][e], sc[b], acc[v][e]);
    }
    // (opaque: or the compiler scales all tiles' sums behind the last one, and holds them until then)
#pragma unroll
    for (int v = 0; v < NV; ++v) asm volatile("" : "+v"(acc[v]));
  };
  // the sums of a row tile and a slice of k, divided by the rows' powers of two, into LDS (or added there)
  auto keep = [&](int rb, bool add) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      f32x4 s = acc[v];
      if constexpr (f32) {  // rows 8 .. 15 have what rows 0 .. 7 left
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[e] = __builtin_amdgcn_ldexpf(s[e], exps[16 * v + 4 * g + e]);
          s[e] += __shfl_xor(s[e], 32);
        }
      }
      f32x4* to = part + (rb * NV + v) * 64 + lane;
      if (add) {
        const f32x4 o = *to;
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = o[e] + s[e];
      }
      *to = s;
    }
  };
  uint64_t odd = 0;  // lanes that had a result that is not finite
  auto store = [&](int t, int64_t at, float v) {  // row t of the tile, column `at`
    if (t >= rows || at >= a.n) return;
    const int64_t o = (int64_t)(row0 + t) * a.ldy + at;
    if (a.y_type == kF32) static_cast<float*>(a.y)[o] = v;
    else static_cast<uint16_t*>(a.y)[o] = (uint16_t)(a.y_type == kF16 ? pack2<kF16>(v, 0.f) : pack2<kBF16>(v, 0.f));
  };

  constexpr int kAhead = SX == 1 ? 4 : SX <= 3 ? 2 : 1;  // row tiles, some 4 KB a wave
  WTile w[kAhead][SX];
  auto first_w = [&]() {
    // (one row tile without a branch, so that a wait for the activations is not one for these too: one row of
    // 4096 x 4096 5.4 us for 5.9; with more, past the last it would load for nothing: 17.6 us for 16.8 for 32
    // rows of 128 experts)
#pragma unroll
    for (int d = 0; d < kAhead; ++d)
#pragma unroll
      for (int t = 0; t < SX; ++t)
        if (kAhead == 1 || first + d < last) load_w((int64_t)(first + d) * kt_n + base + t, w[d][t]);
  };
  // Many activations take longer than the weights, which then come first (47 rows of 14336 x 4096 22.0 us for
  // 24.8; one row the other way round 9.7 for 10.4).
  if (!f32 && rows > 16 * NV - 4 && base == own && (base + SX) * 128 <= K) {
    first_w();
    load_whole();
    make_operands(std::true_type());
  } else {
    if constexpr (NV == 2) first_w();
    load_x(0);
    if constexpr (NV == 1) first_w();
    make_operands(std::false_type());
  }
  for (int b = first; b < last; b += plan.rb) {
    const int tiles = min(plan.rb, last - b);
    for (int chunk = 0; chunk < (CHUNKS ? plan.chunks : 1); ++chunk) {
      if (CHUNKS && (b != first || chunk != 0)) {
        load_x(chunk);
        make_operands(std::false_type());
      }
      for (int rb = 0; rb < tiles; rb += kAhead) {
        // the kAhead row tiles that come after these
        int nr = b + rb + kAhead, nc = chunk;
        if (rb + kAhead >= tiles) {
          nr = b, nc = chunk + 1;
          if (!CHUNKS || nc == plan.chunks) nr = b + plan.rb, nc = 0;
        }
        slice_of(nc, base, own);
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
          if (rb + d < tiles) {
#pragma unroll
            for (int v = 0; v < NV; ++v) acc[v] = f32x4{0.f, 0.f, 0.f, 0.f};
          }
#pragma unroll
          for (int t = 0; t < SX; ++t) {
            if (rb + d < tiles) multiply(t, w[d][t]);
            if (nr + d < last) load_w((int64_t)(nr + d) * kt_n + base + t, w[d][t]);
            __builtin_amdgcn_sched_barrier(0);  // (the tiles' operands, mixed, would not fit the registers)
          }
          if (rb + d < tiles) keep(rb + d, chunk > 0);
        }
      }
    }
    lds_barrier();
    for (int q = slice; q < tiles * NV; q += KS) {
      const uint8_t* p = lds + kXLds + (q * 64 + lane) * 16;
      f32x4 s = *reinterpret_cast<const f32x4*>(p);
      for (int v = 1; v < KS; ++v) {
        const f32x4 o = *reinterpret_cast<const f32x4*>(p + v * wave_lds);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = s[e] + o[e];
      }
      const int v = q % NV;
      const int64_t at = (int64_t)(b + q / NV) * 16 + c;
      if constexpr (XT != kF16) {
// (four rows without any hold what LDS held; a sum past the largest number only looks in vain)
        odd |= __ballot((f32 ? 8 : 16) * v + 4 * g < rows && !(fabsf(s[0]) + fabsf(s[1]) + (fabsf(s[2]) + fabsf(s[3])) < __builtin_inff()));
      }
      if (!f32 || g < 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e) store((f32 ? 8 : 16) * v + 4 * g + e, at, s[e]);
      }
    }
    if (b + plan.rb < last) lds_barrier();  // the sums are read before the next ones are written
  }
  if constexpr (XT != kF16) {
    // Results that are not finite are made again (here, where the operands' registers are free), each from where the
    // lane stored it; those of a row that holds a NaN (a batch's padding may be full of them) are right.  What a row
    // holds a wave looks up once.  (16 rows of 4096 x 4096, eight of them with an infinity 47 us, with a NaN 19, with
    // neither 7 in bfloat16 and 9 in binary32.)
    if (__builtin_expect(odd == 0, 1)) return;
    constexpr int kRows = f32 ? 8 : 16;  // of an operand
    // (counted anew: of the lane number above, what is made of it here would be made before, and kept)
    const int lane = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    const int g = lane >> 4, c = lane & 15;
    uint32_t known = 0, nan = 0, inf = 0;
    for (int b = first; b < last; b += plan.rb)
      for (int q = slice; q < min(plan.rb, last - b) * NV; q += KS) {
        const int64_t rt = b + q / NV;
#pragma nounroll
        for (int e = 0; e < 4; ++e) {
          const int t = kRows * (q % NV) + 4 * g + e;
          bool again = false;
          if (4 * g < kRows && t < rows && rt * 16 + c < a.n && !(nan >> t & 1)) {
            const int64_t o = (int64_t)(row0 + t) * a.ldy + rt * 16 + c;
            if (a.y_type == kF32) again = !(fabsf(static_cast<const float*>(a.y)[o]) < __builtin_inff());
            else again = (~static_cast<const uint16_t*>(a.y)[o] & (a.y_type == kF16 ? 0x7C00 : 0x7F80)) == 0;
          }
#pragma nounroll
          for (int u = 0; u < kRows / 4; ++u) {  // the rows of this e
            if ((__ballot(again) >> (16 * u) & 0xFFFF) == 0) continue;
            const int at = kRows * (q % NV) + 4 * u + e;
            const int64_t xr = x_row(at);
            if (!(known >> at & 1)) {
              uint32_t top = 0;
              const char* row = static_cast<const char*>(a.x) + xr * a.ldx * (f32 ? 4 : 2);
              for (int k = 8 * lane; k < K; k += 512) top = max(top, g4_top<XT>(row, k, K));
              known |= 1u << at;
              if (__ballot(top > 0x7F800000u)) nan |= 1u << at;
              else if (__ballot(top == 0x7F800000u)) inf |= 1u << at;
            }
            if (nan >> at & 1) continue;
            const float v = g4_again<XT, G>(a, W, xr, rt, inf >> at & 1, lane);
            if (again && g == u) store(t, rt * 16 + c, v);
          }
        }
      }
  }
}

template <int XT, int NV, int SX, int G, bool CHUNKS = false>
static int launch_g4_kernel(const G4Args& a, G4Plan p, int64_t places, hipStream_t s) {
  // (at most 4096 workgroups or one a tile of X, 2^21: far from a grid's 2^32 threads)
  p.kt_n = g4_k_tiles(a.k);
  p.rt_n = (int)g4_row_tiles(a.n);
  p.y = p.cols < 32768 ? p.cols : 32768;
  p.chunks = (p.kt_n + p.ks * SX - 1) / (p.ks * SX);
  // Workgroups go to the eight XCDs in turn: with a multiple of eight along the row tiles, those that have the same
  // weights meet in one L2 (60 rows of 13000 x 4096 22.5 us for 23.8).  Only where the device holds those too: the ones
  // without row tiles all fall to the same XCDs, and the others then get more of the rest than they hold (47 rows of
  // 14336 x 6144, 264 for 246 of them, 56 us for 32).  Not by expert, where that would leave some XCDs
  // more workgroups than others (488 rows of 128 experts 35 us for 25).
  unsigned along = (unsigned)((p.rt_n + p.per - 1) / p.per);
  const unsigned even = (along + 7) / 8 * 8;
  if (!a.offsets && p.cols > 1 && along >= 32 && (int64_t)even * p.cols <= places) along = even;
  const dim3 grid(along, (unsigned)p.y, (unsigned)((p.cols + p.y - 1) / p.y));
  const int lds = p.ks * (g4_x_lds(XT, NV, SX, G) + p.rb * NV * 1024);
  hipLaunchKernelGGL((g4_kernel<XT, NV, SX, G, CHUNKS>), grid, dim3(64 * p.ks), lds, s, a, p);
  return check_launch("g4_kernel");
}

// k over up to eight waves, sx code tiles of each in registers (as many as those hold; where that is
// not all of k, one slice after another).
template <int XT, int G>
static int launch_g4_group(const G4Args& a, hipStream_t s) {
  const int64_t rt_n = g4_row_tiles(a.n);
  const int kt_n = g4_k_tiles(a.k);
  int64_t cols, busy;  // tiles of rows of X: the grid's, and those that have rows
  auto columns = [&](int nv) {
    const int bm = XT == kF32 ? 8 * nv : 16 * nv;
    busy = cols = (a.m + bm - 1) / bm;
    if (!a.offsets) return;
    // each expert's last tile may be partial, on average half of one; if the rows choose at random, as many
    // experts as `some` have any
    cols = a.m / bm + a.n_expert < a.m ? a.m / bm + a.n_expert : a.m;
    const double some = a.n_expert * -expm1(-(double)a.m / a.n_expert), tiles = (double)a.m / bm + some / 2;
    busy = (int64_t)ceil(tiles > some ? tiles : some);
    if (busy > cols) busy = cols;
  };
  // Two operands of rows of X where there are rows for them (an expert's on average), all of k fits the registers
  // with them, and they leave every CU a workgroup; by expert, where many tiles are not full, sixteen.
  // bfloat16, 64 rows of 2048 x 4096: 9.9 us with two, 8.5 with one; 33 rows of 4096 x 4096 11.9 and 13.6; 47 rows of
  // 14336 x 6144 37.3 and 29.3; 9 experts of 1991 x 1312 with 32 rows each 17.7 and 14.9; 128 of 2048 x 768 with 19
  // each 47 and 49.
  const int64_t rows = a.offsets ? (a.m + a.n_expert - 1) / a.n_expert : a.m;
  int nv = rows > (XT == kF32 ? 8 : 16) && kt_n <= 32 ? 2 : 1;
  columns(nv);
  if (nv == 2 && rt_n * busy * (kt_n < 8 ? kt_n : 8) <= (a.offsets ? 16 : 1) * 2048) columns(nv = 1);
  int sx = (kt_n + 7) / 8;
  // short rows: two tiles a wave where there is work for twice the device's waves all the same (128 experts
  // of 2048 x 768, 488 rows: 23.4 us for 29.6)
  if (sx == 1 && kt_n > 1 && rt_n * busy * ((kt_n + 1) / 2) >= 8192) sx = 2;
  if (sx == 5) sx = 6;
  if (sx == 3 && nv == 2) sx = 4;
  // longer rows in slices of six tiles or four, whichever fill their last round better (one row of
  // 4096 x 14336: 14.7 us with six, 12.8 with four)
  const bool chunks = sx > 6;
  if (chunks) sx = (kt_n + 47) / 48 * 6 <= (kt_n + 31) / 32 * 4 ? 6 : 4;
  G4Plan p{};
  p.ks = (kt_n + sx - 1) / sx;
  if (p.ks > 8) p.ks = 8;
  p.cols = (int)cols;
  // Row tiles a workgroup: as few as let the device hold all workgroups at once.  Its registers hold 8 waves a CU, or
  // 16 of those with few activations (or one row that soon is operands); of more than four waves, one
  // workgroup or two.  14336 x 4096 in bfloat16, 16 rows: 12.4 us with 8 waves, 16.4 with 16; one row 9.7 and 11.6, in
  // binary16 11.1 and 10.0, four rows 11.2 and 12.2; 128 experts of 1536 x 2048, 32 rows: 16.0 with 32, 14.8
  // with 16.  A few workgroups too many cost as much as all: 33 rows of 4217 x 2944 17.5 us with 264 workgroups of six
  // waves, 13.9 with 176; by expert, where some end early, 128 experts of 2048 x 768 with 488 rows 26.0 with 1500 of
  // three, 21.5 with 1380 (and 22.5 with 1250).
  const bool few = nv * sx < 4 || (XT == kF16 && a.m == 1);
  const int64_t places = p.ks <= 4 ? (few ? 4096 : 2048) / p.ks : few ? 512 : 256;
  // workgroups along the row tiles, which share them evenly
  const int64_t share = (rt_n * busy + places - 1) / places;
  int64_t along = a.offsets ? (rt_n + share - 1) / share : busy < places ? places / busy : 1;
  if (along > rt_n) along = rt_n;
  p.per = (int)((rt_n + along - 1) / along);
  // joins: every four row tiles (a multiple of those that a wave loads ahead), or, where each would load X again,
  // as many as the CU's LDS holds (57 rows of 6097 x 8768, six row tiles each: 49.5 us with two joins, 40.9 with one)
  const int room = (160 * 1024 / 8 - g4_x_lds(XT, 1, 6, G)) / 1024;
  const int rb = chunks ? room : 4;
  p.rb = p.per < rb ? p.per : rb;
  if (chunks) return sx == 6 ? launch_g4_kernel<XT, 1, 6, G, true>(a, p, places, s) : launch_g4_kernel<XT, 1, 4, G, true>(a, p, places, s);
  switch (10 * nv + sx) {
    case 11: return launch_g4_kernel<XT, 1, 1, G>(a, p, places, s);
    case 12: return launch_g4_kernel<XT, 1, 2, G>(a, p, places, s);
    case 13: return launch_g4_kernel<XT, 1, 3, G>(a, p, places, s);
    case 14: return launch_g4_kernel<XT, 1, 4, G>(a, p, places, s);
    case 16: return launch_g4_kernel<XT, 1, 6, G>(a, p, places, s);
    case 21: return launch_g4_kernel<XT, 2, 1, G>(a, p, places, s);
    case 22: return launch_g4_kernel<XT, 2, 2, G>(a, p, places, s);
    default: return launch_g4_kernel<XT, 2, 4, G>(a, p, places, s);
  }
}

}  // namespace iq4
