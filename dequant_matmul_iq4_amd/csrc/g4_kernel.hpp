// g4_kernel.hpp -- the product of few rows with group-scaled 4-bit weights (g4.hpp): the kernel
// and its launch, compiled once per type of the activations (g4_f32.hip, g4_f16.hip, g4_bf16.hip).
//
// Mathematics.  With d = sum over 32 (or the whole group's) k of (q - z) x, a row's result is the
// sum of s d over its groups.  q - z is a whole number of four bits and a sign, exact in binary16
// and in bfloat16, so the matrix instruction's products are exact and its sums are binary32;
// each group's d is scaled by one fused multiply-add.  No weight is rounded anywhere.
//
// Operands of v_mfma_f32_16x16x32 (lane l = 16 g + c): the activations are the first one, rows of
// X by c; the weights the second, 16 rows of W by c, so that a lane's scale is that of the row
// whose codes it holds; the lane receives D[4g + i][c], four rows of X times row c of W.
//   binary16  q - z = (1024 + q) - (1024 + z), two at a time (the codes are or-ed into the bits
//             of 1024): 11 operations for eight weights.
//   bfloat16  q - z = (128 + q) - (128 + z) by a two-term dot product with (1, 0) or (0, 1) into
//             binary32, then rounded (exactly) in pairs: 19 operations.
//   binary32  an activation is the sum of three bfloat16 numbers, its leading, middle and last
//             eight bits (cut, not rounded: exact, and no part overflows).  Up to four rows:
//             row 4 p + t of the first operand is part p of row t, one instruction for all parts;
//             more rows: three instructions.
#pragma once
#include "experts.hpp"
#include "g4.hpp"
#include "pieces.hpp"

namespace iq4 {

enum G4Mode {
  kG4Half,     // binary16 activations, 16 rows a tile
  kG4Brain,    // bfloat16, 16 rows a tile
  kG4Parts4,   // binary32, four rows a tile: the parts are rows of the operand
  kG4Parts16,  // binary32, 16 rows a tile: one instruction per part
};

// Eight weights, q - z, as matrix-core operand; `z` is the zero point's byte of a word.
__device__ __forceinline__ u32x4 g4_half(uint32_t w, uint32_t bias) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u;
    const f16x2 d = __builtin_bit_cast(f16x2, v) - __builtin_bit_cast(f16x2, bias);
    r[i] = __builtin_bit_cast(uint32_t, d);
  }
  return r;
}
__device__ __forceinline__ u32x4 g4_brain(uint32_t w, float bias, uint32_t one_lo, uint32_t one_hi) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf16x2 v = __builtin_bit_cast(bf16x2, ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u);
    const bf16x2 d = {(__bf16)__builtin_amdgcn_fdot2_f32_bf16(v, __builtin_bit_cast(bf16x2, one_lo), bias, false),
                      (__bf16)__builtin_amdgcn_fdot2_f32_bf16(v, __builtin_bit_cast(bf16x2, one_hi), bias, false)};
    r[i] = __builtin_bit_cast(uint32_t, d);
  }
  return r;
}

// The three parts of eight binary32 numbers.  An infinity's rest counts as zero (infinity minus
// itself would make a NaN of it).
struct G4Parts {
  u32x4 p[3];
};
__device__ __forceinline__ G4Parts g4_parts(const u32x4 (&x)[2]) {
  G4Parts r;
  float v[8], top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(x[i >> 2][i & 3]);
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
  const bool inf = __ballot(top == __builtin_inff()) != 0;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.p[q][i] = __builtin_amdgcn_perm(__float_as_uint(v[2 * i + 1]), __float_as_uint(v[2 * i]), 0x07060302u);
    if (q == 2) break;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float rest = v[i] - __uint_as_float(__float_as_uint(v[i]) & 0xFFFF0000u);
      if (inf) rest = fabsf(v[i]) == __builtin_inff() ? 0.f : rest;
      v[i] = rest;
    }
  }
  return r;
}

// A workgroup of KS waves: RT row tiles of W against one tile of NT x 16 (kG4Parts4: 4) rows of
// X, k split over the waves (wave s takes the code tiles s, s + KS, ...), whose sums are added
// through LDS in the waves' order.  Every operand goes from memory straight into registers, D
// tiles of 128 along k ahead of its products.
template <int XM, int NT, int RT, int G, int D>
__global__ void __launch_bounds__(512) g4_kernel(G4Args a, uint32_t row_groups, uint32_t cols) {
  constexpr int kTok = XM == kG4Parts4 ? 4 : 16, kBM = kTok * NT, kMaxWaves = 8;
  constexpr int kXs = XM == kG4Parts4 ? 2 : XM == kG4Parts16 ? 8 : 4;  // 16-byte words of a row tile's x a lane
  constexpr int kSets = 128 / G, kSteps = G / 32;                     // groups of a code tile, steps of a group
  constexpr int kElem = XM == kG4Half || XM == kG4Brain ? 2 : 4;
  constexpr int kStageRow = 128 * 2 + 16;  // a part's row of 128, 16 bytes on: 16 rows begin in different banks
  __shared__ f32x4 part[kMaxWaves * RT * NT * 64];
  __shared__ uint8_t stage[XM == kG4Parts4 ? kMaxWaves * 12 * kStageRow : 16];
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int slice = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), KS = blockDim.x >> 6;
  // workgroups go round-robin to eight XCDs: the column tiles that share rows of W go to one
  const uint32_t in = blockIdx.x / 8, rg = in / cols * 8 + blockIdx.x % 8;
  const int col = (int)(in % cols);
  if (rg >= row_groups) return;
  const uint8_t* W = a.W;
  int row0 = col * kBM, rows;
  if (a.offsets) {
    int e;
    if (!expert_tile(a.offsets, a.n_expert, (int)a.m, kBM, col, e, row0, rows)) return;
    W += e * a.w_stride;
  } else {
    rows = (int)min((int64_t)kBM, a.m - row0);
  }
  const int kt_n = g4_k_tiles(a.k), kq_n = g4_k_quads(a.k), K = (int)a.k;
  const int64_t rt_n = g4_row_tiles(a.n), rt0 = (int64_t)rg * RT;
  const uint8_t* wq[RT];
  const uint8_t* ws[RT];
  const uint8_t* wz[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {  // row tiles past the last repeat it and are not stored
    const int64_t rt = min(rt0 + r, rt_n - 1);
    wq[r] = W + rt * kt_n * kG4TileBytes + lane * 16;
    ws[r] = W + g4_code_plane(a.n, a.k) + (rt * kq_n * 16 + c) * (512 / G) * 2;
    wz[r] = W + g4_code_plane(a.n, a.k) + g4_scale_plane(a.n, a.k, G) + (rt * kq_n * 16 + c) * (512 / G);
  }
  struct WTile {
    u32x4 q[RT];
    uint32_t s[RT][G == 32 ? 2 : 1], z[RT];
  };
  struct XTile {
    u32x4 x[NT][kXs];
  };
  auto load_w = [&](int j, WTile& o) {
    const int at = (j >> 2) * 16 * (512 / G) + (j & 3) * kSets;  // in scales
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      o.q[r] = *reinterpret_cast<const u32x4*>(wq[r] + (int64_t)j * kG4TileBytes);
      if constexpr (G == 32) {
        const u32x2 s = *reinterpret_cast<const u32x2*>(ws[r] + 2 * at);
        o.s[r][0] = s[0], o.s[r][1] = s[1];
      } else if constexpr (G == 64) {
        o.s[r][0] = *reinterpret_cast<const uint32_t*>(ws[r] + 2 * at);
      } else {
        o.s[r][0] = *reinterpret_cast<const uint16_t*>(ws[r] + 2 * at);
      }
      o.z[r] = 0x08080808u;
      if (a.zeros) {
        if constexpr (G == 32) o.z[r] = *reinterpret_cast<const uint32_t*>(wz[r] + at);
        else if constexpr (G == 64) o.z[r] = *reinterpret_cast<const uint16_t*>(wz[r] + at);
        else o.z[r] = *(wz[r] + at);
      }
    }
  };
  // this lane's rows of X: row 16 i + c of the tile (rows past the last repeat it and are not
  // stored), from element 8 g on; kG4Parts4: row g, from element 8 c on
  const uint8_t* xp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    int64_t r = row0 + min(XM == kG4Parts4 ? g : 16 * i + c, rows - 1);
    if (a.pairs) r = a.pairs[r] / a.top_k;
    if (a.offsets) r = min(max(r, (int64_t)0), a.n_rows - 1);
    xp[i] = static_cast<const uint8_t*>(a.x) + (r * a.ldx + 8 * (XM == kG4Parts4 ? c : g)) * kElem;
  }
  auto load_x = [&](int j, XTile& o) {
    if constexpr (XM == kG4Parts4) {
      const uint8_t* p = xp[0] + (int64_t)j * 128 * 4;
      o.x[0][0] = o.x[0][1] = u32x4{0u, 0u, 0u, 0u};
      if (128 * j + 8 * c < K) o.x[0][0] = get16<false>(p), o.x[0][1] = get16<false>(p + 16);
    } else {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint8_t* p = xp[i] + ((int64_t)j * 128 + 32 * s) * kElem;
          const bool is = 128 * j + 32 * s < K;  // the same in all lanes
          if constexpr (XM == kG4Parts16) {
            o.x[i][2 * s] = o.x[i][2 * s + 1] = u32x4{0u, 0u, 0u, 0u};
            if (is) o.x[i][2 * s] = get16<false>(p), o.x[i][2 * s + 1] = get16<false>(p + 16);
          } else {
            o.x[i][s] = u32x4{0u, 0u, 0u, 0u};
            if (is) o.x[i][s] = get16<false>(p);
          }
        }
      }
    }
  };
  f32x4 acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint32_t one_lo = 0x00003F80u, one_hi = 0x3F800000u;  // (1, 0) and (0, 1) as bfloat16 pairs
  asm("" : "+s"(one_lo), "+s"(one_hi));                   // opaque: kept in registers
  uint8_t* mine = stage + (XM == kG4Parts4 ? slice * 12 * kStageRow : 0);
  auto multiply = [&](const WTile& w, const XTile& x) {
    u32x4 xf[4];  // kG4Parts4: the four steps' operands
    if constexpr (XM == kG4Parts4) {
      // from row g, elements 8 c .. 8 c + 7 to the parts' rows; the wave's own LDS, in order
      const G4Parts p = g4_parts(x.x[0]);
#pragma unroll
      for (int q = 0; q < 3; ++q) *reinterpret_cast<u32x4*>(mine + (4 * q + g) * kStageRow + 16 * c) = p.p[q];
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      const uint8_t* row = mine + (c < 12 ? c : c - 12) * kStageRow + 16 * g;  // (rows 12 .. 15 of the result are not used)
#pragma unroll
      for (int s = 0; s < 4; ++s) xf[s] = *reinterpret_cast<const u32x4*>(row + 64 * s);
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
#pragma unroll
    for (int b = 0; b < kSets; ++b) {
      f32x4 d[RT][NT];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < NT; ++i) d[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < kSteps; ++t) {
        const int s = b * kSteps + t;
        u32x4 wf[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          if constexpr (XM == kG4Half) {
            // 1024 + z twice: the zero point's byte under the byte 0x64
            const uint32_t bias = __builtin_amdgcn_perm(0x64646464u, w.z[r], 0x04000400u + 0x00010001u * b);
            wf[r] = g4_half(w.q[r][s], bias);
          } else {
            wf[r] = g4_brain(w.q[r][s], -128.0f - (float)((w.z[r] >> (8 * b)) & 0xFFu), one_lo, one_hi);
          }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if constexpr (XM == kG4Half) {
#pragma unroll
            for (int r = 0; r < RT; ++r) d[r][i] = mfma_f16(x.x[i][s], wf[r], d[r][i]);
          } else if constexpr (XM == kG4Brain) {
#pragma unroll
            for (int r = 0; r < RT; ++r) d[r][i] = mfma_bf16(x.x[i][s], wf[r], d[r][i]);
          } else if constexpr (XM == kG4Parts4) {
#pragma unroll
            for (int r = 0; r < RT; ++r) d[r][i] = mfma_bf16(xf[s], wf[r], d[r][i]);
          } else {
            const u32x4 two[2] = {x.x[i][2 * s], x.x[i][2 * s + 1]};
            const G4Parts p = g4_parts(two);
#pragma unroll
            for (int q = 2; q >= 0; --q)
#pragma unroll
              for (int r = 0; r < RT; ++r) d[r][i] = mfma_bf16(p.p[q], wf[r], d[r][i]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const uint32_t bits = w.s[r][b >> 1] >> (16 * (b & 1)) & 0xFFFFu;
        const float sc = a.scale_type == kF16 ? h2f((uint16_t)bits) : __uint_as_float(bits << 16);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][i][e] = fmaf(d[r][i][e], sc, acc[r][i][e]);
      }
    }
  };
  const int n = (kt_n - slice + KS - 1) / KS;
  WTile w[D];
  XTile x[D];
#pragma unroll
  for (int v = 0; v < D; ++v)
    if (v < n) {
      load_w(slice + v * KS, w[v]);
      load_x(slice + v * KS, x[v]);
    }
  for (int i0 = 0; i0 < n; i0 += D) {
#pragma unroll
    for (int v = 0; v < D; ++v) {
      const int i = i0 + v;
      if (i >= n) break;
      multiply(w[v], x[v]);
      if (i + D < n) {
        load_w(slice + (i + D) * KS, w[v]);
        load_x(slice + (i + D) * KS, x[v]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < NT; ++i) part[((slice * RT + r) * NT + i) * 64 + lane] = acc[r][i];
  __syncthreads();
  auto store = [&](int t, int64_t at, float v) {  // row t of the tile, column `at`
    if (t >= rows || at >= a.n) return;
    const int64_t o = (int64_t)(row0 + t) * a.ldy + at;
    if (a.y_type == kF32) static_cast<float*>(a.y)[o] = v;
    else static_cast<uint16_t*>(a.y)[o] = (uint16_t)(a.y_type == kF16 ? pack2<kF16>(v, 0.f) : pack2<kBF16>(v, 0.f));
  };
  for (int q = slice; q < RT * NT; q += KS) {
    const int r = q / NT, i = q % NT;
    if (rt0 + r >= rt_n) continue;
    const int64_t at = (rt0 + r) * 16 + c;
    if constexpr (XM == kG4Parts4) {  // lane (g, c): row g, the sum over its three parts
      float s = 0.f;
      for (int v = 0; v < KS; ++v)
#pragma unroll
        for (int p = 0; p < 3; ++p) s = s + part[(v * RT + r) * 64 + 16 * p + c][g];
      store(g, at, s);
    } else {
      f32x4 s = part[q * 64 + lane];
      for (int v = 1; v < KS; ++v) {
        const f32x4 o = part[(v * RT * NT + q) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = s[e] + o[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) store(16 * i + 4 * g + e, at, s[e]);
    }
  }
}

template <int XM, int NT, int RT, int G, int D>
static int launch_g4_tile(const G4Args& a, hipStream_t s) {
  constexpr int kBM = (XM == kG4Parts4 ? 4 : 16) * NT;
  const int64_t row_groups = (g4_row_tiles(a.n) + RT - 1) / RT;
  int64_t cols = (a.m + kBM - 1) / kBM;
  // by expert: each expert's last tile may be partial
  if (a.offsets) cols = a.m / kBM + a.n_expert < a.m ? a.m / kBM + a.n_expert : a.m;
  const int kt_n = g4_k_tiles(a.k);
  int ks = kt_n < 8 ? kt_n : 8;
  const int each = (kt_n + ks - 1) / ks;
  ks = (kt_n + each - 1) / each;
  const int64_t groups = (row_groups + 7) / 8 * 8 * cols;
  if (groups * 64 * ks >= (int64_t)1 << 32)
    return set_error(-3, "iq4_g4 product: too many workgroups (n * m too large)");
  hipLaunchKernelGGL((g4_kernel<XM, NT, RT, G, D>), dim3((unsigned)groups), dim3(64 * ks), 0, s, a, (uint32_t)row_groups,
                     (uint32_t)cols);
  return check_launch("g4_kernel");
}

template <int XM, int NT, int RT, int D>
static int launch_g4_group(const G4Args& a, hipStream_t s) {
  if (a.group == 32) return launch_g4_tile<XM, NT, RT, 32, D>(a, s);
  if (a.group == 64) return launch_g4_tile<XM, NT, RT, 64, D>(a, s);
  return launch_g4_tile<XM, NT, RT, 128, D>(a, s);
}

}  // namespace iq4
