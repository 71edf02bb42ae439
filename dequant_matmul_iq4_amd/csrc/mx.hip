// mx.hip -- products of microscaled rows: Y = X W^T with W in MXFP4 and X in MXFP4 or
// MXFP8 rows (rows.hpp), fp32 sums, on gfx950's scaled matrix instruction
// v_mfma_scale_f32_16x16x128_f8f6f4: 16 x 16 outputs, 128 products each, the powers of two
// of both operands' blocks of 32 applied inside the instruction (no decoded weight exists
// anywhere).  One matrix, or one matrix per expert with the rows sorted by expert.
//
// Operand layout (lane l = 16 g + c).  E2M1: the lane holds elements 32g .. 32g+31 of row c,
// 16 bytes.  E4M3: elements 16g .. 16g+15 and 64+16g .. 64+16g+15 of row c, 32 bytes.
// Either way the lane's scale byte is that of the row's block g.  The weights are the first
// operand, so the lane receives D[4g + i][c]: four consecutive columns of one row of Y.
#include <type_traits>

#include "common.hpp"
#include "mx.hpp"
#include "rows.hpp"

namespace iq4 {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ---- pack -------------------------------------------------------------------------------
// Code tile (rt, kt) at (rt * KT + kt) * 1024: lane 16g + c has the 16 bytes of row 16 rt + c,
// block 4 kt + g.  Scale word of four tiles (rt, kq) after all codes, at (rt * KQ + kq) * 256:
// lane 16g + c, byte j has the scale of block 4 (4 kq + j) + g.  What lies past n or k is zero
// (a zero code times any scale below 255 adds nothing).
// A lane moves the 16-byte blocks of four tiles and a scale word, so that the packed form is
// written in whole kilobytes.  Run once per matrix: 14336 x 4096, 31 MB each way, 35 us (1.8 TB/s, a
// copy takes 12): blocks are loaded byte by byte, which spares the source any alignment.  A small matrix
// is a launch: 128 of 1536 x 2048 in 128 calls 910 us, 7.1 each.
__global__ void __launch_bounds__(256) mx_pack_kernel(const uint8_t* __restrict__ codes, int64_t ldq,
                                                      const uint8_t* __restrict__ scales, int64_t lds, int64_t n,
                                                      int blocks, int kt_n, int kq_n, uint8_t* __restrict__ packed) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t quad = i >> 6;  // four tiles along k
  const int lane = (int)(i & 63), g = lane >> 4, c = lane & 15;
  const int64_t rt = quad / kq_n;
  const int kq = (int)(quad - rt * kq_n);
  if (rt >= mx_row_tiles(n)) return;
  const int64_t row = rt * 16 + c;
  uint32_t sw = 0;
  for (int j = 0; j < 4; ++j) {
    const int kt = 4 * kq + j;
    if (kt >= kt_n) break;
    const int b = 4 * kt + g;
    const bool in = row < n && b < blocks;
    uint8_t* o = packed + (rt * kt_n + kt) * kMxTileBytes + lane * 16;
    uint32_t w[4];
    for (int q = 0; q < 4; ++q) {  // byte by byte: the source's rows need no alignment
      uint32_t v = 0;
      if (in)
        for (int e = 0; e < 4; ++e) v |= (uint32_t)codes[row * ldq + 16 * (int64_t)b + 4 * q + e] << (8 * e);
      w[q] = v;
    }
    *reinterpret_cast<u32x4*>(o) = u32x4{w[0], w[1], w[2], w[3]};
    if (in) sw |= (uint32_t)scales[row * lds + b] << (8 * j);
  }
  *reinterpret_cast<uint32_t*>(packed + mx_row_tiles(n) * kt_n * kMxTileBytes + quad * kMxScaleBytes + lane * 4) = sw;
}

int launch_mx_pack(const uint8_t* codes, int64_t ldq, const uint8_t* scales, int64_t lds, int64_t n, int64_t k,
                   uint8_t* packed, hipStream_t s) {
  const int64_t waves = mx_row_tiles(n) * mx_k_quads(k);
  hipLaunchKernelGGL(mx_pack_kernel, dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, s, codes, ldq, scales, lds, n,
                     (int)(k / 32), mx_k_tiles(k), mx_k_quads(k), packed);
  return check_launch("mx_pack_kernel");
}

// ---- shared pieces ------------------------------------------------------------------------

// A launch has fewer than 2^32 threads.
static int check_grid(int64_t groups, int threads) {
  if (groups * threads >= (int64_t)1 << 32) return set_error(-3, "iq4_mx product: too many workgroups (n * m too large)");
  return 0;
}

template <int FMT>
struct Act {  // one 16-row x 128-element operand of activations
  static constexpr int kWords = FMT == kRowsMxfp4 ? 4 : 8;
  static constexpr int kTileBytes = FMT == kRowsMxfp4 ? 64 : 128;  // of one row
};

// An MXFP8 operand is multiplied in two parts, the codes of magnitude 2 and above and the
// rest (exponent bit 3 of E4M3, bit 6 of the byte, tells which; the other part's codes are
// zero).  An instruction adds small groups of neighbouring products first, and such a sum keeps 13
// binary places below the largest of the group's exponents (a product's counted as the sum of its
// codes').  Over the whole range of E4M3 that is not enough: it lost up to 5.6e-5 of the sum of the
// magnitudes.  The upper part's products have exponents up to 8 + 2 and their last place at 2^-2 * 2^-1,
// 13 below; the lower part's up to 0 + 2 and 2^-9 * 2^-1, 12 below; E2M1 ones (no split) 4 and 2^-2.  So
// no group loses anything, and as a group lies within a block, whatever the scales are.  The groups'
// sums are added as binary32 ones: with one scale every sum of 128 products measured was the exact one,
// rounded once; with scales up to 2^20 apart in a row they were off by up to 5e-7 of the magnitudes.
template <int FMT>
struct Frag {
  u32x4 lo[Act<FMT>::kWords / 4], hi[FMT == kRowsMxfp4 ? 1 : 2];
};
template <int FMT>
__device__ __forceinline__ Frag<FMT> split(const u32x4 (&x)[Act<FMT>::kWords / 4]) {
  Frag<FMT> f;
  if constexpr (FMT == kRowsMxfp4) {
    f.lo[0] = x[0];
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // bit 6 of every byte spread over the byte: the permute's selectors 8 .. 11 give the signs
        // of the second operand's and the first operand's 16-bit halves
        const uint32_t mask = __builtin_amdgcn_perm(x[h][i] << 9, x[h][i] << 1, 0x090B080Au);
        f.hi[h][i] = x[h][i] & mask;
        f.lo[h][i] = x[h][i] ^ f.hi[h][i];
      }
  }
  return f;
}

// acc += W X^T of one 16 x 16 x 128 step; `sel` is the byte of the weights' scale word.
template <int FMT, int SEL>
__device__ __forceinline__ f32x4 mma(u32x4 w, uint32_t sw, const Frag<FMT>& x, uint32_t sx, f32x4 acc) {
  const i32x8 a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  if constexpr (FMT == kRowsMxfp4) {
    const i32x8 b = {(int)x.lo[0][0], (int)x.lo[0][1], (int)x.lo[0][2], (int)x.lo[0][3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 4, SEL, (int)sw, 0, (int)sx);
  } else {
    i32x8 l, h;
#pragma unroll
    for (int i = 0; i < 8; ++i) l[i] = (int)x.lo[i >> 2][i & 3], h[i] = (int)x.hi[i >> 2][i & 3];
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, l, acc, 4, 0, SEL, (int)sw, 0, (int)sx);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, h, acc, 4, 0, SEL, (int)sw, 0, (int)sx);
  }
}
template <int FMT>
__device__ __forceinline__ f32x4 mma(int sel, u32x4 w, uint32_t sw, const Frag<FMT>& x, uint32_t sx, f32x4 acc) {
  switch (sel) {
    case 0: return mma<FMT, 0>(w, sw, x, sx, acc);
    case 1: return mma<FMT, 1>(w, sw, x, sx, acc);
    case 2: return mma<FMT, 2>(w, sw, x, sx, acc);
    default: return mma<FMT, 3>(w, sw, x, sx, acc);
  }
}

// acc += W X^T of one 32 x 32 x 64 half step: byte J of the weights' scale word, byte 2 H of
// the rows'.
template <int FMT, int J, int H>
__device__ __forceinline__ f32x16 mma32(u32x4 w, uint32_t sw, const Frag<FMT>& x, uint32_t sx, f32x16 acc) {
  const i32x8 a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  if constexpr (FMT == kRowsMxfp4) {
    const i32x8 b = {(int)x.lo[0][0], (int)x.lo[0][1], (int)x.lo[0][2], (int)x.lo[0][3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, 4, 4, J, (int)sw, 2 * H, (int)sx);
  } else {
    i32x8 l, h;
#pragma unroll
    for (int i = 0; i < 8; ++i) l[i] = (int)x.lo[i >> 2][i & 3], h[i] = (int)x.hi[i >> 2][i & 3];
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, l, acc, 4, 0, J, (int)sw, 2 * H, (int)sx);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, h, acc, 4, 0, J, (int)sw, 2 * H, (int)sx);
  }
}

// Four consecutive columns of a row of Y; `left` of them exist.
__device__ __forceinline__ void store_y4(const MxArgs& a, int64_t row, int64_t col, f32x4 v) {
  const int64_t left = a.n - col;
  if (left <= 0) return;
  const int64_t at = row * a.ldy + col;
  if (a.y_type == kF32) {
    float* o = static_cast<float*>(a.y) + at;
    if (a.vec_y && left >= 4) {
      *reinterpret_cast<f32x4*>(o) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) o[i] = v[i];
    }
    return;
  }
  uint16_t* o = static_cast<uint16_t*>(a.y) + at;
  const u32x2 p = a.y_type == kF16 ? u32x2{pack2<kF16>(v[0], v[1]), pack2<kF16>(v[2], v[3])}
                                   : u32x2{pack2<kBF16>(v[0], v[1]), pack2<kBF16>(v[2], v[3])};
  if (a.vec_y && left >= 4) {
    *reinterpret_cast<u32x2*>(o) = p;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) o[i] = (uint16_t)(p[i >> 1] >> (16 * (i & 1)));
  }
}

// ---- rows by expert -------------------------------------------------------------------------
// The rows [o0[c], o1[c]) of experts e0 + 64 c + lane, clamped to [0, m]: whatever the offsets
// hold, no row outside is touched.  All loads at once; the upper two sets only if they hold an expert
// (nothing is to be done for them if this says false).
constexpr int kGroupExperts = 256;
__device__ __forceinline__ bool expert_rows(const MxArgs& a, int e0, int (&o0)[4], int (&o1)[4]) {
  const int m = (int)a.m, lane = threadIdx.x & 63;
  const bool upper = e0 + 128 < a.n_expert;
  auto load = [&](int c) {
    const int el = min(e0 + 64 * c + lane, a.n_expert - 1);
    o0[c] = a.offsets[el];
    o1[c] = a.offsets[el + 1];
  };
  auto clamp = [&](int c) {
    o0[c] = min(max(o0[c], 0), m);
    o1[c] = e0 + 64 * c + lane < a.n_expert ? min(max(o1[c], o0[c]), m) : o0[c];
  };
  load(0), load(1);
  if (upper) load(2), load(3);
  else o0[2] = o1[2] = o0[3] = o1[3] = 0;
  clamp(0), clamp(1);
  if (upper) clamp(2), clamp(3);
  return upper;
}

// Sums of a value over lanes 0 .. own (one wave, without LDS: row shifts and broadcasts).
__device__ __forceinline__ int scan64(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);  // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);  // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);  // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1, 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2, 3
  return v;
}

// The tiles of `bm` rows that the experts' rows make, found by every wave on its own from the
// offsets: lanes hold the experts 64 c + lane, four c at a time.
struct ExpertTiles {
  int row[4], rows[4], upto[4];  // first row, rows, tiles of the group's experts up to this one
  int total;                     // tiles of the group
};
__device__ __forceinline__ ExpertTiles group_tiles(const MxArgs& a, int e0, int bm) {
  ExpertTiles g;
  int o1[4];
  const bool upper = expert_rows(a, e0, g.row, o1);
  g.total = 0;
  auto add = [&](int c) {
    g.rows[c] = o1[c] - g.row[c];
    g.upto[c] = g.total + scan64((g.rows[c] + bm - 1) / bm);
    g.total = __builtin_amdgcn_readlane(g.upto[c], 63);
  };
  add(0), add(1);
  if (upper) add(2), add(3);
  else g.rows[2] = g.rows[3] = 0, g.upto[2] = g.upto[3] = g.total;
  return g;
}
// Tile t < g.total of the group: its expert, first row and rows.
__device__ __forceinline__ void group_find(const ExpertTiles& g, int e0, int t, int bm, int& e, int64_t& row0, int& rows) {
  int c = 0, row = g.row[0], count = g.rows[0], upto = g.upto[0];
#pragma unroll
  for (int q = 1; q < 4; ++q) {  // (selects: an index would put the sets into memory)
    const bool past = __builtin_amdgcn_readlane(g.upto[q - 1], 63) <= t;
    c = past ? q : c;
    row = past ? g.row[q] : row;
    count = past ? g.rows[q] : count;
    upto = past ? g.upto[q] : upto;
  }
  const int l = __builtin_ctzll(__ballot(upto > t) | 1ull << 63);
  const int mine = __builtin_amdgcn_readlane(count, l);
  const int at = (t - (__builtin_amdgcn_readlane(upto, l) - (mine + bm - 1) / bm)) * bm;  // rows before it
  e = e0 + 64 * c + l;
  row0 = __builtin_amdgcn_readlane(row, l) + at;
  rows = min(bm, mine - at);
}

// Activation row of a pair (or p itself, without pairs), inside the buffer whatever `pairs` holds.
__device__ __forceinline__ int act_row(const MxArgs& a, int p) {
  // p / top_k: p is below 2^22, so (p + 1/2) / top_k is further from a whole number (1 / (2 top_k))
  // than the product's error (2^-23 of it)
  const int r = a.pairs ? (int)(((float)p + 0.5f) * a.inv_top) : p;
  return min(max(r, 0), (int)a.n_rows - 1);
}

// ---- few rows -----------------------------------------------------------------------------
// A workgroup of KS waves: a row tile of W against MT x 16 rows of Y, its k split over the waves
// (wave s takes the quads s, s + KS, ...), whose sums are added through LDS in the waves'
// order.  (One tile a workgroup: a wave's place is free as soon as it ends.  Four waves of one
// tile each: 128 experts of 2048 x 768, 128 pairs 16.1 us, one wave 15.1; 32 pairs of 1536 x 2048,
// MXFP8 12.8 for 12.0; 50000 x 2048, m = 4 13.9 for 12.6.)  Every operand goes from memory straight into registers, the
// rows one quad (four tiles along k) ahead of their products, the weights kAhead quads.
//
// Bound by the weights' way from memory: a row tile's quad is 4.3 KB for 4 (MXFP8 8)
// instructions of 16 clocks.  The waves over k are there to have enough of it under way.  In
// graphs of launches: 4096 x 4096, m = 1 3.3 us (2.7 TB/s; an empty launch takes 1.7); 2560 x 6144,
// m = 4, MXFP8 4.9 to 5.8 by the card; 128 experts of 1536 x 2048, 32 pairs, MXFP8 12.1 (2.6 TB/s).
// (2560 rows and eight waves, in one run: k = 4096, a quad a wave, 5.1 us; 6144, two quads in half of the
// waves, 5.8, in MXFP4 4.8; 8192, two in each, 6.6.  The quads' loads are all under way at once: it is the
// bytes, the second quad and, for MXFP8, twice the loads of rows and twice the instructions.)
//
// Rows by expert: workgroup column i stands for output row i; it works if row i begins a tile
// of its expert (MT x 16 rows from the expert's first on), so a wave finds its expert with one
// comparison per expert and no sum over them.
template <int FMT, int MT, int KS, bool GROUPED>
__global__ void __launch_bounds__(64 * KS) mx_rows_kernel(MxArgs a) {
  __shared__ f32x4 part[KS > 1 ? KS * MT * 64 : 1];
  constexpr int kWords = Act<FMT>::kWords / 4, kAhead = 2;
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int slice = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t rt_n = mx_row_tiles(a.n), rt = blockIdx.x % rt_n, at = blockIdx.x / rt_n;
  const uint8_t* W = a.W;
  int64_t row0 = at * (16 * MT);
  int rows = 16 * MT;
  if constexpr (GROUPED) {
    const int i = (int)at;
    int o0 = 0, o1 = 0, e = -1;
    for (int e0 = 0; e0 < a.n_expert; e0 += kGroupExperts) {
      int b0[4], b1[4];
      expert_rows(a, e0, b0, b1);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint64_t in = __ballot(b0[q] <= i && i < b1[q]);
        if (in && e < 0) {
          const int l = __builtin_ctzll(in);
          e = e0 + 64 * q + l;
          o0 = __builtin_amdgcn_readlane(b0[q], l);
          o1 = __builtin_amdgcn_readlane(b1[q], l);
        }
      }
    }
    if (e < 0 || (i - o0) % (16 * MT)) return;
    W += e * a.w_stride;
    row0 = i;
    rows = min(rows, o1 - i);
  } else {
    rows = (int)min((int64_t)rows, a.m - row0);
  }
  const int kt_n = mx_k_tiles(a.k), kq_n = mx_k_quads(a.k);
  const uint8_t* wc = W + rt * kt_n * kMxTileBytes + lane * 16;
  const uint8_t* ws = W + mx_code_plane(a.n, a.k) + rt * kq_n * kMxScaleBytes + lane * 4;
  struct WQuad {
    u32x4 w[4];
    uint32_t s;
  };
  struct XQuad {
    u32x4 x[MT][4][kWords], s[MT];
  };
  // this wave's quad number u is slice + u KS (tiles past the last repeat it and are not multiplied)
  const int u_n = (kq_n - slice + KS - 1) / KS;
  auto load_w = [&](int u, WQuad& o) {
    if (u >= u_n) return;
    const int q = slice + u * KS;
    o.s = *reinterpret_cast<const uint32_t*>(ws + (int64_t)q * kMxScaleBytes);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o.w[j] = *reinterpret_cast<const u32x4*>(wc + (int64_t)min(4 * q + j, kt_n - 1) * kMxTileBytes);
  };
  const uint8_t* xc[MT];
  const uint8_t* xs[MT];
  auto load_x = [&](int u, XQuad& o) {
    if (u >= u_n) return;
    const int q = slice + u * KS;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      o.s[i] = *reinterpret_cast<const u32x4*>(xs[i] + q * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < kWords; ++h)
          o.x[i][j][h] = *reinterpret_cast<const u32x4*>(xc[i] + (int64_t)min(4 * q + j, kt_n - 1) * Act<FMT>::kTileBytes + 64 * h);
    }
  };
  WQuad w[kAhead];
  XQuad x[2];
  // the pair ids first, then the first weights, then (the ids have arrived) the rows
  int64_t xr[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    xr[i] = row0 + min(16 * i + c, rows - 1);  // rows past the last repeat it and are not stored
    if constexpr (GROUPED) {
      if (a.pairs) xr[i] = a.pairs[xr[i]];
    }
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load_w(u, w[u]);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    int64_t r = xr[i];
    if constexpr (GROUPED) r = act_row(a, (int)r);
    xc[i] = a.codes + r * a.ldq + 16 * g;
    xs[i] = a.scales + r * a.lds;
  }
  load_x(0, x[0]);
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int u0 = 0; u0 < u_n; u0 += kAhead) {
#pragma unroll
    for (int v = 0; v < kAhead; ++v) {
      const int u = u0 + v;
      if (u >= u_n) break;
      load_x(u + 1, x[(v + 1) & 1]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (4 * (slice + u * KS) + j >= kt_n) break;
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[i] = mma<FMT>(j, w[v].w[j], w[v].s, split<FMT>(x[v & 1].x[i][j]), x[v & 1].s[i][j] >> (8 * g), acc[i]);
      }
      load_w(u + kAhead, w[v]);
    }
  }
  if constexpr (KS > 1) {
#pragma unroll
    for (int i = 0; i < MT; ++i) part[(slice * MT + i) * 64 + lane] = acc[i];
    __syncthreads();
    // wave s adds up and stores the pieces s, s + KS, ...
    for (int i = slice; i < MT; i += KS) {
      f32x4 s = part[i * 64 + lane];
#pragma unroll
      for (int w = 1; w < KS; ++w) {
        const f32x4 v = part[(w * MT + i) * 64 + lane];
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] = s[k] + v[k];
      }
      if (16 * i + c < rows) store_y4(a, row0 + 16 * i + c, rt * 16 + 4 * g, s);
    }
  } else {
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (16 * i + c < rows) store_y4(a, row0 + 16 * i + c, rt * 16 + 4 * g, acc[i]);
  }
}

template <int FMT, int MT, int KS, bool GROUPED>
static int launch_rows_ks(const MxArgs& a, hipStream_t s) {
  const int64_t groups = mx_row_tiles(a.n) * (GROUPED ? a.m : (a.m + 16 * MT - 1) / (16 * MT));
  if (int e = check_grid(groups, 64 * KS)) return e;
  hipLaunchKernelGGL((mx_rows_kernel<FMT, MT, KS, GROUPED>), dim3((unsigned)groups), dim3(64 * KS), 0, s, a);
  return check_launch("mx_rows_kernel");
}

// Waves over k: as many as bring the device to 2,048 waves (eight a CU), and no more than
// there are quads.  Depends on n and k alone for one matrix (MT = 1: every row of a call of up
// to 16 is computed as a single row is).
template <int FMT, int MT, bool GROUPED>
static int launch_rows(const MxArgs& a, hipStream_t s) {
  const int64_t waves = mx_row_tiles(a.n) * (GROUPED ? (a.m < a.n_expert ? a.m : a.n_expert) : 1);
  const int kq_n = mx_k_quads(a.k);
  int ks = 1;
  while (ks < 8 && ks < kq_n && waves * ks < 2048) ks *= 2;
  switch (ks) {
    case 1: return launch_rows_ks<FMT, MT, 1, GROUPED>(a, s);
    case 2: return launch_rows_ks<FMT, MT, 2, GROUPED>(a, s);
    case 4: return launch_rows_ks<FMT, MT, 4, GROUPED>(a, s);
    default: return launch_rows_ks<FMT, MT, 8, GROUPED>(a, s);
  }
}

// ---- many rows ------------------------------------------------------------------------------
// 32 x 32 x 64 instructions (lane l = 32 h + r: row r, E2M1 elements 32h .. 32h+31 or E4M3
// elements 16h .. 16h+15 and 32+16h .. 32+16h+15, scale of block h; it receives
// D[8 (i / 4) + 4 h + i % 4][r]).  WN x WM waves, each FN x FM pieces of 32 x 32.
//
// A step is 128 elements of k.  Its operands are copied from memory straight into LDS by
// global_load_lds, S stages deep: packed weight tiles as they are; rows of X with their
// 16-byte chunks exchanged inside a row (chunk q of row r at place q ^ f(r)) so that the 16
// lanes of a read phase fall on different banks.  The scales of four steps (a quad) come the
// same way into one buffer, which is free again when the quad's second step begins (they are
// then in registers).  The copies are written as inline assembly so that the
// compiler, which cannot tell the stages apart, does not wait for all of them before each
// LDS read; the counts of copies in flight are worked out below.
//
// What bounds it: the matrix pipe and what interrupts it.  13056 x 14336 x 4096 in MXFP4
// takes 399-434 us by the card (3.8 PFLOP/s; the same instructions alone reach 7.7): 60 % of the
// clocks have a matrix instruction running.  A workgroup of 256 x 128 spends 1.9 us before its
// first copies are issued, 27 in the loop and 3 storing, and the CU's other workgroup fills only a
// part of that.  Without the copies the loop takes 20 us, without the matrix instructions 17.
// MXFP8 loops also have the split (5 operations a word): its clocks add to the matrix
// instructions', even between them (333 x 5000 x 2592: 976 clocks a step, 670 without).
//
// Order in step t (two halves of 64 elements):
//   read the operands of half 1;  multiply half 0;
//   wait: half 1's reads done, stage t+1 landed;  barrier: so for every wave;
//   copy stage t+S (into stage t, which no wave reads any more);
//   read the operands of half 0 of step t+1;  multiply half 1.
// A wave's LDS reads so run under its own matrix instructions.

template <int N>
__device__ __forceinline__ void wait_copies() {  // at most N copies still in flight, and no LDS read
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (0 << 8));
}
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)p;
}
// Lane l's 16 bytes at base + voff to LDS address lds + 16 l.  M0 carries the LDS address; one
// wait state lies between its write and the copy.
__device__ __forceinline__ void copy16(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(voff), "s"(base), "{m0}"(lds) : "memory");
}
// The same from an address of the lane's own.
__device__ __forceinline__ void copy16(const uint8_t* at, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(at), "{m0}"(lds) : "memory");
}

// A pointer that is the same in all lanes, in scalar registers.
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const uint8_t*>((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)v) |
                                          (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32);
}

// Workgroup b of a grid of >= 8 ceil(G / 8) to tile 0 .. G - 1 (or -1): hardware deals
// workgroups round-robin to the eight XCDs, so each XCD gets a run of neighbouring tiles,
// which share operands in its own L2.
__device__ __forceinline__ int xcd_tile(uint32_t b, uint32_t G) {
  const uint32_t per = (G + 7) / 8, i = b / 8;
  if (i >= per) return -1;
  const uint32_t L = (b % 8) * per + i;
  return L < G ? (int)L : -1;
}

// Which tile of bn x bm outputs this workgroup makes: its place along n, its first row, its
// rows, its matrix.  False: none.  (All counts fit 32 bits: a grid has fewer workgroups.)
template <bool GROUPED>
__device__ __forceinline__ bool place_tile(const MxArgs& a, int bn, int bm, int& nt, int64_t& row0, int& rows,
                                           const uint8_t*& W) {
  const uint32_t nt_n = ((uint32_t)a.n + bn - 1) / bn;
  if constexpr (GROUPED) {
    ExpertTiles g = group_tiles(a, 0, bm);
    int total = g.total;
    for (int e0 = kGroupExperts; e0 < a.n_expert; e0 += kGroupExperts) total += group_tiles(a, e0, bm).total;
    const int L = xcd_tile(blockIdx.x, (uint32_t)total * nt_n);
    if (L < 0) return false;
    int e, t = (int)((uint32_t)L / nt_n), e0 = 0;
    nt = L - t * (int)nt_n;
    while (t >= g.total) {
      t -= g.total;
      e0 += kGroupExperts;
      if (e0 >= a.n_expert) return false;
      g = group_tiles(a, e0, bm);
    }
    group_find(g, e0, t, bm, e, row0, rows);
    W += e * a.w_stride;
  } else {
    const uint32_t mt_n = ((uint32_t)a.m + bm - 1) / bm;
    const int L = xcd_tile(blockIdx.x, mt_n * nt_n);
    if (L < 0) return false;
    // bands of eight row tiles, walked row tile first: the 32 CUs of an XCD hold about
    // 8 x 4 tiles and read 12 operand panels for them
    const uint32_t band = (uint32_t)L / (8 * nt_n), in = (uint32_t)L - band * 8 * nt_n;
    const uint32_t high = min(8u, mt_n - 8 * band);
    nt = (int)(high == 8 ? in / 8 : in / high);
    const uint32_t mt = 8 * band + in - (uint32_t)nt * high;
    row0 = (int64_t)mt * bm;
    rows = (int)min((int64_t)bm, a.m - row0);
  }
  return true;
}

static int64_t tile_grid(const MxArgs& a, int bn, int bm) {
  const int64_t nt = (a.n + bn - 1) / bn;
  int64_t tiles = (a.m + bm - 1) / bm;
  // by expert: each expert's last tile may be partial
  if (a.offsets) tiles = a.m / bm + a.n_expert < a.m ? a.m / bm + a.n_expert : a.m;
  return (nt * tiles + 7) / 8 * 8;
}

template <int FMT, int FN, int FM, int WN, int WM, int S>
struct Tile {
  static constexpr int kWaves = WN * WM;
  static constexpr int kBN = 32 * FN * WN, kBM = 32 * FM * WM;
  static constexpr int kRowB = Act<FMT>::kTileBytes;             // bytes of a row of X per step
  static constexpr int kChunks = kRowB / 16;                     // 16-byte chunks of them
  static constexpr int kWBytes = kBN * 64, kXBytes = kBM * kRowB;  // a stage
  static constexpr int kStage = kWBytes + kXBytes;
  static constexpr int kCW = kWBytes / 1024 / kWaves, kCX = kXBytes / 1024 / kWaves;  // copies a wave per step
  static constexpr int kC = kCW + kCX;
  static constexpr int kWS = kBN * 16, kXS = kBM * 16;           // scales of a quad
  static constexpr int kScales = kWS + kXS;
  static constexpr int kCWS = (kWS / 1024 + kWaves - 1) / kWaves, kCXS = (kXS / 1024 + kWaves - 1) / kWaves;
  static constexpr int kD = S - 1;                               // stages copied ahead
  static constexpr int kLds = S * kStage + kScales;
  static_assert(kWBytes % (1024 * kWaves) == 0 && kXBytes % (1024 * kWaves) == 0, "copies split evenly");
  static_assert(kWS % 1024 == 0 && kXS % 1024 == 0, "whole scale copies");
  static_assert(kD >= 1 && kD <= 3, "the counts below");
  static_assert(kLds <= 160 * 1024, "LDS");
  // Copies younger than stage t+1's when step t (place j in its quad) waits for it: those of
  // stages t+2 .. t+D, and the next quad's scales if they were issued since (before stage
  // u+D's copies, after the barrier that begins place u % 4 == 1).
  static constexpr int in_flight(int j) { return (kD - 1) * kC + (j >= 1 && j < kD ? kCWS + kCXS : 0); }
  // Copies that may still be in flight when step 0 begins.  The first stages are copied W of all
  // of them, then X of all of them (X's addresses are known later): younger than stage 0's X is
  // X of the others, but with three stages ahead step 0's own wait counts whole stages behind
  // stage 1, so stage 1's X has to be there by now.
  static constexpr int kFirst = kD == 3 ? kCX : (kD - 1) * kCX;

  // The counts, checked against the order in which a wave issues its copies: whatever step t
  // waits for must be older than the copies it lets fly.
  static constexpr bool counts_hold() {
    int op[512] = {}, n = 0;  // what each copy brings: a stage, or 1000 + a quad's scales
    int done = 0;             // copies before this one are known to have landed (they land in order)
    auto put = [&](int count, int what) {
      for (int i = 0; i < count; ++i) op[n++] = what;
    };
    auto landed = [&](int flying, int stage, int quad) {  // all stages and quads up to these
      if (n - flying > done) done = n - flying;
      for (int i = done; i < n; ++i)
        if (op[i] >= 1000 ? op[i] <= 1000 + quad : op[i] <= stage) return false;
      return true;
    };
    put(kCWS, 1000);
    for (int t = 0; t < kD; ++t) put(kCW, t);
    put(kCXS, 1000);
    for (int t = 0; t < kD; ++t) put(kCX, t);
    if (!landed(kFirst, 0, 0)) return false;
    put(kC, kD);
    for (int t = 0; t < 16; ++t) {
      if (!landed(in_flight(t % 4), t + 1, (t + 1) / 4)) return false;
      if (t % 4 == 0) put(kCWS + kCXS, 1000 + t / 4 + 1);
      put(kC, t + 1 + kD);
    }
    return true;
  }
};

// Lanes of a wave read what others of it wrote to LDS: the hardware keeps a wave's accesses in order,
// and this keeps the compiler from moving them past each other.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// `rows` x `cols` values of Y's type in LDS (rows of PITCH, at most 32 x COLS) to Y from (row0,
// col0) on, by one wave: eight columns a lane, past the L2 (nothing here reads Y again: the long
// prompt's 374 MB of results took 428 us with ordinary stores and 412 with these).  Rows that are no
// multiple of 16 bytes are stored element by element: 13056 x 14335 x 4096 to bf16 565 us with ldy = n, 409
// with ldy = 14336 (f32 776, 14336 x 4096 535).
template <typename E, int COLS, int PITCH>
__device__ __forceinline__ void store_rows_piece(const MxArgs& a, const E* part, int64_t row0, int rows, int64_t col0,
                                                 int cols) {
  constexpr int kLanes = COLS / 8, kStep = 64 / kLanes;  // lanes a row, rows a step
  const int lane = threadIdx.x & 63, c = 8 * (lane % kLanes), r0 = lane / kLanes;
  const E* from = part + r0 * PITCH + c;
  E* to = static_cast<E*>(a.y) + (row0 + r0) * a.ldy + col0 + c;
  if (a.vec_y && cols == COLS) {
#pragma unroll
    for (int r = 0; r < 32; r += kStep) {
      u32x4 v[sizeof(E) / 2];
#pragma unroll
      for (int i = 0; i < (int)sizeof(E) / 2; ++i) v[i] = reinterpret_cast<const u32x4*>(from + r * PITCH)[i];
      if (r0 + r < rows) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(E) / 2; ++i) __builtin_nontemporal_store(v[i], reinterpret_cast<u32x4*>(to + r * a.ldy) + i);
      }
    }
    return;
  }
#pragma unroll 1
  for (int r = 0; r0 + r < rows; r += kStep)
#pragma unroll 1
    for (int i = 0; i < 8 && c + i < cols; ++i) to[r * a.ldy + i] = from[r * PITCH + i];
}

// A wave's pieces to Y through LDS (`part`, its own, in Y's type), 32 rows at a time, so that the
// rows are written in runs of 64 FN or 128 FN bytes (a lane holds four columns of 32 different
// rows; stored from the registers, 32 bytes a row and store, the long prompt took 450 us for 432).
// `first`: the wave's first row in the tile, `col0` its first column.
template <int TYPE, int FN, int FM>
__device__ __forceinline__ void store_tile(const MxArgs& a, uint8_t* lds, const f32x16 (&acc)[FN][FM], int64_t row0, int first,
                                           int rows, int64_t col0) {
  using E = std::conditional_t<TYPE == kF32, float, uint16_t>;
  constexpr int kCols = 32 * FN, kPitch = kCols + 16 / (int)sizeof(E);
  E* part = reinterpret_cast<E*>(lds);
  const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
  const int cols = (int)min((int64_t)kCols, a.n - col0);
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    if (first + 32 * m >= rows || cols <= 0) break;
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v[4] = {acc[n][m][4 * q], acc[n][m][4 * q + 1], acc[n][m][4 * q + 2], acc[n][m][4 * q + 3]};
        E* to = part + r * kPitch + 32 * n + 8 * q + 4 * h;
        if constexpr (TYPE == kF32) *reinterpret_cast<f32x4*>(to) = f32x4{v[0], v[1], v[2], v[3]};
        else *reinterpret_cast<u32x2*>(to) = u32x2{pack2<TYPE>(v[0], v[1]), pack2<TYPE>(v[2], v[3])};
      }
    wave_fence();
    store_rows_piece<E, kCols, kPitch>(a, part, row0 + first + 32 * m, min(32, rows - first - 32 * m), col0, cols);
    wave_fence();
  }
}

// FAR: the rows a tile reads may lie 4 GiB apart or more; each lane then holds their addresses, and not
// 32-bit offsets from one base.
// waves a SIMD: registers are given out so that as many workgroups share a CU as LDS allows (two at most)
template <int FMT, int FN, int FM, int WN, int WM, int S, bool GROUPED, bool FAR>
__global__ void __launch_bounds__(64 * WN * WM)
__attribute__((amdgpu_waves_per_eu(Tile<FMT, FN, FM, WN, WM, S>::kWaves / 4 * (Tile<FMT, FN, FM, WN, WM, S>::kLds <= 80 * 1024 ? 2 : 1))))
mx_tile_kernel(MxArgs a) {
  using T = Tile<FMT, FN, FM, WN, WM, S>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::kLds];
  const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave % WN, wm = wave / WN;

  int nt, rows;
  int64_t row0;
  const uint8_t* W = a.W;
  if (!place_tile<GROUPED>(a, T::kBN, T::kBM, nt, row0, rows, W)) return;
  const int kt_n = mx_k_tiles(a.k), kq_n = mx_k_quads(a.k);
  const int rt_n = (int)mx_row_tiles(a.n), rt0 = nt * (T::kBN / 16);
  const uint32_t lds0 = lds_offset(lds);

  // ---- what this lane copies ------------------------------------------------------------
  // W: tiles wave * kCW ..; those past n repeat the last one (read in bounds, not stored)
  const uint8_t* wt[T::kCW];
#pragma unroll
  for (int i = 0; i < T::kCW; ++i) wt[i] = scalar(W + (int64_t)min(rt0 + wave * T::kCW + i, rt_n - 1) * (kt_n * (int64_t)kMxTileBytes));
  // X: kilobytes wave * kCX ..; rows past the last repeat it.  (By expert: the pair ids are
  // loaded here, and used after W's first copies have been issued.)  Without pair ids a tile's
  // rows lie one after another and are counted from its first.
  std::conditional_t<FAR, const uint8_t*, uint32_t> xo[T::kCX], xso[T::kCXS];
  uint32_t xr[T::kCX], xsr[T::kCXS];
  int xsl[T::kCXS];
  auto row_of = [&](int row) -> uint32_t {
    const uint32_t src = min(row, rows - 1);
    if constexpr (GROUPED) return a.pairs ? (uint32_t)a.pairs[row0 + src] : src;
    return src;
  };
#pragma unroll
  for (int i = 0; i < T::kCX; ++i) xr[i] = row_of(((wave * T::kCX + i) * 64 + lane) / T::kChunks);
#pragma unroll
  for (int i = 0; i < T::kCXS; ++i) {
    const int kb = (wave * T::kCXS + i) % (T::kXS / 1024);
    xsl[i] = T::kWS + kb * 1024;
    xsr[i] = row_of(kb * 64 + lane);
  }
  __builtin_amdgcn_sched_barrier(0);
  // scales: every wave issues the same number of copies, some of them twice (the same bytes
  // to the same place)
  uint32_t wso[T::kCWS];
  int wsl[T::kCWS];
#pragma unroll
  for (int i = 0; i < T::kCWS; ++i) {
    const int kb = (wave * T::kCWS + i) % (T::kWS / 1024);
    wsl[i] = kb * 1024;
    // four row tiles a kilobyte, relative to the workgroup's first
    const int rt = min(rt0 + 4 * kb + (lane >> 4), rt_n - 1) - rt0;
    wso[i] = (uint32_t)(rt * kq_n) * kMxScaleBytes + 16 * (lane & 15);
  }
  const int64_t xfirst = GROUPED && a.pairs ? 0 : row0;
  const uint8_t* xbase = scalar(a.codes + xfirst * a.ldq);
  const uint8_t* xsbase = scalar(a.scales + xfirst * a.lds);
  const uint8_t* wsbase = scalar(W + mx_code_plane(a.n, a.k) + (int64_t)rt0 * (kq_n * kMxScaleBytes));

  // from where `at` says, `ahead` bytes along the row
  auto copy_x = [&](const uint8_t* base, int64_t ahead, auto at, uint32_t to) {
    if constexpr (FAR) copy16(at + ahead, to);
    else copy16(base + ahead, at, to);
  };
  // (steps and quads past the last copy it again: the counts hold to the end)
  auto copy_part = [&](int t, int i0, int i1) {  // copies i0 .. i1 - 1 of this wave's kC
    const uint32_t st = lds0 + (uint32_t)(t % S) * T::kStage;
    const int k = min(t, kt_n - 1);
#pragma unroll
    for (int i = 0; i < T::kC; ++i) {
      if (i < i0 || i >= i1) continue;
      if (i < T::kCW) copy16(wt[i] + (int64_t)k * kMxTileBytes, 16 * lane, st + (wave * T::kCW + i) * 1024);
      else copy_x(xbase, (int64_t)k * T::kRowB, xo[i - T::kCW], st + T::kWBytes + (wave * T::kCX + i - T::kCW) * 1024);
    }
  };
  auto copy_wscales = [&](int q) {
#pragma unroll
    for (int i = 0; i < T::kCWS; ++i) copy16(wsbase + (int64_t)min(q, kq_n - 1) * kMxScaleBytes, wso[i], lds0 + S * T::kStage + wsl[i]);
  };
  auto copy_xscales = [&](int q) {
#pragma unroll
    for (int i = 0; i < T::kCXS; ++i) copy_x(xsbase, (int64_t)min(q, kq_n - 1) * 16, xso[i], lds0 + S * T::kStage + xsl[i]);
  };

  // ---- operands from LDS --------------------------------------------------------------------
  struct Ops {
    u32x4 w[FN], x[FM][Act<FMT>::kWords / 4];
  };
  // where this lane reads: weights 32 (FN wn + i) + r, rows 32 (FM wm + i) + r
  const int wrow = 32 * FN * wn + r, xrow = 32 * FM * wm + r;
  auto read_half = [&](int t, int s, Ops& o) {
    const uint8_t* st = lds + (t % S) * T::kStage;
#pragma unroll
    for (int i = 0; i < FN; ++i)
      o.w[i] = *reinterpret_cast<const u32x4*>(st + (wrow / 16 + 2 * i) * 1024 + (16 * (2 * s + h) + (r & 15)) * 16);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int c = 0; c < Act<FMT>::kWords / 4; ++c) {
        const int chunk = FMT == kRowsMxfp4 ? 2 * s + h : 4 * s + 2 * c + h;
        const int place = chunk ^ (FMT == kRowsMxfp4 ? (r >> 2) & 3 : (r >> 1) & 7);
        o.x[i][c] = *reinterpret_cast<const u32x4*>(st + T::kWBytes + (xrow + 32 * i) * T::kRowB + place * 16);
      }
  };
  struct Scales {
    uint32_t w[FN][2];
    u32x4 x[FM];  // of step j in word j, this lane's blocks h and 2 + h in bytes 0 and 2
  };
  auto read_scales = [&](Scales& o) {
    const uint8_t* st = lds + S * T::kStage;
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        o.w[i][s] = *reinterpret_cast<const uint32_t*>(st + (wrow / 16 + 2 * i) * 256 + (16 * (2 * s + h) + (r & 15)) * 4);
#pragma unroll
    for (int i = 0; i < FM; ++i) o.x[i] = *reinterpret_cast<const u32x4*>(st + T::kWS + (xrow + 32 * i) * 16) >> (8 * h);
  };

  f32x16 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
  // one half step; `before(m)` runs before the products of row piece m
  auto multiply = [&](auto jj, auto ss, const Ops& o, const Scales& sc, auto before) {
    constexpr int j = decltype(jj)::value, s = decltype(ss)::value;
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      before(m);
      const Frag<FMT> x = split<FMT>(o.x[m]);
#pragma unroll
      for (int n = 0; n < FN; ++n) acc[n][m] = mma32<FMT, j, s>(o.w[n], sc.w[n][s], x, sc.x[m][j], acc[n][m]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // the operands are in registers here: keeps the reads where they are issued
  auto arrived = [&](Ops& o) {
#pragma unroll
    for (int i = 0; i < FN; ++i) asm volatile("" : "+v"(o.w[i]));
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int c = 0; c < Act<FMT>::kWords / 4; ++c) asm volatile("" : "+v"(o.x[i][c]));
  };

  // ---- main loop ------------------------------------------------------------------------------
  copy_wscales(0);
#pragma unroll
  for (int t = 0; t < T::kD; ++t) copy_part(t, 0, T::kCW);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < T::kCX; ++i) {
    const int at = (wave * T::kCX + i) * 64 + lane, row = at / T::kChunks, place = at % T::kChunks;
    const int chunk = place ^ (FMT == kRowsMxfp4 ? (row >> 2) & 3 : (row >> 1) & 7);
    if constexpr (GROUPED) xr[i] = act_row(a, (int)xr[i]);
    if constexpr (FAR) xo[i] = xbase + (int64_t)xr[i] * a.ldq + 16 * chunk;
    else xo[i] = xr[i] * (uint32_t)a.ldq + 16 * chunk;
  }
#pragma unroll
  for (int i = 0; i < T::kCXS; ++i) {
    if constexpr (GROUPED) xsr[i] = act_row(a, (int)xsr[i]);
    if constexpr (FAR) xso[i] = xsbase + (int64_t)xsr[i] * a.lds;
    else xso[i] = xsr[i] * (uint32_t)a.lds;
  }
  copy_xscales(0);
#pragma unroll
  for (int t = 0; t < T::kD; ++t) copy_part(t, T::kCW, T::kC);
  static_assert(T::counts_hold(), "the copies in flight");
  wait_copies<T::kFirst>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  copy_part(T::kD, 0, T::kC);
  Ops o0, o1;
  // Large MXFP8 pieces: a half is read right before it is multiplied.  Their products take four
  // times as long as their reads, the CU's other workgroup fills the gap, and the registers
  // for a half ahead are not there.
  constexpr bool kAhead = FMT == kRowsMxfp4 || FN * FM <= 2;
  Scales sc;
  read_scales(sc);
  if constexpr (kAhead) read_half(0, 0, o0);
  auto step = [&](auto jj, int t) {
    constexpr int j = decltype(jj)::value;
    if constexpr (kAhead) {
      read_half(t, 1, o1);
      __builtin_amdgcn_sched_barrier(0);
    } else {
      read_half(t, 0, o0);
    }
    multiply(jj, std::integral_constant<int, 0>{}, o0, sc, [](int) {});
    if constexpr (!kAhead) read_half(t, 1, o0);
    asm volatile("" ::: "memory");
    wait_copies<T::in_flight(j)>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if constexpr (kAhead) {
      read_half(t + 1, 0, o0);
      __builtin_amdgcn_sched_barrier(0);
    }
    multiply(jj, std::integral_constant<int, 1>{}, kAhead ? o1 : o0, sc, [&](int m) {
      if (j == 0 && m == 0) {  // every wave has read this quad's
        copy_wscales(t / 4 + 1);
        copy_xscales(t / 4 + 1);
      }
      copy_part(t + 1 + T::kD, m * T::kC / FM, (m + 1) * T::kC / FM);
    });
    if constexpr (kAhead) arrived(o0);
    if constexpr (j == 3) read_scales(sc);  // the next quad's, for the next step
  };
  for (int t = 0;; t += 4) {
    step(std::integral_constant<int, 0>{}, t);
    if (t + 1 >= kt_n) break;
    step(std::integral_constant<int, 1>{}, t + 1);
    if (t + 2 >= kt_n) break;
    step(std::integral_constant<int, 2>{}, t + 2);
    if (t + 3 >= kt_n) break;
    step(std::integral_constant<int, 3>{}, t + 3);
    if (t + 4 >= kt_n) break;
  }
  // ---- store ------------------------------------------------------------------------------------
  wait_copies<0>();
  __builtin_amdgcn_s_barrier();  // no copy lands in LDS any more, and no wave reads the stages
  asm volatile("" ::: "memory");
  constexpr int kPart = 32 * (32 * FN + 4);
  static_assert(T::kWaves * kPart * 4 <= T::kLds, "the parts fit");
  uint8_t* part = lds + wave * kPart * 4;
  const int first = 32 * FM * wm;
  const int64_t col0 = (int64_t)nt * T::kBN + 32 * FN * wn;
  if (a.y_type == kF32) store_tile<kF32, FN, FM>(a, part, acc, row0, first, rows, col0);
  else if (a.y_type == kF16) store_tile<kF16, FN, FM>(a, part, acc, row0, first, rows, col0);
  else store_tile<kBF16, FN, FM>(a, part, acc, row0, first, rows, col0);
}

template <int FMT, int FN, int FM, int WN, int WM, int S, bool GROUPED, bool FAR = false>
static int launch_tiles(const MxArgs& a, hipStream_t s) {
  using T = Tile<FMT, FN, FM, WN, WM, S>;
  const int64_t groups = tile_grid(a, T::kBN, T::kBM);
  if (int e = check_grid(groups, 64 * T::kWaves)) return e;
  hipLaunchKernelGGL((mx_tile_kernel<FMT, FN, FM, WN, WM, S, GROUPED, FAR>), dim3((unsigned)groups), dim3(64 * T::kWaves), 0, s, a);
  return check_launch("mx_tile_kernel");
}

// Which kernel, by the workgroups each tile gives (times in us on an MI355X, MXFP4 unless
// MXFP8 is named).  The larger tile reads less per product; below some 160-220 workgroups of it
// the 256 CUs are not filled and the next smaller one is faster:
//   256 x 128 from 224: 14336 x 4096, m = 512 (224): 21.2, 128 x 128 22.6; 5000 x 2592,
//     m = 1024 (160): 19.6 for 17.2.  MXFP8, 128 x 64 on the other side: m = 512 47.0 for 55.2; 5000 x 2592
//     36.4 for 28.5.
//   128 x 128 from 160, MXFP4 only: 4096 x 4096, m = 1024 (256): 14.4, 128 x 64 16.1; m = 512
//     (128): 12.6 for 10.3.  MXFP8: 33.3 for 29.2; 29.4 for 18.1.
//   128 x 64 from 160, else 64 x 64: 4096 x 4096, m = 333 (192): 9.7 for 11.2; m = 256 (128): 9.6 for 8.9.
//     MXFP8: 17.9 for 19.7; 16.7 for 14.0.
//   Up to 32 rows straight from memory unless 64 x 64 fills the CUs: 4096 x 4096, m = 32
//     (64): 5.1 for 6.1; 14336 x 4096 (224): 14.4 for 8.9.  MXFP8: 7.6 for 12.1; 22.9 for 13.2 (near the border,
//     10000 x 2592, m = 24 (157): MXFP4 6.5 for 6.9, MXFP8 13.6 for 10.1).
template <int FMT>
static int launch_dense(const MxArgs& a, hipStream_t s) {
  constexpr bool k4 = FMT == kRowsMxfp4;
  auto count = [&](int bn, int bm) { return ((a.n + bn - 1) / bn) * ((a.m + bm - 1) / bm); };
  if (a.m <= 16) return launch_rows<FMT, 1, false>(a, s);
  // the tile kernel's row offsets have 32 bits
  if (256 * (a.ldq > a.lds ? a.ldq : a.lds) >= ((int64_t)1 << 32)) return launch_rows<FMT, 2, false>(a, s);
  if (a.m <= 32 && count(64, 64) < 160) return launch_rows<FMT, 2, false>(a, s);
  if (count(256, 128) >= 224) return launch_tiles<FMT, 4, 2, 2, 2, k4 ? 3 : 2, false>(a, s);
  if constexpr (k4)
    if (count(128, 128) >= 160) return launch_tiles<FMT, 2, 2, 2, 2, 4, false>(a, s);
  if (count(128, 64) >= 160) return launch_tiles<FMT, 2, 1, 2, 2, 4, false>(a, s);
  return launch_tiles<FMT, 1, 1, 2, 2, 4, false>(a, s);
}

// By expert: how the rows fall is not known here, only their average r.  Straight from memory
// up to r = 2: 128 experts of 1536 x 2048, r = 1 16.9 us, 128 x 64 tiles 18.4; r = 2 28.5 for 26.6; r = 4 40.9
// for 34.1; 64 experts of 512 x 1024, r = 2 5.0 for 5.4, r = 4 6.6 for 6.4.  MXFP8: 22.0 for 24.2, 37.5 for
// 33.2, 54.4 for 42.2; 7.4 for 7.3, 8.9 for 8.2.
// 256 x 128 tiles from r = 32 (MXFP8 64) if there are enough of them.  128 experts of 1536 x 2048, r = 16 49.5, 128 x
// 64 tiles 47.1; r = 32 53.2 for 53.4; r = 64 57.4 for 61.2; 16 experts, r = 128, some 144 tiles 12.9 for 11.9.  MXFP8:
// 79.8 for 59.8, 82.0 for 64.7, 90.0 for 84.6, r = 128 113 for 121; with 128 experts of 2048 x 768 r = 32 45.9
// for 44.9, r = 64 51.2 for 56.9; 16 experts 26.4 for 17.4.
template <int FMT>
static int launch_grouped(const MxArgs& a, hipStream_t s) {
  constexpr bool k4 = FMT == kRowsMxfp4;
  const int64_t experts = a.m < a.n_expert ? a.m : a.n_expert;
  if (a.m <= 2 * a.n_expert) return launch_rows<FMT, 1, true>(a, s);
  // with pair ids a tile's rows may lie anywhere in X, without them they are neighbours.  (8 experts of
  // 4096 x 14336, MXFP8, 310,000 gathered rows in 4.4 GB: 20.9 ms, 1.74 PFLOP/s; 290,000 in 4.2 GB, by
  // offsets: 19.9 ms, 1.71.)
  const int64_t apart = (a.pairs ? a.n_rows : 128) * (a.ldq > a.lds ? a.ldq : a.lds);
  const bool far = apart >= ((int64_t)1 << 32);
  if (a.m >= (k4 ? 32 : 64) * (int64_t)a.n_expert && ((a.n + 255) / 256) * (a.m / 128 + experts / 2) >= 192)
    return far ? launch_tiles<FMT, 4, 2, 2, 2, k4 ? 3 : 2, true, true>(a, s)
               : launch_tiles<FMT, 4, 2, 2, 2, k4 ? 3 : 2, true>(a, s);
  return far ? launch_tiles<FMT, 2, 1, 2, 2, 4, true, true>(a, s) : launch_tiles<FMT, 2, 1, 2, 2, 4, true>(a, s);
}

int launch_mx_gemm(MxArgs a, int fmt, hipStream_t s) {
  a.inv_top = a.pairs ? 1.0f / (float)a.top_k : 0.0f;
  a.vec_y = a.ldy % (a.y_type == kF32 ? 4 : 8) == 0 && aligned(a.y, 16);
  if (a.offsets) return fmt == kRowsMxfp4 ? launch_grouped<kRowsMxfp4>(a, s) : launch_grouped<kRowsMxfp8>(a, s);
  return fmt == kRowsMxfp4 ? launch_dense<kRowsMxfp4>(a, s) : launch_dense<kRowsMxfp8>(a, s);
}

}  // namespace iq4
