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
#include "common.hpp"
#include "mx.hpp"
#include "rows.hpp"

namespace iq4 {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---- pack -------------------------------------------------------------------------------
// Code tile (rt, kt) at (rt * KT + kt) * 1024: lane 16g + c has the 16 bytes of row 16 rt + c,
// block 4 kt + g.  Scale word of four tiles (rt, kq) after all codes, at (rt * KQ + kq) * 256:
// lane 16g + c, byte j has the scale of block 4 (4 kq + j) + g.  What lies past n or k is zero
// (a zero code times any scale below 255 adds nothing).
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

template <int FMT>
struct Act {  // one 16-row x 128-element operand of activations
  static constexpr int kWords = FMT == kRowsMxfp4 ? 4 : 8;
  static constexpr int kTileBytes = FMT == kRowsMxfp4 ? 64 : 128;  // of one row
};

template <int FMT>
__device__ __forceinline__ f32x4 mma(u32x4 w, uint32_t sw, int sel, const uint32_t (&x)[Act<FMT>::kWords], uint32_t sx,
                                     f32x4 acc) {
  const i32x8 a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  i32x8 b = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < Act<FMT>::kWords; ++i) b[i] = (int)x[i];
  constexpr int kB = FMT == kRowsMxfp4 ? 4 : 0;  // E2M1 or E4M3
  switch (sel) {  // the byte of the weights' scale word
    case 0: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, kB, 0, (int)sw, 0, (int)sx);
    case 1: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, kB, 1, (int)sw, 0, (int)sx);
    case 2: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, kB, 2, (int)sw, 0, (int)sx);
    default: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, kB, 3, (int)sw, 0, (int)sx);
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

// Tile `t` of the grouped rows in tiles of `bm`: its expert, first row and rows, found by
// every wave on its own from the offsets (64 experts a step: tiles per expert, a running
// sum over the lanes, the first lane past t).  Offsets are clamped to [0, m]: whatever they
// hold, no row outside is touched.  False: there are fewer tiles.
__device__ __forceinline__ bool find_tile(const MxArgs& a, int64_t t, int bm, int& e, int64_t& row0, int& rows) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int e0 = 0; e0 < a.n_expert; e0 += 64) {
    const int el = e0 + lane;
    int64_t o0 = 0, o1 = 0;
    if (el < a.n_expert) {
      o0 = min(max((int64_t)a.offsets[el], (int64_t)0), a.m);
      o1 = min(max((int64_t)a.offsets[el + 1], o0), a.m);
    }
    const int mine = (int)((o1 - o0 + bm - 1) / bm);
    int run = mine;
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(run, d);
      if (lane >= d) run += up;
    }
    const uint64_t past = __ballot(before + run > t);
    if (past) {
      const int src = __builtin_ctzll(past);
      const int64_t first = before + __shfl(run, src) - __shfl(mine, src);  // tiles before this expert
      const int64_t b0 = __shfl((int)o0, src), b1 = __shfl((int)o1, src);
      e = e0 + src;
      row0 = b0 + (t - first) * bm;
      rows = (int)min((int64_t)bm, b1 - row0);
      return true;
    }
    before += __shfl(run, 63);
  }
  return false;
}

// Activation row of output row i (grouped), inside the buffer whatever `pairs` holds.
__device__ __forceinline__ int64_t act_row(const MxArgs& a, int64_t i) {
  const int64_t r = a.pairs ? a.pairs[i] / a.top_k : i;
  return min(max(r, (int64_t)0), a.n_rows - 1);
}

// ---- few rows -----------------------------------------------------------------------------
// One workgroup: 16 weight rows, MT x 16 rows of Y, all of k.  Its waves take turns at the
// quads of four tiles along k (every operand straight from memory into registers) and their
// sums are added through LDS in the waves' order.
template <int FMT, int MT, int NW, bool GROUPED>
__global__ void __launch_bounds__(64 * NW) mx_rows_kernel(MxArgs a) {
  __shared__ f32x4 part[NW > 1 ? NW * MT * 64 : 1];
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t nt = mx_row_tiles(a.n);
  const int64_t rt = blockIdx.x % nt, mt = blockIdx.x / nt;
  const uint8_t* W = a.W;
  int64_t row0 = mt * (16 * MT);
  int rows = 16 * MT;
  if constexpr (GROUPED) {
    int e;
    if (!find_tile(a, mt, 16 * MT, e, row0, rows)) return;
    W += e * a.w_stride;
  } else {
    rows = (int)min((int64_t)rows, a.m - row0);
  }
  const int kt_n = mx_k_tiles(a.k), kq_n = mx_k_quads(a.k);
  const uint8_t* wc = W + rt * kt_n * kMxTileBytes + lane * 16;
  const uint8_t* wsc = W + mx_code_plane(a.n, a.k) + rt * kq_n * kMxScaleBytes + lane * 4;
  const uint8_t* xc[MT];
  const uint8_t* xs[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    int64_t r = row0 + min(16 * i + c, rows - 1);  // rows past the last repeat it and are not stored
    if constexpr (GROUPED) r = act_row(a, r);
    xc[i] = a.codes + r * a.ldq + 16 * g;
    xs[i] = a.scales + r * a.lds;
  }
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int kq = wave; kq < kq_n; kq += NW) {
    const uint32_t sw = *reinterpret_cast<const uint32_t*>(wsc + kq * kMxScaleBytes);
    u32x4 sx[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) sx[i] = *reinterpret_cast<const u32x4*>(xs[i] + kq * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int kt = 4 * kq + j;
      if (kt >= kt_n) break;
      const u32x4 w = *reinterpret_cast<const u32x4*>(wc + kt * kMxTileBytes);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint32_t x[Act<FMT>::kWords];
#pragma unroll
        for (int h = 0; h < Act<FMT>::kWords / 4; ++h) {
          const u32x4 t = *reinterpret_cast<const u32x4*>(xc[i] + (int64_t)kt * Act<FMT>::kTileBytes + 64 * h);
#pragma unroll
          for (int q = 0; q < 4; ++q) x[4 * h + q] = t[q];
        }
        acc[i] = mma<FMT>(w, sw, j, x, sx[i][j] >> (8 * g), acc[i]);
      }
    }
  }
  if constexpr (NW > 1) {
#pragma unroll
    for (int i = 0; i < MT; ++i) part[(wave * MT + i) * 64 + lane] = acc[i];
    __syncthreads();
    // wave w adds up and stores the pieces w, w + NW, ...
    for (int i = wave; i < MT; i += NW) {
      f32x4 s = part[i * 64 + lane];
      for (int w = 1; w < NW; ++w) {
        const f32x4 p = part[(w * MT + i) * 64 + lane];
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] = s[q] + p[q];
      }
      if (16 * i + c < rows) store_y4(a, row0 + 16 * i + c, rt * 16 + 4 * g, s);
    }
  } else {
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (16 * i + c < rows) store_y4(a, row0 + 16 * i + c, rt * 16 + 4 * g, acc[i]);
  }
}

template <int FMT, int MT, int NW>
static int launch_rows(const MxArgs& a, hipStream_t s) {
  const int64_t nt = mx_row_tiles(a.n);
  const bool grouped = a.offsets != nullptr;
  // grouped: every expert's last tile may be partial
  int64_t tiles = (a.m + 16 * MT - 1) / (16 * MT);
  if (grouped) tiles = a.m / (16 * MT) + a.n_expert < a.m ? a.m / (16 * MT) + a.n_expert : a.m;
  const dim3 grid((unsigned)(nt * tiles));
  if (grouped) hipLaunchKernelGGL((mx_rows_kernel<FMT, MT, NW, true>), grid, dim3(64 * NW), 0, s, a);
  else hipLaunchKernelGGL((mx_rows_kernel<FMT, MT, NW, false>), grid, dim3(64 * NW), 0, s, a);
  return check_launch("mx_rows_kernel");
}

int launch_mx_gemm(MxArgs a, int fmt, hipStream_t s) {
  a.vec_y = a.ldy % 4 == 0 && aligned(a.y, a.y_type == kF32 ? 16 : 8);
  if (fmt == kRowsMxfp4) return a.m <= 16 ? launch_rows<kRowsMxfp4, 1, 8>(a, s) : launch_rows<kRowsMxfp4, 4, 4>(a, s);
  return a.m <= 16 ? launch_rows<kRowsMxfp8, 1, 8>(a, s) : launch_rows<kRowsMxfp8, 4, 4>(a, s);
}

}  // namespace iq4
