// g4.hip -- products of few rows with 4-bit weights that have a scale and a zero point per
// group of 32, 64 or 128 weights: Y[i][r] = sum over groups G of row r of
//   s[r][G] * sum_{k in G} (q[r][k] - z[r][G]) X[i][k],
// for one matrix or for one matrix per expert with the rows sorted by expert.
#include "g4.hpp"
#include "pieces.hpp"

namespace iq4 {

// ---- pack -------------------------------------------------------------------------------
// A lane makes the 16 bytes of one row's 32 codes: word b of lane 16 g + c of code tile
// (rt, kt) has elements 8g .. 8g+7 of block 4 kt + b of row 16 rt + c, elements 0, 2, 4, 6 in the
// low half's nibbles and 1, 3, 5, 7 in the high half's.  Scales and zero points keep their order
// inside a (row tile, quad).  What lies past n or k is zero.  Run once per matrix; the source
// is read byte by byte, which spares it any alignment.
__global__ void __launch_bounds__(256) g4_pack_kernel(G4Pack a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int lane = (int)(i & 63), g = lane >> 4, c = lane & 15;
  const int64_t quad = i >> 6;
  const int kt_n = g4_k_tiles(a.k), kq_n = g4_k_quads(a.k);
  const int64_t rt = quad / kq_n;
  if (rt >= g4_row_tiles(a.n)) return;
  const int kq = (int)(quad - rt * kq_n);
  const int64_t row = rt * 16 + c;
  for (int j = 0; j < 4; ++j) {
    const int kt = 4 * kq + j;
    if (kt >= kt_n) break;
    uint32_t w[4];
    for (int b = 0; b < 4; ++b) {
      const int64_t at = (int64_t)kt * 128 + 32 * b + 8 * g;  // the first of eight elements
      uint32_t v = 0;
      if (row < a.n && at < a.k)
        for (int e = 0; e < 4; ++e) {
          const uint32_t two = a.codes[row * a.ldq + at / 2 + e];
          v |= (two & 15u) << (4 * e) | (two >> 4) << (16 + 4 * e);
        }
      w[b] = v;
    }
    *reinterpret_cast<u32x4*>(a.packed + (rt * kt_n + kt) * kG4TileBytes + lane * 16) = u32x4{w[0], w[1], w[2], w[3]};
  }
  const int per = 512 / a.group;  // groups of a row in a quad
  uint16_t* s = reinterpret_cast<uint16_t*>(a.packed + g4_code_plane(a.n, a.k) + quad * g4_scale_bytes(a.group));
  uint8_t* z = a.packed + g4_code_plane(a.n, a.k) + g4_scale_plane(a.n, a.k, a.group) + quad * g4_zero_bytes(a.group);
  const int64_t groups = (a.k + a.group - 1) / a.group;
  for (int e = lane; e < 16 * per; e += 64) {
    const int64_t r = rt * 16 + e / per, q = (int64_t)kq * per + e % per;
    const bool in = r < a.n && q < groups;
    const uint8_t* at = reinterpret_cast<const uint8_t*>(a.scales) + 2 * (r * a.lds + q);
    s[e] = in ? (uint16_t)(at[0] | at[1] << 8) : (uint16_t)0;
    if (a.zeros) z[e] = in ? a.zeros[r * a.ldz + q] & 15 : 0;
  }
}

int launch_g4_pack(const G4Pack& a, hipStream_t s) {
  const int64_t waves = g4_row_tiles(a.n) * g4_k_quads(a.k);
  hipLaunchKernelGGL(g4_pack_kernel, dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, s, a);
  return check_launch("g4_pack_kernel");
}

// ---- product ------------------------------------------------------------------------------

template <int TYPE>
__device__ __forceinline__ float element(const void* p, int64_t at) {
  if constexpr (TYPE == kF32) return static_cast<const float*>(p)[at];
  const uint16_t h = static_cast<const uint16_t*>(p)[at];
  if constexpr (TYPE == kF16) return h2f(h);
  return __uint_as_float((uint32_t)h << 16);
}

// One lane per output.
template <int TX>
__global__ void __launch_bounds__(256) g4_simple_kernel(G4Args a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / a.n;
  const int64_t r = i - row * a.n;
  if (row >= a.m) return;
  const uint8_t* W = a.W;
  int64_t xr = row;
  if (a.offsets) {
    int e = 0;
    while (e < a.n_expert && !(a.offsets[e] <= row && row < a.offsets[e + 1])) ++e;
    if (e == a.n_expert) return;
    W += e * a.w_stride;
    if (a.pairs) xr = a.pairs[row] / a.top_k;
    xr = min(max(xr, (int64_t)0), a.n_rows - 1);
  }
  const int64_t rt = r >> 4;
  const int c = (int)(r & 15), per = 512 / a.group;
  const uint8_t* codes = W + rt * g4_k_tiles(a.k) * kG4TileBytes;
  const uint16_t* ss = reinterpret_cast<const uint16_t*>(W + g4_code_plane(a.n, a.k));
  const uint8_t* zs = W + g4_code_plane(a.n, a.k) + g4_scale_plane(a.n, a.k, a.group);
  const char* x = static_cast<const char*>(a.x) + xr * a.ldx * (TX == kF32 ? 4 : 2);
  float acc = 0.f;
  for (int64_t k0 = 0; k0 < a.k; k0 += a.group) {
    const int64_t at = ((rt * g4_k_quads(a.k) + k0 / 512) * 16 + c) * per + k0 % 512 / a.group;
    const uint16_t sb = ss[at];
    const float s = a.scale_type == kF16 ? h2f(sb) : __uint_as_float((uint32_t)sb << 16);
    const int z = a.zeros ? zs[at] : 8;
    float d = 0.f;
    for (int64_t k = k0; k < min(k0 + a.group, a.k); ++k) {
      const int b = (int)(k >> 5 & 3), g = (int)(k >> 3 & 3), e = (int)(k & 7);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + (k >> 7) * kG4TileBytes + (16 * g + c) * 16 + 4 * b);
      const int q = (int)(w >> (16 * (e & 1) + 4 * (e >> 1)) & 15u);
      d = fmaf((float)(q - z), element<TX>(x, k), d);
    }
    acc = fmaf(s, d, acc);
  }
  if (a.y_type == kF32) static_cast<float*>(a.y)[row * a.ldy + r] = acc;
  else static_cast<uint16_t*>(a.y)[row * a.ldy + r] = (uint16_t)(a.y_type == kF16 ? pack2<kF16>(acc, 0.f) : pack2<kBF16>(acc, 0.f));
}

int launch_g4_qmv(const G4Args& a, int x_type, hipStream_t s) {
  const int64_t groups = (a.m * a.n + 255) / 256;
  if (groups * 256 >= (int64_t)1 << 32) return set_error(-3, "iq4_g4 product: too many workgroups (n * m too large)");
  const dim3 grid((unsigned)groups);
  if (x_type == kF32) hipLaunchKernelGGL(g4_simple_kernel<kF32>, grid, dim3(256), 0, s, a);
  else if (x_type == kF16) hipLaunchKernelGGL(g4_simple_kernel<kF16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(g4_simple_kernel<kBF16>, grid, dim3(256), 0, s, a);
  return check_launch("g4_simple_kernel");
}

}  // namespace iq4
