// g4.hip -- 4-bit weights that have a scale and a zero point per group of 32, 64 or 128: the
// packed layout, and which kernel (g4_kernel.hpp) multiplies.
#include "g4.hpp"

namespace iq4 {

// ---- pack -------------------------------------------------------------------------------
// A wave makes a code tile: word b of lane 16 g + c has elements 8g .. 8g+7 of block b (of 32) of
// row 16 rt + c, elements 0, 2, 4, 6 in the low half's nibbles and 1, 3, 5, 7 in the high half's.
// Scales and zero points keep their order inside a tile's row.  What lies past n or k is zero.  Run
// once per matrix; the source is read byte by byte, which spares it any alignment and bounds it (14336 x
// 4096 25 us, 2.5 TB/s).
__global__ void __launch_bounds__(256) g4_pack_kernel(G4Pack a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int lane = (int)(i & 63), g = lane >> 4, c = lane & 15;
  const int64_t tile = i >> 6;
  const int kt_n = g4_k_tiles(a.k);
  const int64_t rt = tile / kt_n;
  if (rt >= g4_row_tiles(a.n)) return;
  const int kt = (int)(tile - rt * kt_n);
  const int64_t row = rt * 16 + c;
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
  *reinterpret_cast<u32x4*>(a.packed + tile * kG4TileBytes + lane * 16) = u32x4{w[0], w[1], w[2], w[3]};
  const int sets = 128 / a.group;  // groups of a row in a tile: lane 16 g + c does group g of row c
  if (g >= sets) return;
  uint16_t* s = reinterpret_cast<uint16_t*>(a.packed + g4_code_plane(a.n, a.k)) + tile * 16 * sets;
  uint8_t* z = a.packed + g4_code_plane(a.n, a.k) + g4_scale_plane(a.n, a.k, a.group) + tile * 16 * sets;
  const int64_t q = (int64_t)kt * sets + g;
  const bool in = row < a.n && q * a.group < a.k;
  const uint8_t* at = reinterpret_cast<const uint8_t*>(a.scales) + 2 * (row * a.lds + q);
  s[c * sets + g] = in ? (uint16_t)(at[0] | at[1] << 8) : (uint16_t)0;
  if (a.zeros) z[c * sets + g] = in ? a.zeros[row * a.ldz + q] & 15 : 0;
}

int launch_g4_pack(const G4Pack& a, hipStream_t s) {
  const int64_t waves = g4_row_tiles(a.n) * g4_k_tiles(a.k);
  hipLaunchKernelGGL(g4_pack_kernel, dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, s, a);
  return check_launch("g4_pack_kernel");
}

int launch_g4_qmv(const G4Args& a, hipStream_t s) {
  if (a.group == 32) return launch_g4_32(a, s);
  return a.group == 64 ? launch_g4_64(a, s) : launch_g4_128(a, s);
}

}  // namespace iq4
