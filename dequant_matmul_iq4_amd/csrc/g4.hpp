// g4.hpp -- 4-bit weights with group scales, w = s (q - z): the packed layout and the
// launchers' arguments (g4.hip).
#pragma once
#include "common.hpp"
#include "rows.hpp"

namespace iq4 {

// Packed layout: a row tile is 16 rows, a code tile a row tile x 128 along k (1 KB).  Codes first,
// then the scales by code tile, then the zero points by code tile.
constexpr int kG4TileBytes = 1024;
inline __host__ __device__ int64_t g4_row_tiles(int64_t n) { return (n + 15) / 16; }
inline __host__ __device__ int g4_k_tiles(int64_t k) { return (int)((k + 127) / 128); }
inline __host__ __device__ int64_t g4_code_plane(int64_t n, int64_t k) {
  return g4_row_tiles(n) * g4_k_tiles(k) * kG4TileBytes;
}
// a code tile has 16 rows x (128 / group) scales of two bytes, and as many zero points of one
inline __host__ __device__ int64_t g4_scale_plane(int64_t n, int64_t k, int group) {
  return g4_row_tiles(n) * g4_k_tiles(k) * 16 * (128 / group) * 2;
}
inline __host__ __device__ int64_t g4_packed_bytes(int64_t n, int64_t k, int group, bool zeros) {
  const int64_t b = g4_code_plane(n, k) + g4_scale_plane(n, k, group) + (zeros ? g4_scale_plane(n, k, group) / 2 : 0);
  return (b + 255) / 256 * 256;  // (a bank's next matrix begins aligned)
}

struct G4Pack {
  const uint8_t* codes;
  int64_t ldq;
  const uint16_t* scales;
  int64_t lds;
  const uint8_t* zeros;  // or null
  int64_t ldz;
  int64_t n, k;
  int group;
  uint8_t* packed;
};
int launch_g4_pack(const G4Pack& a, hipStream_t s);

struct G4Args {
  const uint8_t* W;
  int64_t w_stride;  // bytes of one expert's matrix
  int64_t n, k;
  int group;         // 32, 64 or 128
  int scale_type;    // kF16 or kBF16
  int zeros;         // != 0: with zero points
  const void* x;
  int x_type;
  int64_t ldx;
  int64_t n_rows;    // rows of x
  int64_t m;         // rows of y
  void* y;
  int y_type;
  int64_t ldy;
  const int32_t* offsets;  // per-expert products
  int n_expert;
  const int32_t* pairs;    // or null
  int top_k;
};
int launch_g4_qmv(const G4Args& a, hipStream_t s);
// by group
int launch_g4_32(const G4Args& a, hipStream_t s);
int launch_g4_64(const G4Args& a, hipStream_t s);
int launch_g4_128(const G4Args& a, hipStream_t s);

}  // namespace iq4
