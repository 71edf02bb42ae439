// mx.hpp -- the MXFP4 weight layout and the arguments of the products on it (mx.hip).
#pragma once
#include "common.hpp"
#include "rows.hpp"

namespace iq4 {

// Packed weights: 16-row x 128-element tiles, codes as the matrix instruction takes them,
// then one 32-bit word of scales per lane for each four tiles along k.
constexpr int kMxTileRows = 16;
constexpr int kMxTileK = 128;
constexpr int kMxTileBytes = 1024;   // codes of one tile: 64 lanes x 16 bytes
constexpr int kMxScaleBytes = 256;   // scales of four tiles: 64 lanes x 4 bytes

inline __host__ __device__ int64_t mx_row_tiles(int64_t n) { return (n + 15) / 16; }
inline __host__ __device__ int mx_k_tiles(int64_t k) { return (int)((k + 127) / 128); }
inline __host__ __device__ int mx_k_quads(int64_t k) { return (int)((k + 511) / 512); }
inline __host__ __device__ int64_t mx_code_plane(int64_t n, int64_t k) { return mx_row_tiles(n) * mx_k_tiles(k) * kMxTileBytes; }
inline int64_t mx_packed_bytes(int64_t n, int64_t k) {
  return mx_code_plane(n, k) + mx_row_tiles(n) * mx_k_quads(k) * kMxScaleBytes;
}

int launch_mx_pack(const uint8_t* codes, int64_t ldq, const uint8_t* scales, int64_t lds, int64_t n, int64_t k,
                   uint8_t* packed, hipStream_t s);

struct MxArgs {
  const uint8_t* W;           // packed; grouped: expert e at e * w_stride
  int64_t w_stride;
  int64_t n, k;
  const uint8_t* codes;       // activation rows
  int64_t ldq;
  const uint8_t* scales;
  int64_t lds;
  int64_t n_rows;             // rows of codes / scales
  int64_t m;                  // output rows (grouped: at most)
  void* y;
  int y_type;
  int64_t ldy;
  int vec_y;                  // y and ldy allow 16-byte stores
  // grouped: expert e's output rows are offsets[e] .. offsets[e + 1]
  const int32_t* offsets;
  int n_expert;
  const int32_t* pairs;       // activation row of output row i: pairs[i] / top_k (null: i)
  int top_k;
  float inv_top;              // 1 / top_k (set by the launcher)
};

int launch_mx_gemm(MxArgs a, int fmt, hipStream_t s);

}  // namespace iq4
