// experts.hpp -- where a tile of rows lies among rows sorted by expert: found by every wave on
// its own from the offsets, without a list of tiles or scratch memory.
#pragma once
#include "common.hpp"

namespace iq4 {

#ifdef __HIPCC__
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

// Tile t of `bm` rows, expert by expert (an expert's last tile may be partial): its expert, first
// row and rows.  False: there are fewer tiles.  128 experts at a time, their loads together.  Offsets are
// clamped to [0, m], an expert's end to its start or more: whatever they hold, no row outside is named.  Ones that
// do not ascend may name a row twice, or more tiles than there are columns for them: such rows are unspecified (a
// look at their order here costs every call 0.06 us).
__device__ __forceinline__ bool expert_tile(const int32_t* offsets, int n_expert, int m, int bm, int t, int& e, int& row0,
                                            int& rows) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < n_expert; e0 += 128) {
    int o0[2], o1[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int x = min(e0 + 64 * h + lane, n_expert - 1);
      o0[h] = offsets[x];
      o1[h] = offsets[x + 1];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      o0[h] = min(max(o0[h], 0), m);
      o1[h] = e0 + 64 * h + lane < n_expert ? min(max(o1[h], o0[h]), m) : o0[h];
      const int n = (o1[h] - o0[h] + bm - 1) / bm;
      const int upto = scan64(n);
      const int total = __builtin_amdgcn_readlane(upto, 63);
      if (t < total) {
        const int l = __builtin_ctzll(__ballot(upto > t));
        const int first = __builtin_amdgcn_readlane(o0[h], l);
        const int at = (t - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(n, l))) * bm;
        e = e0 + 64 * h + l;
        row0 = first + at;
        rows = min(bm, __builtin_amdgcn_readlane(o1[h], l) - row0);
        return true;
      }
      t -= total;
    }
  }
  return false;
}
#endif  // __HIPCC__

}  // namespace iq4
