// g4_f32.hip -- group-scaled 4-bit weights times binary32 rows (g4_kernel.hpp).
#include "g4_kernel.hpp"

namespace iq4 {

int launch_g4_f32(const G4Args& a, hipStream_t s) {
  // rows of a tile: by expert as many as an expert has on average
  const int64_t rows = a.offsets ? (a.m + a.n_expert - 1) / a.n_expert : a.m;
  if (rows <= 4) return launch_g4_group<kG4Parts4, 1, 1, 4>(a, s);
  if (rows <= 16) return launch_g4_group<kG4Parts16, 1, 1, 2>(a, s);
  return launch_g4_group<kG4Parts16, 2, 1, 2>(a, s);
}

}  // namespace iq4
