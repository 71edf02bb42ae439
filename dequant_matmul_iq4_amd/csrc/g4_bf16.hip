// g4_bf16.hip -- group-scaled 4-bit weights times bfloat16 rows (g4_kernel.hpp).
#include "g4_kernel.hpp"

namespace iq4 {

int launch_g4_bf16(const G4Args& a, hipStream_t s) {
  const int64_t rows = a.offsets ? (a.m + a.n_expert - 1) / a.n_expert : a.m;
  if (rows <= 16) return launch_g4_group<kG4Brain, 1, 1, 4>(a, s);
  if (rows <= 32) return launch_g4_group<kG4Brain, 2, 1, 2>(a, s);
  if (rows <= 48) return launch_g4_group<kG4Brain, 3, 1, 2>(a, s);
  return launch_g4_group<kG4Brain, 4, 1, 2>(a, s);
}

}  // namespace iq4
