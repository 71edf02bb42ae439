// g4_32.hip -- products with 4-bit weights that have a scale per 32 (g4_kernel.hpp).
#include "g4_kernel.hpp"

namespace iq4 {

int launch_g4_32(const G4Args& a, hipStream_t s) {
  if (a.x_type == kF32) return launch_g4_group<kF32, 32>(a, s);
  return a.x_type == kF16 ? launch_g4_group<kF16, 32>(a, s) : launch_g4_group<kBF16, 32>(a, s);
}

}  // namespace iq4
