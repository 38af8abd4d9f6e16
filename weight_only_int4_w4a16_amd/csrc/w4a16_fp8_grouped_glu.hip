// w4a16_fp8_grouped_glu.hip - instantiations: the same with the SwiGLU epilogue.
#include "w4a16_fp8_tile.hpp"

namespace w4a16 {
namespace fp8 {
hipError_t launch_grouped_glu(const TileParams& p, int kind, bool exact, unsigned grid, int gy, hipStream_t s) {
  return launch_kind<true, false, GROUPED>(p, kind, exact, grid, gy, s);
}
}  // namespace fp8
}  // namespace w4a16
