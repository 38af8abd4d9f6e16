// w4a16_fp8_grouped.hip - instantiations: products of sorted rows with their groups' weights.
#include "w4a16_fp8_tile.hpp"

namespace w4a16 {
namespace fp8 {
hipError_t launch_grouped_plain(const TileParams& p, int kind, bool exact, unsigned grid, int gy, hipStream_t s) {
  return launch_kind<false, false, GROUPED>(p, kind, exact, grid, gy, s);
}
}  // namespace fp8
}  // namespace w4a16
