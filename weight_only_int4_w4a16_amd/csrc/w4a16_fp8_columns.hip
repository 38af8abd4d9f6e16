// w4a16_fp8_columns.hip - instantiations: gradients of weights, plain and by group.
#include "w4a16_fp8_tile.hpp"

namespace w4a16 {
namespace fp8 {
hipError_t launch_columns(const TileParams& p, int kind, bool exact, unsigned grid, int gy, hipStream_t s) {
  return launch_kind<false, true, DENSE>(p, kind, exact, grid, gy, s);
}
hipError_t launch_by_group(const TileParams& p, int kind, bool exact, unsigned grid, int gy, hipStream_t s) {
  return launch_kind<false, true, BY_GROUP>(p, kind, exact, grid, gy, s);
}
}  // namespace fp8
}  // namespace w4a16
