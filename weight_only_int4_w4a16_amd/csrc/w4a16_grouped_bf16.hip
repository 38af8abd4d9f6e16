// The grouped W4A16 kernel for few rows a group, instantiated for bf16 activations.
#include "w4a16_grouped_kernel.hpp"

namespace w4a16 {
namespace grouped {
template hipError_t launch_few<ACT_BF16>(const GroupedParams&, const GroupedGeometry&, int, bool, bool, hipStream_t);
}  // namespace grouped
}  // namespace w4a16
