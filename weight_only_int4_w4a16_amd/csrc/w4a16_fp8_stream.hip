// w4a16_fp8_stream.hip - instantiations: products of up to sixteen rows (a tile).
#include "w4a16_fp8_stream.hpp"

namespace w4a16 {
namespace fp8 {

namespace {

// two slots a wave: more leave fewer workgroups on a compute unit, which costs more than the deeper ring gains
// (one row of 8192x10240, 16 columns, four waves: 18.6 us with two, 19.3, 25.6, 34.9 with four, six and eight)
template <int NT, int XC, int W, bool GLU, bool GROUPED>
hipError_t run(const StreamParams& p, unsigned grid, hipStream_t s) {
  const size_t lds = Stream<NT, XC, 2>::lds_bytes(W, XC ? 0 : p.slice * p.M);
  if (p.once) hipLaunchKernelGGL((fp8_stream_kernel<NT, XC, 2, W, GLU, GROUPED, true>), dim3(grid), dim3(64 * W), lds, s, p);
  else hipLaunchKernelGGL((fp8_stream_kernel<NT, XC, 2, W, GLU, GROUPED, false>), dim3(grid), dim3(64 * W), lds, s, p);
  return hipGetLastError();
}

template <int NT, int XC, bool GLU, bool GROUPED>
hipError_t by_waves(const StreamParams& p, int W, unsigned grid, hipStream_t s) {
  return W == 8 ? run<NT, XC, 8, GLU, GROUPED>(p, grid, s) : run<NT, XC, 4, GLU, GROUPED>(p, grid, s);
}

}  // namespace

// NT 1 (plain) or 2, XC 0 (x of 16 bits), 1 (ungrouped rows) or 2
hipError_t launch_stream(const StreamParams& p, int NT, int XC, int W, bool glu, bool grouped, unsigned grid, hipStream_t s) {
  if (grouped) {
    if (glu) return by_waves<2, 2, true, true>(p, W, grid, s);
    return NT == 1 ? by_waves<1, 2, false, true>(p, W, grid, s) : by_waves<2, 2, false, true>(p, W, grid, s);
  }
  if (XC == 0) {
    if (glu) return by_waves<2, 0, true, false>(p, W, grid, s);
    return NT == 1 ? by_waves<1, 0, false, false>(p, W, grid, s) : by_waves<2, 0, false, false>(p, W, grid, s);
  }
  if (glu) return XC == 1 ? by_waves<2, 1, true, false>(p, W, grid, s) : by_waves<2, 2, true, false>(p, W, grid, s);
  if (NT == 1) return XC == 1 ? by_waves<1, 1, false, false>(p, W, grid, s) : by_waves<1, 2, false, false>(p, W, grid, s);
  return XC == 1 ? by_waves<2, 1, false, false>(p, W, grid, s) : by_waves<2, 2, false, false>(p, W, grid, s);
}

}  // namespace fp8
}  // namespace w4a16
