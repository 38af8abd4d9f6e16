// w4a16_fp8_stream.hip - instantiations: products of up to sixteen rows (a tile), or 32.
#include "w4a16_fp8_stream.hpp"

namespace w4a16 {
namespace fp8 {

namespace {

// two slots a wave: more leave fewer workgroups on a compute unit, which costs more than the deeper ring gains
// (one row of 8192x10240, 16 columns, four waves: 18.6 us with two, 19.3, 25.6, 34.9 with four, six and eight)
template <int NT, int XC, int W, bool GLU>
hipError_t run(const StreamParams& p, unsigned grid, hipStream_t s) {
  const size_t lds = Stream<NT, XC, 2>::lds_bytes(W, XC ? 0 : p.slice * p.M);
  if (p.once) hipLaunchKernelGGL((fp8_stream_kernel<NT, XC, 2, W, GLU, true>), dim3(grid), dim3(64 * W), lds, s, p);
  else hipLaunchKernelGGL((fp8_stream_kernel<NT, XC, 2, W, GLU, false>), dim3(grid), dim3(64 * W), lds, s, p);
  return hipGetLastError();
}

template <int NT, int XC, bool GLU>
hipError_t by_waves(const StreamParams& p, int W, unsigned grid, hipStream_t s) {
  return W == 8 ? run<NT, XC, 8, GLU>(p, grid, s) : run<NT, XC, 4, GLU>(p, grid, s);
}

}  // namespace

// NT 1 (plain) or 2; XC 0 (x of 16 bits), 1, 2 or 4 (the latter with eight waves)
hipError_t launch_stream(const StreamParams& p, int NT, int XC, int W, bool glu, unsigned grid, hipStream_t s) {
  const auto with = [&](auto xc) {
    constexpr int C = decltype(xc)::value;
    if constexpr (C == 4) {
      if (glu) return run<2, C, 8, true>(p, grid, s);
      return NT == 1 ? run<1, C, 8, false>(p, grid, s) : run<2, C, 8, false>(p, grid, s);
    } else {
      if (glu) return by_waves<2, C, true>(p, W, grid, s);
      return NT == 1 ? by_waves<1, C, false>(p, W, grid, s) : by_waves<2, C, false>(p, W, grid, s);
    }
  };
  switch (XC) {
    case 0: return with(std::integral_constant<int, 0>{});
    case 1: return with(std::integral_constant<int, 1>{});
    case 2: return with(std::integral_constant<int, 2>{});
    default: return with(std::integral_constant<int, 4>{});
  }
}

}  // namespace fp8
}  // namespace w4a16
