// The skinny kernel's grouped launches: rows sorted by group, tiles of 32 or 64 rows.
#include "w4a16_grouped_kernel.hpp"
#include "w4a16_skinny_kernel.hpp"

namespace w4a16 {

namespace {

using namespace skinny;

template <int ACT, int GPC, int FMT, int MT>
hipError_t launch_mt(const GemmArgs& a, const GroupedSkinnyParams& p) {
  const dim3 grid(p.groups.bound * p.tiles_n), block(64 * skinny_waves(MT));
  const size_t lds = skinny_lds_bytes(MT);
  if (a.glu)
    hipLaunchKernelGGL((skinny_kernel<ACT, GPC, FMT, MT, true, GroupedSkinnyParams>), grid, block, lds, a.stream, p);
  else
    hipLaunchKernelGGL((skinny_kernel<ACT, GPC, FMT, MT, false, GroupedSkinnyParams>), grid, block, lds, a.stream, p);
  return hipGetLastError();
}

template <int ACT, int GPC, int MT>
hipError_t launch_fmt(const GemmArgs& a, const GroupedSkinnyParams& p) {
  if (a.nf4) return launch_mt<ACT, GPC, skinny::FMT_NF4, MT>(a, p);
  if (a.qzeros) return launch_mt<ACT, GPC, skinny::FMT_ASYM, MT>(a, p);
  return launch_mt<ACT, GPC, skinny::FMT_SYM, MT>(a, p);
}

template <int ACT, int MT>
hipError_t launch_gpc(const GemmArgs& a, const GroupedSkinnyParams& p) {
  switch (a.group_size) {
    case 128: return launch_fmt<ACT, 1, MT>(a, p);
    case 64: return launch_fmt<ACT, 2, MT>(a, p);
    default: return launch_fmt<ACT, 4, MT>(a, p);
  }
}

template <int MT>
hipError_t launch_act(const GemmArgs& a, const GroupedSkinnyParams& p) {
  return a.act == ACT_F16 ? launch_gpc<ACT_F16, MT>(a, p) : launch_gpc<ACT_BF16, MT>(a, p);
}

}  // namespace

hipError_t launch_grouped_skinny(const GemmArgs& a, const GroupTiles& t, int rows) {
  GroupedSkinnyParams p;
  p.x = static_cast<const uint16_t*>(a.x);
  p.M = t.S;
  p.K = a.K;
  p.N = a.N;
  p.packed = reinterpret_cast<const u4_t*>(a.packed);
  p.scales = static_cast<const uint16_t*>(a.scales);
  p.qzeros = a.qzeros;
  p.codebook = a.codebook;
  p.out = a.out;
  p.out_dtype = a.out_dtype;
  p.KC = ceil_div(a.K, 128);
  p.NT = a.N / 16;
  p.NG = a.K / a.group_size;
  p.slice = ceil_div(p.KC, skinny_waves(rows / 32));
  p.half = p.NT / 2;
  p.groups = t;
  p.tiles_n = a.glu ? ceil_div(p.half, 2) : ceil_div(p.NT, 2 * kSkinnyPairs);
  return rows == 32 ? launch_act<1>(a, p) : launch_act<2>(a, p);
}

}  // namespace w4a16
