// w4a16_grouped.hip - launch geometry of the grouped W4A16 products.
#include "w4a16_grouped_kernel.hpp"

namespace w4a16 {
namespace grouped {
extern template hipError_t launch_few<ACT_F16>(const GroupedParams&, const GroupedGeometry&, int, bool, bool, hipStream_t);
extern template hipError_t launch_few<ACT_BF16>(const GroupedParams&, const GroupedGeometry&, int, bool, bool, hipStream_t);
}  // namespace grouped

using namespace grouped;

const char* grouped_name(int S, int K, int N, int E, int group_size) {
  (void)S, (void)K, (void)N, (void)E, (void)group_size;
  return "w4a16_grouped_16x64";
}

// a launch holds fewer than 2^32 threads
bool grouped_fits(const RouteLayout& r, int K, int N) {
  (void)K;
  return (long long)tile_bound(r.S, r.E, 0) * ceil_div(N / 16, 4) * 64 * kMaxWaves < (1LL << 32);
}

hipError_t launch_grouped(const GemmArgs& a, const RouteLayout& r, const int32_t* plan, bool gather) {
  GroupedParams p;
  p.x = static_cast<const uint16_t*>(a.x);
  p.plan = plan;
  p.S = r.S;
  p.E = r.E;
  p.topk = r.topk;
  p.order = r.order;
  p.tokens = gather ? r.S / r.topk : 0;
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
  p.half = p.NT / 2;
  GroupedGeometry g;
  g.SW = 4;
  g.waves = p.KC >= 2 * kMaxWaves ? kMaxWaves : p.KC >= 8 ? 4 : 2;
  p.slice = ceil_div(p.KC, g.waves);
  p.tiles = r.tiles[0];
  p.bound = tile_bound(r.S, r.E, 0);
  p.col_tiles = ceil_div(p.NT, g.SW);
  return a.act == ACT_F16 ? launch_few<ACT_F16>(p, g, a.group_size, a.nf4, a.glu, a.stream)
                          : launch_few<ACT_BF16>(p, g, a.group_size, a.nf4, a.glu, a.stream);
}

}  // namespace w4a16
