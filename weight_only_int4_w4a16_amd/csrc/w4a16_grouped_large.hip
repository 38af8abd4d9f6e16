// The batched kernel's grouped launches: rows sorted by group on the 128 x 512 tile.
#include "w4a16_tiled_kernel.hpp"

namespace w4a16 {

namespace tiled {
W4A16_TILED_INSTANTIATE_GROUPED(LargeTile)
}  // namespace tiled

hipError_t launch_grouped_large(const GemmArgs& a, const GroupTiles& t) {
  tiled::GroupedTiledParams p;
  p.x = static_cast<const uint16_t*>(a.x);
  p.M = 0;  // a tile ends where its entry in the list says
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
  p.tiles_m = t.bound;
  p.tiles_n = ceil_div(a.N, tiled::LargeTile::kBN);
  p.S = 1;
  p.kps = p.KC;
  p.partials = nullptr;
  p.half = p.NT / 2;
  p.groups = t;
  return tiled::launch_grouped_act<tiled::LargeTile>(a, p, dim3(p.tiles_m * p.tiles_n));
}

}  // namespace w4a16
