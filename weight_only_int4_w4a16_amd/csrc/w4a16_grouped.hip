// w4a16_grouped.hip - which kernel takes a grouped W4A16 product, and its launch geometry.
#include <stdlib.h>
#include <string.h>

#include "w4a16_grouped_kernel.hpp"

namespace w4a16 {
namespace grouped {
extern template hipError_t launch_few<ACT_F16>(const GroupedParams&, const GroupedGeometry&, int, bool, bool, hipStream_t);
extern template hipError_t launch_few<ACT_BF16>(const GroupedParams&, const GroupedGeometry&, int, bool, bool, hipStream_t);
}  // namespace grouped

using namespace grouped;

namespace {

// tile rows of a launch, as indices of the plan's tile lists
enum Tile { TILE_16 = 0, TILE_32 = 1, TILE_64 = 2, TILE_128 = 3 };

// W4A16_GROUPED_ROWS=16|32|64|128 pins the row tile (for benchmarking one against another); read
// once per process.
int forced_tile() {
  static const int forced = [] {
    const char* v = getenv("W4A16_GROUPED_ROWS");
    if (!v) return -1;
    for (int j = 0; j < kTileLists; ++j)
      if (atoi(v) == kTileRows[j]) return j;
    return -1;
  }();
  return forced;
}

// The rows of each group are known on the device only, so the tile goes by their mean over the groups that can have
// rows.
Tile choose_tile(int S, int E) {
  if (forced_tile() >= 0) return (Tile)forced_tile();
  const int mean = S / (E < S ? E : S);
  return mean <= 12 ? TILE_16 : mean <= 24 ? TILE_32 : mean <= 64 ? TILE_64 : TILE_128;
}

int tile_cols(Tile t) { return t == TILE_128 ? 512 : 64; }
int tile_threads(Tile) { return 64 * 8; }

}  // namespace

const char* grouped_name(int S, int K, int N, int E, int group_size) {
  (void)K, (void)N, (void)group_size;
  switch (choose_tile(S, E)) {
    case TILE_16: return "w4a16_grouped_16x64";
    case TILE_32: return "w4a16_grouped_32x64";
    case TILE_64: return "w4a16_grouped_64x64";
    default: return "w4a16_grouped_128x512";
  }
}

// a launch holds fewer than 2^32 threads
bool grouped_fits(const RouteLayout& r, int N) {
  const Tile t = choose_tile(r.S, r.E);
  return (long long)tile_bound(r.S, r.E, t) * ceil_div(N, tile_cols(t)) * tile_threads(t) < (1LL << 32);
}

hipError_t launch_grouped(const GemmArgs& a, const RouteLayout& r, const int32_t* plan, bool gather) {
  const Tile tile = choose_tile(r.S, r.E);
  GroupTiles t;
  t.plan = plan;
  t.S = r.S;
  t.E = r.E;
  t.topk = r.topk;
  t.order = r.order;
  t.list = r.tiles[tile];
  t.bound = tile_bound(r.S, r.E, tile);
  t.tokens = gather ? r.S / r.topk : 0;
  if (tile == TILE_128) return launch_grouped_large(a, t);
  if (tile != TILE_16) return launch_grouped_skinny(a, t, kTileRows[tile]);
  GroupedParams p;
  p.x = static_cast<const uint16_t*>(a.x);
  p.groups = t;
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
  p.col_tiles = ceil_div(p.NT, g.SW);
  return a.act == ACT_F16 ? launch_few<ACT_F16>(p, g, a.group_size, a.nf4, a.glu, a.stream)
                          : launch_few<ACT_BF16>(p, g, a.group_size, a.nf4, a.glu, a.stream);
}

}  // namespace w4a16
