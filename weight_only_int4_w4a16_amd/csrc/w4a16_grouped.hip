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

// row tiles to expect: full ones, and about one part-filled for every second group
long long expected_tiles(int S, int groups, int rows) { return S / rows + (groups + 1) / 2; }

// Sixty-four rows: the waves side by side where that still makes two workgroups a compute unit (8
// experts of 4096x14336 at a mean of 64/128 rows 113/199 -> 102/166 us; 64 of 2048x2816 at 24/64/128:
// 59/100/174 -> 53/81/138).
bool side_by_side(int S, int groups, int N, long long cus) {
  return expected_tiles(S, groups, 64) * ceil_div(N / 16, kStrips * kWaves) >= 2 * cus;
}

// The rows of each group are known on the device only, so the tile goes by their mean over the
// groups that can have rows. That mean counts the slots of no group, whose number is known on the device only too: a
// call most of whose slots are such gets a taller tile than its rows need (8 of 64 experts of 4096x14336 on this
// device, bf16 g128, 512 tokens x 8, 496 live rows: the 128-row tile, 211 us; 64-row tiles 157; the live rows by
// themselves 108). A caller that can drop them before route() gains both. A taller tile forms W_hat once for more rows, but takes more registers
// and LDS, so that fewer waves run; the limits lie where tiles win on routings as uneven as gates make
// them (top-k of normal scores with expert biases of 0.7 sigma). us with 16/32/64/128 rows a tile, fp16
// g128 with zeros, by mean rows:
//   8 of 4096x14336   4 51/50/55, 8 45/43/46, 16 72/60/62, 24 88/70/75, 32 101/85/70, 48 135/104/92,
//                     128 320/237/167/217, 256 -/-/295/323, 384 -/-/432/430, 512 -/-/559/552, 768 -/-/821/711
//   64 of 2048x2816   4 31/33/37, 8 41/39/43, 16 53/46/45, 24 68/57/54, 32 83/69/61, 128 261/193/136/222,
//                     384 -/-/349/407, 768 -/-/664/669
// Deeper K (sorted rows, cold weights, the mean of four routings): the 32-row tile gains little between the others, but
// for groups of 32, whose four scales and zeros a block cost the 64-row tile a wave a SIMD:
//   8 of 14336x4096   g128 4 43/53/43, 8 50/59/48, 12 64/52/55, 16 72/70/61, 20 84/77/62, 28 109/85/92, 36 136/108/100,
//                     96 331/264/195/283, 128 406/369/292/283, 144 463/414/342/282, 192 577/536/471/287
//                     g32 4 59/56/79, 8 66/59/88, 16 94/87/99, 28 132/113/134, 40 164/129/154, 48 198/159/162
//                     NF4 bf16 4 54/73/56, 8 65/76/60, 12 84/64/64, 20 103/86/73, 28 130/94/106, 40 164/128/124
//   8 of 28672x8192   g128 3 154/146/152, 7 199/188/182, 12 234/207/205, 16 271/242/229, 24 393/310/292
//                     g32 5 201/204/289, 9 253/235/347, 16 321/292/372, 24 432/364/423
// Past 384 rows (144 where K > 8192) the 128 x 512 tile can still leave much of the chip idle (few groups, narrow N,
// a last round of workgroups with little in it): there the tile goes by a model of the time, in us. 64 x 64 tiles:
// 0.32 a tile and k-block with the waves side by side, 0.5 with K split over them (groups of 32: 0.42 and 0.65), divided
// by the compute units; 128 x 512: 26 a round of workgroups and 2.8 a round and k-block, 2.6 where one round holds them
// all. Fitted to both tiles' times at 320 points (28 shapes from 2 of 256x4096 to 8 of 28672x8192, means of 160 to 1536;
// fp16 g128 and g32, bf16 g128 and NF4): its choice is 0.7% above the better tile's time on average, more than 5% at 13
// points, among them one round and a few workgroups (16 of 11008x4096 at 192 rows: 510 for 390). 64/128 rows a tile:
//   64 of 1024x2048   400 142/189, 640 210/264, 1024 333/384;  64 of 2048x2816  400 364/413, 640 539/596, 1024 877/869
//   8 of 4096x14336   400 453/435, 640 676/589, 1024 1053/913; 8 of 14336x4096  256 343/305, 400 480/384, 512 598/656
double large_tile_us(int S, int groups, int KC, int N, long long cus) {
  const long long wgs = (S / 128 + groups / 2) * (long long)ceil_div(N, 512);
  const long long rounds = (wgs + cus - 1) / cus;
  return rounds > 1 ? rounds * (26 + 2.8 * KC) : 26 + 2.6 * KC;
}
double small_tile_us(int S, int groups, int KC, int N, int group_size, long long cus) {
  const bool split = !side_by_side(S, groups, N, cus);
  const double each = group_size == 32 ? (split ? 0.65 : 0.42) : (split ? 0.5 : 0.32);
  return (S / 64.0 + groups / 2) * ceil_div(N, 64) * KC * each / cus;
}

// a launch holds fewer than 2^32 threads
bool tile_fits(Tile t, int S, int E, int N) {
  return (long long)tile_bound(S, E, t) * ceil_div(N, t == TILE_128 ? 512 : 64) * 512 < (1LL << 32);
}

Tile choose_tile(int S, int E, int K, int N, int group_size) {
  if (forced_tile() >= 0) return (Tile)forced_tile();
  const int groups = E < S ? E : S;
  const int mean = S / (groups > 0 ? groups : 1);
  if (K > 8192) {
    if (mean <= 5) return TILE_16;
    if (group_size == 32 && mean <= 44) return TILE_32;
    if (mean <= 144) return TILE_64;
  } else {
    if (mean <= 6) return TILE_16;
    if (mean <= 28) return TILE_32;
    if (mean <= 384) return TILE_64;
  }
  const long long cus = device_cu_count();
  const int KC = ceil_div(K, 128);
  const bool small = small_tile_us(S, groups, KC, N, group_size, cus) < large_tile_us(S, groups, KC, N, cus);
  return small && tile_fits(TILE_64, S, E, N) ? TILE_64 : TILE_128;
}

}  // namespace

const char* grouped_name(int S, int K, int N, int E, int group_size) {
  switch (choose_tile(S, E, K, N, group_size)) {
    case TILE_16: return "w4a16_grouped_16x64";
    case TILE_32: return "w4a16_grouped_32x64";
    case TILE_64: return "w4a16_grouped_64x64";
    default: return "w4a16_grouped_128x512";
  }
}

// a tile's rows hold fewer than 2^31 bytes
bool grouped_fits(const RouteLayout& r, int K, int N, int group_size) {
  return K < (1 << 23) && tile_fits(choose_tile(r.S, r.E, K, N, group_size), r.S, r.E, N);
}

hipError_t launch_grouped(const GemmArgs& a, const RouteLayout& r, const int32_t* plan, bool gather) {
  const Tile tile = choose_tile(r.S, r.E, a.K, a.N, a.group_size);
  GroupTiles t;
  t.plan = plan;
  t.E = r.E;
  t.token = r.token;
  t.list = r.tiles[tile];
  t.bound = tile_bound(r.S, r.E, tile);
  t.tokens = gather ? r.S / r.topk : 0;
  if (tile == TILE_128) return launch_grouped_large(a, t);
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
  g.MT = kTileRows[tile] / 16;
  g.waves = kWaves;
  const long long cus = device_cu_count();
  const int groups = r.E < r.S ? r.E : r.S;
  const long long tiles = expected_tiles(r.S, groups, kTileRows[tile]);
  // Sixteen rows: eight waves share a deep K where the workgroups leave room on the compute units
  // (8 experts of 14336x4096 at 4 rows each, 512 workgroups: 55 -> 43 us; at K 4096 and 2048 four
  // waves are as good or better by up to 10%).
  const long long wgs = (tiles > groups ? tiles : groups) * ceil_div(p.NT, kStrips);
  if (g.MT == 1 && p.KC >= 64 && wgs <= 3 * cus) g.waves = 8;
  if (g.MT == 4 && side_by_side(r.S, groups, a.N, cus)) g.waves = 0;
  p.slice = g.waves ? ceil_div(p.KC, g.waves) : p.KC;
  p.col_tiles = ceil_div(p.NT, kStrips * (g.waves ? 1 : kWaves));
  return a.act == ACT_F16 ? launch_few<ACT_F16>(p, g, a.group_size, a.nf4, a.glu, a.stream)
                          : launch_few<ACT_BF16>(p, g, a.group_size, a.nf4, a.glu, a.stream);
}

}  // namespace w4a16
