// w4a16_routed.hpp - internal launchers of the routed operators (rows of one batch that go to
// different weights), behind the C ABI.
#pragma once

#include "w4a16_device.hpp"
#include "w4a16_launch.hpp"

namespace w4a16 {

// The plan w4a16_route writes, in int32 words from its start: offsets [E + 1], order [S],
// slot [S], the token of each sorted row [S] (with topk 1 the order itself), the tile lists, and
// (many slots) the per-block counts of the sort. S = tokens * topk.
// Tile list j cuts every group's rows into tiles of kTileRows[j] rows: a count, three unused
// words, then (group, first row, end, 0) per tile; group E's tiles are the slots of no group.
constexpr int kTileLists = 4;
constexpr int kTileRows[kTileLists] = {16, 32, 64, 128};
constexpr int kMaxGroups = 1024;
constexpr int kMaxSlots = 1 << 26;
constexpr int kRouteBlockSlots = 2048;  // slots per workgroup of the sort where there are several
constexpr int kRouteWholeSlots = 4096;  // most slots that one workgroup sorts alone
// Rows of so many bytes in one call, a quarter of the last-level cache, are stored (and read for the last
// time) past the caches. The gain is on rows that the caches do not hold: bf16, dispatch and combine of 8192 x 4096
// at topk 2 (128 MiB of sorted rows) 88 -> 71 us, adapters of 4096 x 8192 (64 MiB) 68 -> 60. Where a call's rows were
// just written, or are read next, the caches would have served it up to about their size (us by MiB of
// rows, 64/128/256/512, cached then streamed):
//   dispatch, combine                              32/60/153/298        34/64/123/245
//   combine_backward, one reader of dys            47/110/219/432       52/105/217/434
//   dispatch, product (4096 deep), combine         356/623/1160/2265    360/621/1160/2244
//   projection, adapters in place, projection      209/364/684/1350     210/366/692/1344
// so between products, as a layer has them, either way costs the other at most 1%.
constexpr size_t kStreamBytes = (size_t)64 << 20;
inline int round64(int n) { return (n + 63) & ~63; }
// most tiles list j can hold: full tiles, and one more for each group with rows
inline int tile_bound(int S, int E, int j) { return S / kTileRows[j] + (E + 1 < S ? E + 1 : S); }
struct RouteLayout {
  int S, E, topk;
  int order, slot, token, tiles[kTileLists], hist, words;  // word offsets; the total
  int blocks;                                        // workgroups of the sort
};
inline RouteLayout route_layout(int tokens, int topk, int E) {
  RouteLayout r;
  r.S = tokens * topk;
  r.E = E;
  r.topk = topk;
  r.blocks = r.S <= kRouteWholeSlots ? 1 : (r.S + kRouteBlockSlots - 1) / kRouteBlockSlots;
  r.order = round64(E + 1);
  r.slot = r.order + round64(r.S);
  int at = r.slot + round64(r.S);
  r.token = r.order;
  if (topk > 1) {
    r.token = at;
    at += round64(r.S);
  }
  for (int j = 0; j < kTileLists; ++j) {
    r.tiles[j] = at;
    at += round64(4 + 4 * tile_bound(r.S, E, j));
  }
  r.hist = at;
  r.words = at + (r.blocks > 1 ? round64(r.blocks * (E + 1)) : 0);
  return r;
}

// What a GEMM kernel's grouped instantiation reads besides its GEMM parameters
struct GroupTiles {
  const int32_t* plan;
  int E;
  int token, list;  // word offsets in the plan: the sorted rows' tokens, the tile list used
  int bound;        // most tiles the list can hold (the grid's)
  int tokens;       // rows of x where they are gathered through the plan, else 0
};
// tile ti of a list: its group e and sorted rows [p0, end); false past the list's end (an entry is in the plan
// whatever ti < bound, so that the count and the entry load at once)
__device__ __forceinline__ bool group_tile(const GroupTiles& g, int ti, int& e, int& p0, int& end) {
  const int32_t* const list = g.plan + g.list;
  const int4 t = *reinterpret_cast<const int4*>(list + 4 + 4 * ti);
  const int count = list[0];
  e = t.x;
  p0 = t.y;
  end = t.z;
  return ti < count;
}

// rows [row0, row0 + rows) by columns [col0, min(col0 + cols, width)) of an output of `width`
// columns cleared by the workgroup
__device__ inline void zero_tile(void* out, int out_dtype, int row0, int rows, int width, int col0, int cols) {
  const int n = min(cols, width - col0);
  for (int i = threadIdx.x; i < rows * n; i += blockDim.x) {
    const int r = i / n;
    store_out(out, (size_t)(row0 + r) * width + col0 + (i - r * n), 0.f, out_dtype);
  }
}

hipError_t launch_route(const int32_t* ids, const RouteLayout& r, int32_t* plan, hipStream_t s);
// A launch holds fewer than 2^32 threads: whether the tokens' rows make launches of the row movers
bool rows_fit(int tokens, int width);
// types of rows: 0 fp16, 1 bf16, 2 fp32 (as w4a16_dtype)
hipError_t launch_dispatch(const void* x, const RouteLayout& r, const int32_t* plan, int width, int dtype,
                           void* xs, hipStream_t s);
// weights NULL: every weight is 1
hipError_t launch_combine(const void* ys, const RouteLayout& r, const int32_t* plan, const float* weights,
                          int width, int dtype, void* y, int out_dtype, hipStream_t s);
hipError_t launch_combine_backward(const void* dy, const void* ys, const RouteLayout& r, const int32_t* plan,
                                   const float* weights, int width, int dtype, void* dys, float* dweights,
                                   hipStream_t s);
// a.x: the rows of the tokens (gather) or of the sorted slots; a.M unused; a.packed, a.scales and
// a.qzeros hold the groups' weights one after another
hipError_t launch_grouped(const GemmArgs& a, const RouteLayout& r, const int32_t* plan, bool gather);
// whether the rows and columns make a launch the kernels can index
bool grouped_fits(const RouteLayout& r, int K, int N, int group_size);
const char* grouped_name(int S, int K, int N, int E, int group_size);
constexpr int kMaxRank = 256;
// its launches on the batched kernel (128-row tiles)
hipError_t launch_grouped_large(const GemmArgs& a, const GroupTiles& t);
struct LoraArgs {
  const void* x;       // act [M][K]
  const void* y;       // ydtype [M][N]
  const void* lora_a;  // act [L][R][K]
  const void* lora_b;  // act [L][N][R]
  const int32_t* ids;  // [M] (read where no plan is given)
  const float* scaling;
  const int32_t* plan;
  void* out;           // ydtype [M][N]; may be y
  int M, K, N, L, R, act, ydtype;
  void* workspace;
  hipStream_t stream;
};
bool lora_fits(int M, int K, int N, int L, int R);  // its launches too, with a plan or without
size_t lora_workspace_bytes(int M, int K, int N, int L, int R, bool planned);
hipError_t launch_lora(const LoraArgs& a);

}  // namespace w4a16
