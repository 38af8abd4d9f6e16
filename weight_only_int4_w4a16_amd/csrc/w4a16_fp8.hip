// w4a16_fp8.hip - which kernel takes a product of e4m3 codes, and its launch geometry.
#include "w4a16_fp8_tile.hpp"

namespace w4a16 {

using namespace fp8;

namespace {

template <class T, bool GLU, bool WROWS, int MODE>
hipError_t launch_tile(TileParams p, int gy, hipStream_t s) {
  const unsigned grid = (unsigned)((size_t)p.tiles_m * p.tiles_n);
  const dim3 blocks(grid, gy), threads(T::kThreads);
  if constexpr (WROWS) {  // a weight's gradient: fp32
    hipLaunchKernelGGL((fp8_tile_kernel<T, GLU, true, MODE, true>), blocks, threads, T::kLdsBytes, s, p);
  } else if (p.out_dtype >= 2) {
    hipLaunchKernelGGL((fp8_tile_kernel<T, GLU, false, MODE, true>), blocks, threads, T::kLdsBytes, s, p);
  } else {
    hipLaunchKernelGGL((fp8_tile_kernel<T, GLU, false, MODE, false>), blocks, threads, T::kLdsBytes, s, p);
  }
  return hipGetLastError();
}

TileParams tile_params(const Fp8Args& a) {
  TileParams p{};
  p.x = a.x;
  p.xs = a.xs;
  p.w = a.w;
  p.ws = a.ws;
  p.out = a.out;
  p.out_scales = a.out_scales;
  p.out_dtype = a.out_dtype;
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.KB = (int)fp8_blocks(a.K);
  p.ldk = a.ldk;
  p.xs_ld = a.xs_ld;
  p.up_blocks = (int)fp8_blocks(a.N);
  p.scale_rows = a.M;
  return p;
}

template <class T>
void set_tiles(TileParams& p, bool glu, int tiles_m) {
  p.tiles_m = tiles_m;
  p.tiles_n = ceil_div(p.N, glu ? T::kBN / 2 : T::kBN);
}

// Whether the 256 x 256 tiles fill the chip
bool large_fills(long long rows_tiles, int N, bool glu) {
  return rows_tiles * ceil_div(N, glu ? 128 : 256) * 2 >= device_cu_count();
}

}  // namespace

bool fp8_fits(int M, int N, int K, bool glu) {
  // offsets within a tile's operands, and of scales, in 31 bits; fewer than 2^32 threads
  const long long wrows = glu ? 2LL * N : 256;
  if ((long long)K >= (1LL << 23) || wrows * K >= (1LL << 31)) return false;
  if ((long long)fp8_blocks(K) * M * 4 >= (1LL << 31) || (long long)(fp8_blocks(N) + 1) * 2 * fp8_blocks(K) * 4 >= (1LL << 31))
    return false;
  return (long long)ceil_div(M, 128) * ceil_div(N, glu ? 64 : 128) * 256 < (1LL << 32);
}

size_t fp8_scratch_bytes(int M, int N, int K, bool glu, int out_dtype) {
  if (out_dtype != kE4M3 || large_fills(ceil_div(M, 256), N, glu)) return 0;
  return align256((size_t)M * N * 4);
}

const char* fp8_name(int M, int N, int K, bool glu) {
  return large_fills(ceil_div(M, 256), N, glu) ? "w4a16_fp8_256x256" : "w4a16_fp8_128x128";
}

hipError_t launch_fp8(const Fp8Args& a) {
  TileParams p = tile_params(a);
  const bool large = large_fills(ceil_div(a.M, 256), a.N, a.glu);
  const bool after = a.out_dtype == kE4M3 && !large;  // h in fp32 first
  if (after) {
    p.out = a.scratch;
    p.out_dtype = 2;
  }
  hipError_t e;
  if (large) {
    set_tiles<Large>(p, a.glu, ceil_div(a.M, 256));
    e = a.glu      ? launch_tile<Large, true, false, DENSE>(p, 1, a.stream)
        : a.w_rows ? launch_tile<Large, false, true, DENSE>(p, 1, a.stream)
                   : launch_tile<Large, false, false, DENSE>(p, 1, a.stream);
  } else {
    set_tiles<Small>(p, a.glu, ceil_div(a.M, 128));
    e = a.glu      ? launch_tile<Small, true, false, DENSE>(p, 1, a.stream)
        : a.w_rows ? launch_tile<Small, false, true, DENSE>(p, 1, a.stream)
                   : launch_tile<Small, false, false, DENSE>(p, 1, a.stream);
  }
  if (e != hipSuccess || !after) return e;
  return launch_fp8_rows(a.scratch, a.M, a.N, 2, static_cast<uint8_t*>(a.out), a.out_scales, a.stream);
}

// ---- grouped ----

namespace {

constexpr int kList128 = kTileLists - 1;

// row tiles of 256 to expect: full ones, and one part-filled a group
bool grouped_large(const RouteLayout& r, int N, bool glu) {
  const int groups = r.E < r.S ? r.E : r.S;
  return r.S / (groups > 0 ? groups : 1) >= 192 && large_fills(r.S / 256 + (groups + 1) / 2, N, glu);
}

GroupTiles group_tiles(const RouteLayout& r, const int32_t* plan, bool gather) {
  GroupTiles t;
  t.plan = plan;
  t.E = r.E;
  t.token = r.token;
  t.list = r.tiles[kList128];
  t.bound = tile_bound(r.S, r.E, kList128);
  t.tokens = gather ? r.S / r.topk : 0;
  return t;
}

}  // namespace

bool fp8_grouped_fits(const RouteLayout& r, int N, int K, bool glu) {
  if (!fp8_fits(r.S, N, K, glu)) return false;
  return (long long)tile_bound(r.S, r.E, kList128) * ceil_div(N, glu ? 64 : 128) * 512 < (1LL << 32);
}

size_t fp8_grouped_scratch_bytes(const RouteLayout& r, int N, int K, bool glu, int out_dtype) {
  if (out_dtype != kE4M3 || grouped_large(r, N, glu)) return 0;
  return align256((size_t)r.S * N * 4);
}

hipError_t launch_fp8_grouped(const Fp8Args& a, const RouteLayout& r, const int32_t* plan, bool gather) {
  TileParams p = tile_params(a);
  p.M = p.scale_rows = r.S;
  p.groups = group_tiles(r, plan, gather);
  const bool large = grouped_large(r, a.N, a.glu);
  const bool after = a.out_dtype == kE4M3 && !large;
  if (after) {
    p.out = a.scratch;
    p.out_dtype = 2;
  }
  hipError_t e;
  if (large) {
    set_tiles<Large>(p, a.glu, p.groups.bound);
    e = a.glu ? launch_tile<Large, true, false, GROUPED>(p, 1, a.stream)
              : launch_tile<Large, false, false, GROUPED>(p, 1, a.stream);
  } else {
    set_tiles<Small>(p, a.glu, p.groups.bound);
    e = a.glu ? launch_tile<Small, true, false, GROUPED>(p, 1, a.stream)
              : launch_tile<Small, false, false, GROUPED>(p, 1, a.stream);
  }
  if (e != hipSuccess || !after) return e;
  return launch_fp8_rows(a.scratch, r.S, a.N, 2, static_cast<uint8_t*>(a.out), a.out_scales, a.stream);
}

hipError_t launch_fp8_by_group(const Fp8Args& a, const RouteLayout& r, const int32_t* plan) {
  TileParams p = tile_params(a);
  p.groups = group_tiles(r, plan, false);
  if (large_fills((long long)ceil_div(a.M, 256) * r.E, a.N, false)) {
    set_tiles<Large>(p, false, ceil_div(a.M, 256));
    return launch_tile<Large, false, true, BY_GROUP>(p, r.E, a.stream);
  }
  set_tiles<Small>(p, false, ceil_div(a.M, 128));
  return launch_tile<Small, false, true, BY_GROUP>(p, r.E, a.stream);
}

}  // namespace w4a16
