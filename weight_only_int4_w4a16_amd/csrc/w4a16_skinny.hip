// w4a16_skinny.hip - launch geometry of the skinny kernel (w4a16_skinny_kernel.hpp).
#include <stdlib.h>

#include "w4a16_skinny_kernel.hpp"

namespace w4a16 {

namespace {

using namespace skinny;

struct SkinnyGeometry {
  int MT;
  int tiles_n, tiles_m, slice;
  size_t lds_bytes;
};

// W4A16_SKINNY_MT=1|2|4 pins the row tiles per workgroup (for benchmarking one against
// another); read once per process.
int forced_skinny_mt() {
  static const int forced = [] {
    const char* v = getenv("W4A16_SKINNY_MT");
    if (!v) return 0;
    const int mt = atoi(v);
    return mt == 1 || mt == 2 || mt == 4 ? mt : 0;
  }();
  return forced;
}

SkinnyGeometry skinny_geometry(int M, int K, int N, bool glu) {
  SkinnyGeometry g;
  const int KC = ceil_div(K, 128);
  g.tiles_n = glu ? (N / 2) / 32 + ((N / 2) % 32 ? 1 : 0) : ceil_div(N, 32 * kSkinnyPairs);
  // 64-row tiles up to 64 rows, and beyond where they fit one launch round; else 128-row tiles
  g.MT = M <= 32 ? 1 : (M <= 64 || (long)g.tiles_n * ceil_div(M, 64) <= device_cu_count()) ? 2 : 4;
  if (forced_skinny_mt()) g.MT = forced_skinny_mt();
  g.tiles_m = ceil_div(M, 32 * g.MT);
  g.slice = ceil_div(KC, skinny_waves(g.MT));
  g.lds_bytes = skinny_lds_bytes(g.MT);
  return g;
}

template <int ACT, int GPC, int FMT, int MT, bool GLU>
hipError_t launch_cfg(const SkinnyParams& p, const SkinnyGeometry& g, hipStream_t s) {
  hipLaunchKernelGGL((skinny_kernel<ACT, GPC, FMT, MT, GLU>), dim3(g.tiles_n, g.tiles_m),
                     dim3(64 * skinny_waves(MT)), g.lds_bytes, s, p);
  return hipGetLastError();
}

template <int ACT, int GPC, int FMT>
hipError_t launch_mt(const GemmArgs& a, const SkinnyParams& p, const SkinnyGeometry& g) {
  if (g.MT == 1)
    return a.glu ? launch_cfg<ACT, GPC, FMT, 1, true>(p, g, a.stream) : launch_cfg<ACT, GPC, FMT, 1, false>(p, g, a.stream);
  if (g.MT == 2)
    return a.glu ? launch_cfg<ACT, GPC, FMT, 2, true>(p, g, a.stream) : launch_cfg<ACT, GPC, FMT, 2, false>(p, g, a.stream);
  return a.glu ? launch_cfg<ACT, GPC, FMT, 4, true>(p, g, a.stream) : launch_cfg<ACT, GPC, FMT, 4, false>(p, g, a.stream);
}

template <int ACT, int GPC>
hipError_t launch_fmt(const GemmArgs& a, const SkinnyParams& p, const SkinnyGeometry& g) {
  if (a.nf4) return launch_mt<ACT, GPC, FMT_NF4>(a, p, g);
  if (a.qzeros) return launch_mt<ACT, GPC, FMT_ASYM>(a, p, g);
  return launch_mt<ACT, GPC, FMT_SYM>(a, p, g);
}

template <int ACT>
hipError_t launch_gpc(const GemmArgs& a, const SkinnyParams& p, const SkinnyGeometry& g) {
  switch (a.group_size) {
    case 128: return launch_fmt<ACT, 1>(a, p, g);
    case 64: return launch_fmt<ACT, 2>(a, p, g);
    default: return launch_fmt<ACT, 4>(a, p, g);
  }
}

}  // namespace

const char* skinny_name(int M, int K, int N) {
  const SkinnyGeometry g = skinny_geometry(M, K, N, false);
  return g.MT == 1 ? "w4a16_skinny_32x64" : g.MT == 2 ? "w4a16_skinny_64x64" : "w4a16_skinny_128x64";
}

// AWQ-scaled activations are not scaled in this kernel: the caller passes x' from the
// pre-pass (M K 2 bytes of workspace)
size_t skinny_awq_workspace_bytes(int M, int K, int N) {
  (void)N;
  return align256((size_t)M * K * 2);
}

hipError_t launch_skinny(const GemmArgs& a) {
  const SkinnyGeometry g = skinny_geometry(a.M, a.K, a.N, a.glu);
  SkinnyParams p;
  p.x = static_cast<const uint16_t*>(a.x);
  if (a.xscale) {
    if (!a.workspace || a.workspace_bytes < (size_t)a.M * a.K * 2) return hipErrorInvalidValue;
    const hipError_t e = launch_awq_scale(a.x, a.xscale, a.M, a.K, a.act, a.workspace, a.stream);
    if (e != hipSuccess) return e;
    p.x = static_cast<const uint16_t*>(a.workspace);
  }
  p.M = a.M;
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
  p.slice = g.slice;
  p.half = p.NT / 2;
  return a.act == ACT_F16 ? launch_gpc<ACT_F16>(a, p, g) : launch_gpc<ACT_BF16>(a, p, g);
}

}  // namespace w4a16
