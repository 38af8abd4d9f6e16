// w4a16_lora.hip - low-rank adapters of many requests beside a projection all rows share:
//
//   out[m] = y[m] + s[a] (x[m] A[a]^T) B[a]^T,  a = ids[m]   (out[m] = y[m] where a is none)
//
// with x[M][K], A[L][R][K], B[L][N][R] of the activation type and y the projection's output. Rows
// are grouped by adapter (the plan of w4a16_route), so a tile of rows reads its adapter once;
// at decode the adapters' bytes R (K + N) bound the call, at prefill those of x, y and out.
//
// Two launches. The first forms t = x A^T, at most R values a row: a workgroup takes a tile of
// rows and a slice of K, its waves parts of the slice, added through LDS in wave order; the slices' fp32 sums go
// to the workspace. The second adds the slices in order and multiplies by B.
//
// t in 16-bit MFMA operands. Rounding t once would cost as much as rounding the product, so t
// is split into parts of the activation type, t = t0 + t1 (+ t2), each the rounding of what
// the ones before left: 22 (fp16), 16 or 24 (bf16, three parts where out is fp32) bits of t,
// and the parts' products with B add in fp32. fp16 parts of a large or small t could leave
// the type's range, so a row is first scaled by the power of two that brings its largest |t|
// into [1, 2); the scale goes back into s.
//
// Operands of the second product. B is the A operand (16 columns n of the output) and t the B
// operand (16 rows m), so a lane ends with consecutive n of one row: the four MFMAs of a
// 64-column strip take the columns n0 + 16 (i/4) + 4 q + i%4, and lane l then holds all
// sixteen of n0 + 16 (l/16) .. of row l%16, two 16-byte accesses to y and out.
#include "w4a16_device.hpp"
#include "w4a16_routed.hpp"

namespace w4a16 {

namespace {

enum { T_F16 = 0, T_BF16 = 1, T_F32 = 2 };

template <int ACT>
struct ActT;
template <>
struct ActT<ACT_F16> { typedef h8_t type; };
template <>
struct ActT<ACT_BF16> { typedef b8_t type; };

constexpr int kShrinkWaves = 8;
constexpr int kExpandWaves = 4;
constexpr int kRankChunk = 64;  // ranks per workgroup of the first product
constexpr int kMaxSlices = 16;

struct LoraParams {
  const uint16_t *x, *a, *b;
  const void* y;
  void* out;
  const float* scaling;
  const int32_t* plan;
  float* part;  // [slices][M][R]
  int order, tiles, bound;
  int M, K, N, L, R;
  int slices, steps;  // K slices; 32-deep steps per wave
};

__device__ __forceinline__ int group_end(const LoraParams& p, int e) { return e < p.L ? p.plan[e + 1] : p.M; }

// t of 16 MT rows and up to 16 RT ranks over one K slice
template <int ACT, int MT, int RT>
__global__ __launch_bounds__(64 * kShrinkWaves) void shrink_kernel(LoraParams p) {
  typedef typename ActT<ACT>::type AT;
  extern __shared__ __attribute__((aligned(16))) float red[];  // [waves][MT][RT][4][64]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t* const list = p.plan + p.tiles;
  if ((int)blockIdx.x >= list[0]) return;
  const int e = list[4 + 2 * blockIdx.x], p0 = list[5 + 2 * blockIdx.x];
  if (e >= p.L) return;  // rows without an adapter
  const int rows = min(16 * MT, group_end(p, e) - p0);
  const int r0 = blockIdx.z * kRankChunk;
  const int koff = 8 * (lane >> 4);
  const uint16_t *xp[MT], *ap[RT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)  // rows past the tile repeat its last, never stored
    xp[mt] = p.x + (size_t)p.plan[p.order + p0 + min(16 * mt + (lane & 15), rows - 1)] * p.K + koff;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)  // and so do ranks past the last
    ap[rt] = p.a + ((size_t)e * p.R + min(r0 + 16 * rt + (lane & 15), p.R - 1)) * p.K + koff;
  f4_t acc[MT][RT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[mt][rt] = f4_t{0.f, 0.f, 0.f, 0.f};
  const int s0 = (blockIdx.y * kShrinkWaves + wave) * p.steps;
  const int s1 = min(s0 + p.steps, p.K / 32);
  constexpr int U = MT == 1 ? 4 : 2;  // steps in flight
  for (int s = s0; s < s1; s += U) {
    u4_t xv[U][MT], av[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = 32 * min(s + u, s1 - 1);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) xv[u][mt] = *reinterpret_cast<const u4_t*>(xp[mt] + k);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) av[u][rt] = *reinterpret_cast<const u4_t*>(ap[rt] + k);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= s1) break;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          acc[mt][rt] = mfma16(__builtin_bit_cast(AT, xv[u][mt]), __builtin_bit_cast(AT, av[u][rt]), acc[mt][rt]);
    }
  }
  // lane l holds rank l%16 and rows 4 (l/16) + i, i < 4
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[(((wave * MT + mt) * RT + rt) * 4 + i) * 64 + lane] = acc[mt][rt][i];
  __syncthreads();
  float* const part = p.part + ((size_t)blockIdx.y * p.M + p0) * p.R + r0;
  for (int q = threadIdx.x; q < rows * RT * 16; q += 64 * kShrinkWaves) {
    const int m = q / (RT * 16), r = q - m * (RT * 16);
    if (r0 + r >= p.R) continue;
    const int at = ((((m >> 4) * RT + (r >> 4)) * 4 + (m & 3)) * 64) + ((m >> 2) & 3) * 16 + (r & 15);
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kShrinkWaves; ++w) v += red[w * MT * RT * 256 + at];
    part[(size_t)m * p.R + r] = v;
  }
}

// sixteen consecutive elements of a row of y or out
template <int YT>
__device__ __forceinline__ void load16(const void* base, size_t at, float (&f)[16]) {
  if constexpr (YT == T_F32) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const f4_t v = *reinterpret_cast<const f4_t*>(static_cast<const float*>(base) + at + 4 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[4 * c + i] = v[i];
    }
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const u4_t v = *reinterpret_cast<const u4_t*>(static_cast<const uint16_t*>(base) + at + 8 * c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint16_t b = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
        f[8 * c + i] = YT == T_F16 ? (float)__builtin_bit_cast(_Float16, b) : __builtin_bit_cast(float, (uint32_t)b << 16);
      }
    }
  }
}
template <int YT>
__device__ __forceinline__ void store16(void* base, size_t at, const float (&f)[16]) {
  if constexpr (YT == T_F32) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<f4_t*>(static_cast<float*>(base) + at + 4 * c) = f4_t{f[4 * c], f[4 * c + 1], f[4 * c + 2], f[4 * c + 3]};
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      u4_t v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = f[8 * c + 2 * i], hi = f[8 * c + 2 * i + 1];
        if constexpr (YT == T_F16)
          v[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)lo) | (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)hi) << 16;
        else
          v[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)lo) | (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16;
      }
      *reinterpret_cast<u4_t*>(static_cast<uint16_t*>(base) + at + 8 * c) = v;
    }
  }
}

// The parts of eight values of t (the first the rounding of t, each next that of the rest). An
// infinity or NaN keeps its first part and has no rest.
template <int ACT, int PARTS>
__device__ __forceinline__ void split8(const float (&t)[8], typename ActT<ACT>::type (&part)[PARTS]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float rest = t[i];
#pragma unroll
    for (int s = 0; s < PARTS; ++s) {
      if constexpr (ACT == ACT_F16)
        part[s][i] = (_Float16)rest;
      else
        part[s][i] = (__bf16)rest;
      rest = __builtin_isfinite(rest) ? rest - (float)part[s][i] : 0.f;
    }
  }
}

// RS: 32-rank steps
template <int ACT, int YT, int RS>
__global__ __launch_bounds__(64 * kExpandWaves) void expand_kernel(LoraParams p, int tile_rows) {
  typedef typename ActT<ACT>::type AT;
  constexpr int PARTS = ACT == ACT_BF16 && YT == T_F32 ? 3 : 2;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t* const list = p.plan + p.tiles;
  if ((int)blockIdx.x >= list[0]) return;
  const int e = list[4 + 2 * blockIdx.x], p0 = list[5 + 2 * blockIdx.x];
  const int rows = min(tile_rows, group_end(p, e) - p0);
  const int n0 = (blockIdx.y * kExpandWaves + wave) * 64;
  const int col = n0 + 16 * (lane >> 4);  // this lane's sixteen columns
  if (n0 >= p.N) return;
  const bool mine = col < p.N;  // N is a multiple of 16
  if (e >= p.L) {               // no adapter: out is y
    if (p.out == p.y) return;
    for (int m = lane & 15; m < rows; m += 16) {
      const size_t at = (size_t)p.plan[p.order + p0 + m] * p.N + col;
      float f[16];
      if (mine) {
        load16<YT>(p.y, at, f);
        store16<YT>(p.out, at, f);
      }
    }
    return;
  }
  u4_t bv[4][RS];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int i = lane & 15, n = min(n0 + 16 * (i >> 2) + 4 * q + (i & 3), p.N - 1);
    const uint16_t* src = p.b + ((size_t)e * p.N + n) * p.R;
#pragma unroll
    for (int rs = 0; rs < RS; ++rs) {
      const int r = 32 * rs + 8 * (lane >> 4);  // R is a multiple of 8
      bv[q][rs] = r < p.R ? *reinterpret_cast<const u4_t*>(src + r) : u4_t{0, 0, 0, 0};
    }
  }
  const float scaling = p.scaling[e];
  for (int m0 = 0; m0 < rows; m0 += 16) {
    const int m = min(m0 + (lane & 15), rows - 1);
    const size_t at = (size_t)p.plan[p.order + p0 + m] * p.N + col;
    float f[16];
    if (mine) load16<YT>(p.y, at, f);
    float t[RS][8];
#pragma unroll
    for (int rs = 0; rs < RS; ++rs)
#pragma unroll
      for (int i = 0; i < 8; ++i) t[rs][i] = 0.f;
    for (int s = 0; s < p.slices; ++s) {
      const float* src = p.part + ((size_t)s * p.M + p0 + m) * p.R;
#pragma unroll
      for (int rs = 0; rs < RS; ++rs) {
        const int r = 32 * rs + 8 * (lane >> 4);
        if (r >= p.R) continue;
        const f4_t lo = *reinterpret_cast<const f4_t*>(src + r), hi = *reinterpret_cast<const f4_t*>(src + r + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          t[rs][i] += lo[i];
          t[rs][4 + i] += hi[i];
        }
      }
    }
    float back = scaling;
    if constexpr (ACT == ACT_F16) {
      float big = 0.f;
#pragma unroll
      for (int rs = 0; rs < RS; ++rs)
#pragma unroll
        for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(t[rs][i]));
      big = fmaxf(big, __shfl_xor(big, 16));
      big = fmaxf(big, __shfl_xor(big, 32));
      // 2^-e of the row's largest value, from its exponent bits (kept off the ends of the range)
      const int ex = min(max((int)(__builtin_bit_cast(uint32_t, big) >> 23), 27), 227);
      const float down = __builtin_bit_cast(float, (uint32_t)(254 - ex) << 23);
      back *= __builtin_bit_cast(float, (uint32_t)ex << 23);
#pragma unroll
      for (int rs = 0; rs < RS; ++rs)
#pragma unroll
        for (int i = 0; i < 8; ++i) t[rs][i] *= down;
    }
    f4_t acc[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int rs = 0; rs < RS; ++rs) {
      AT part[PARTS];
      split8<ACT, PARTS>(t[rs], part);
#pragma unroll
      for (int s = 0; s < PARTS; ++s)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = mfma16(__builtin_bit_cast(AT, bv[q][rs]), part[s], acc[q]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) f[4 * q + i] = __builtin_fmaf(back, acc[q][i], f[4 * q + i]);
    if (mine && m0 + (lane & 15) < rows) store16<YT>(p.out, at, f);
  }
}

struct LoraGeometry {
  int shrink_list, expand_list;  // tile lists
  int slices, steps;
};

LoraGeometry lora_geometry(int M, int K, int N, int L, int R) {
  (void)N;
  LoraGeometry g;
  const int groups = L < M ? L : M;
  const int per_group = M / (groups > 0 ? groups : 1);
  g.shrink_list = per_group >= 48 ? 2 : 0;
  g.expand_list = per_group >= 48 ? 2 : 0;
  // slices of K until the tiles fill the compute units, at least four steps a wave
  const long long tiles = (long long)(M / kTileRows[g.shrink_list] + (groups + 1) / 2 + 1) * ceil_div(R, kRankChunk);
  const int steps = K / 32;
  int slices = (int)(device_cu_count() / tiles);
  const int most = steps / (4 * kShrinkWaves);
  if (slices > most) slices = most;
  if (slices > kMaxSlices) slices = kMaxSlices;
  if (slices < 1) slices = 1;
  g.steps = ceil_div(steps, slices * kShrinkWaves);
  g.slices = ceil_div(steps, g.steps * kShrinkWaves);
  return g;
}

template <int ACT, int MT>
void launch_shrink(const LoraParams& p, dim3 grid, hipStream_t s) {
  const dim3 block(64 * kShrinkWaves);
  const size_t lds = (size_t)kShrinkWaves * MT * 256 * 4;  // per rank tile
  if (p.R <= 16)
    hipLaunchKernelGGL((shrink_kernel<ACT, MT, 1>), grid, block, lds, s, p);
  else if (p.R <= 32)
    hipLaunchKernelGGL((shrink_kernel<ACT, MT, 2>), grid, block, 2 * lds, s, p);
  else
    hipLaunchKernelGGL((shrink_kernel<ACT, MT, 4>), grid, block, 4 * lds, s, p);
}

template <int ACT, int YT>
void launch_expand(const LoraParams& p, dim3 grid, int rows, hipStream_t s) {
  const dim3 block(64 * kExpandWaves);
  if (p.R <= 32)
    hipLaunchKernelGGL((expand_kernel<ACT, YT, 1>), grid, block, 0, s, p, rows);
  else if (p.R <= 64)
    hipLaunchKernelGGL((expand_kernel<ACT, YT, 2>), grid, block, 0, s, p, rows);
  else if (p.R <= 128)
    hipLaunchKernelGGL((expand_kernel<ACT, YT, 4>), grid, block, 0, s, p, rows);
  else
    hipLaunchKernelGGL((expand_kernel<ACT, YT, 8>), grid, block, 0, s, p, rows);
}

}  // namespace

size_t lora_workspace_bytes(int M, int K, int N, int L, int R, bool planned) {
  const LoraGeometry g = lora_geometry(M, K, N, L, R);
  const size_t plan = planned ? 0 : align256((size_t)route_layout(M, 1, L).words * 4);
  return plan + align256((size_t)g.slices * M * R * 4);
}

hipError_t launch_lora(const LoraArgs& a) {
  const LoraGeometry g = lora_geometry(a.M, a.K, a.N, a.L, a.R);
  const RouteLayout r = route_layout(a.M, 1, a.L);
  char* ws = static_cast<char*>(a.workspace);
  LoraParams p;
  p.plan = a.plan;
  if (!p.plan) {
    int32_t* plan = reinterpret_cast<int32_t*>(ws);
    ws += align256((size_t)r.words * 4);
    const hipError_t e = launch_route(a.ids, r, plan, a.stream);
    if (e != hipSuccess) return e;
    p.plan = plan;
  }
  p.x = static_cast<const uint16_t*>(a.x);
  p.a = static_cast<const uint16_t*>(a.lora_a);
  p.b = static_cast<const uint16_t*>(a.lora_b);
  p.y = a.y;
  p.out = a.out;
  p.scaling = a.scaling;
  p.part = reinterpret_cast<float*>(ws);
  p.order = r.order;
  p.M = a.M;
  p.K = a.K;
  p.N = a.N;
  p.L = a.L;
  p.R = a.R;
  p.slices = g.slices;
  p.steps = g.steps;
  p.tiles = r.tiles[g.shrink_list];
  p.bound = tile_bound(r.S, r.E, g.shrink_list);
  const dim3 sgrid(p.bound, g.slices, ceil_div(a.R, kRankChunk));
  if (a.act == ACT_F16)
    g.shrink_list ? launch_shrink<ACT_F16, 4>(p, sgrid, a.stream) : launch_shrink<ACT_F16, 1>(p, sgrid, a.stream);
  else
    g.shrink_list ? launch_shrink<ACT_BF16, 4>(p, sgrid, a.stream) : launch_shrink<ACT_BF16, 1>(p, sgrid, a.stream);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  p.tiles = r.tiles[g.expand_list];
  p.bound = tile_bound(r.S, r.E, g.expand_list);
  const dim3 egrid(p.bound, ceil_div(a.N, 64 * kExpandWaves));
  const int rows = kTileRows[g.expand_list];
  if (a.act == ACT_F16)
    a.ydtype == T_F32 ? launch_expand<ACT_F16, T_F32>(p, egrid, rows, a.stream)
                      : launch_expand<ACT_F16, T_F16>(p, egrid, rows, a.stream);
  else
    a.ydtype == T_F32 ? launch_expand<ACT_BF16, T_F32>(p, egrid, rows, a.stream)
                      : launch_expand<ACT_BF16, T_BF16>(p, egrid, rows, a.stream);
  return hipGetLastError();
}

}  // namespace w4a16
