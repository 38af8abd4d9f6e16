// w4a16_route.hip - the plan that sends rows of one batch to different weights: a stable
// counting sort of the slots (token, choice) by group, and lists of row tiles for the kernels
// that multiply each group's rows with its own weight.
//
//   order[p]  the slot in sorted row p: groups ascending, slots ascending within a group, the
//             slots of no group (id outside [0, E)) last
//   slot[i]   the sorted row of slot i, or -1 for a slot of no group
//   offsets   group e's rows are [offsets[e], offsets[e + 1])
//
// A slot's sorted row is the sum of three counts of earlier slots: all of smaller groups, its
// own group's in earlier waves' (and workgroups') shares, and its own group's earlier in its
// wave. Lanes of one group find each other with one ballot per bit of the group number, so
// the rank inside a wave needs no atomics and the order never varies.
//
// The bytes are few (4 S read, 8 S written); a call is bound by the latency of its dependent
// steps. Up to 8192 slots one workgroup does everything in one launch; more take a count, a
// scan and a scatter launch over workgroups of 8192 slots.
#include "w4a16_device.hpp"
#include "w4a16_routed.hpp"

namespace w4a16 {

namespace {

constexpr int kThreads = 64 * kRouteWaves;

struct RouteParams {
  const int32_t* ids;
  int32_t* plan;
  RouteLayout r;
  int bits;  // of the largest group number E (the slots of no group)
};

struct WaveSlots {
  int g[kRouteBatches], rank[kRouteBatches];  // group (-1 past the end); earlier slots of it in the wave
};

// The wave's share of the block's slots: each lane's groups and their ranks within the wave, and
// in cnt[0..E] (LDS, zeroed) the wave's slots per group.
__device__ __forceinline__ void count_wave(const RouteParams& p, int first, int batches, int lane,
                                           int* cnt, WaveSlots& ws) {
  const int E = p.r.E;
#pragma unroll
  for (int b = 0; b < kRouteBatches; ++b) {
    const int i = first + b * 64 + lane;
    ws.g[b] = -1;
    if (b < batches && i < p.r.S) {
      const uint32_t id = (uint32_t)p.ids[i];
      ws.g[b] = id < (uint32_t)E ? (int)id : E;
    }
  }
#pragma unroll
  for (int b = 0; b < kRouteBatches; ++b) {
    if (b >= batches) break;
    const int g = ws.g[b];
    uint64_t same = __ballot(g >= 0);
    for (int t = 0; t < p.bits; ++t) {
      const uint64_t v = __ballot((g >> t) & 1);
      same &= ((g >> t) & 1) ? v : ~v;
    }
    ws.rank[b] = 0;
    if (g >= 0) {
      const int lower = __popcll(same & ((1ull << lane) - 1));
      // every lane of a group reads the count before the group's first lane adds to it
      const int before = __hip_atomic_load(cnt + g, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      ws.rank[b] = before + lower;
      __builtin_amdgcn_wave_barrier();
      if (lower == 0)
        __hip_atomic_store(cnt + g, before + __popcll(same), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// exclusive sums over the wave's lanes
__device__ __forceinline__ int wave_exclusive(int v, int lane, int& total) {
  int s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(s, o);
    if (lane >= o) s += u;
  }
  total = __shfl(s, 63);
  return s - v;
}

// One wave: out[g] = exclusive sum of ceil(tot[g] / rows) over g = 0..E, out[E + 1] the sum
__device__ __forceinline__ void scan_groups(const int* tot, int* out, int E, int rows, int lane) {
  int carry = 0;
  for (int g0 = 0; g0 <= E; g0 += 64) {
    const int g = g0 + lane;
    int total;
    const int n = g <= E ? (tot[g] + rows - 1) / rows : 0;
    const int s = wave_exclusive(n, lane, total);
    if (g <= E) out[g] = carry + s;
    carry += total;
  }
  if (lane == 0) out[E + 1] = carry;
}

// The groups' totals (LDS) -> offsets and tile lists of the plan, and off[0..E] in LDS. `scan`:
// (kTileLists + 1) * (E + 2) words of LDS.
__device__ __forceinline__ void write_groups(const RouteParams& p, const int* tot, int* scan) {
  const int E = p.r.E, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (wave == 0)
    scan_groups(tot, scan, E, 1, lane);
  else if (wave <= kTileLists)
    scan_groups(tot, scan + wave * (E + 2), E, kTileRows[wave - 1], lane);
  __syncthreads();
  for (int g = threadIdx.x; g <= E; g += kThreads) p.plan[g] = scan[g];
#pragma unroll
  for (int j = 0; j < kTileLists; ++j) {
    const int* first = scan + (j + 1) * (E + 2);
    int32_t* const list = p.plan + p.r.tiles[j];
    const int n = first[E + 1];
    if (threadIdx.x == 0) list[0] = n;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      int lo = 0, hi = E;  // the last group whose first tile is at or before i
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= i)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int row = scan[lo] + (i - first[lo]) * kTileRows[j];
      *reinterpret_cast<int4*>(list + 4 + 4 * i) = int4{lo, row, min(row + kTileRows[j], scan[lo + 1]), 0};
    }
  }
}

__device__ __forceinline__ void scatter_wave(const RouteParams& p, int first, int batches, int lane,
                                             const int* base, const WaveSlots& ws) {
  const int E = p.r.E;
#pragma unroll
  for (int b = 0; b < kRouteBatches; ++b) {
    if (b >= batches) break;
    const int g = ws.g[b];
    if (g < 0) continue;
    const int i = first + b * 64 + lane;
    const int row = base[g] + ws.rank[b];
    p.plan[p.r.order + row] = i;
    if (p.r.topk > 1) p.plan[p.r.token + row] = i / p.r.topk;
    p.plan[p.r.slot + i] = g < E ? row : -1;
  }
}

// cnt[w][g] -> the slots of group g in earlier waves (in place), tot[g] the block's
__device__ __forceinline__ void prefix_waves(int* cnt, int* tot, int E) {
  for (int g = threadIdx.x; g <= E; g += kThreads) {
    int s = 0;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) {
      const int v = cnt[w * (E + 1) + g];
      cnt[w * (E + 1) + g] = s;
      s += v;
    }
    tot[g] = s;
  }
}

// WHOLE: one workgroup sorts every slot. Otherwise the SCATTER pass of a block, after its
// first rows per group were scanned into the plan's hist, or the COUNT pass that fills hist.
enum { WHOLE = 0, COUNT = 1, SCATTER = 2 };
template <int PASS>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteParams p) {
  extern __shared__ int lds[];
  const int E = p.r.E, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int* const cnt = lds;                            // [kRouteWaves][E + 1]
  int* const tot = cnt + kRouteWaves * (E + 1);    // [E + 1]
  int* const scan = tot + (E + 1);                 // [kTileLists + 1][E + 2] (WHOLE)
  for (int i = threadIdx.x; i < kRouteWaves * (E + 1); i += kThreads) cnt[i] = 0;
  __syncthreads();
  // the waves take equal shares of the block's slots, in whole batches
  const int s0 = blockIdx.x * kRouteSlots;
  const int n = min(kRouteSlots, p.r.S - s0);
  const int batches = (n + 64 * kRouteWaves - 1) / (64 * kRouteWaves);
  const int first = s0 + wave * batches * 64;
  WaveSlots ws;
  count_wave(p, first, batches, lane, cnt + wave * (E + 1), ws);
  __syncthreads();
  prefix_waves(cnt, tot, E);
  __syncthreads();
  if constexpr (PASS == COUNT) {
    for (int g = threadIdx.x; g <= E; g += kThreads) p.plan[p.r.hist + blockIdx.x * (E + 1) + g] = tot[g];
    return;
  } else {
    if constexpr (PASS == WHOLE) {
      write_groups(p, tot, scan);
    } else {
      for (int g = threadIdx.x; g <= E; g += kThreads) scan[g] = p.plan[p.r.hist + blockIdx.x * (E + 1) + g];
      __syncthreads();
    }
    for (int i = threadIdx.x; i < kRouteWaves * (E + 1); i += kThreads) cnt[i] += scan[i % (E + 1)];
    __syncthreads();
    scatter_wave(p, first, batches, lane, cnt + wave * (E + 1), ws);
  }
}

// Between COUNT and SCATTER, one workgroup: hist[b][g] becomes block b's first row of group g
__global__ __launch_bounds__(kThreads) void route_scan_kernel(RouteParams p) {
  extern __shared__ int lds[];
  const int E = p.r.E;
  int* const tot = lds;
  int* const scan = lds + (E + 1);
  int32_t* const hist = p.plan + p.r.hist;
  for (int g = threadIdx.x; g <= E; g += kThreads) {
    int s = 0;
    for (int b = 0; b < p.r.blocks; ++b) s += hist[b * (E + 1) + g];
    tot[g] = s;
  }
  __syncthreads();
  write_groups(p, tot, scan);
  for (int g = threadIdx.x; g <= E; g += kThreads) {
    int s = scan[g];
    for (int b = 0; b < p.r.blocks; ++b) {
      const int v = hist[b * (E + 1) + g];
      hist[b * (E + 1) + g] = s;
      s += v;
    }
  }
}

}  // namespace

hipError_t launch_route(const int32_t* ids, const RouteLayout& r, int32_t* plan, hipStream_t s) {
  RouteParams p;
  p.ids = ids;
  p.plan = plan;
  p.r = r;
  p.bits = 0;
  while ((r.E >> p.bits) != 0) ++p.bits;
  const size_t count_lds = (size_t)(kRouteWaves + 1) * (r.E + 1) * 4;
  const size_t groups_lds = (size_t)(kTileLists + 1) * (r.E + 2) * 4;
  if (r.blocks == 1) {
    hipLaunchKernelGGL((route_kernel<WHOLE>), dim3(1), dim3(kThreads), count_lds + groups_lds, s, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((route_kernel<COUNT>), dim3(r.blocks), dim3(kThreads), count_lds, s, p);
  hipLaunchKernelGGL(route_scan_kernel, dim3(1), dim3(kThreads), (size_t)(r.E + 1) * 4 + groups_lds, s, p);
  hipLaunchKernelGGL((route_kernel<SCATTER>), dim3(r.blocks), dim3(kThreads), count_lds + (size_t)(r.E + 1) * 4, s, p);
  return hipGetLastError();
}

}  // namespace w4a16
