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
// steps: read, rank, count, scan, place. So the scans use DPP, and the tile lists are written side by
// side, each by its share of the threads. Up to 4096 slots one workgroup does everything in one
// launch (four waves up to 512 slots, whose barriers are cheaper). More take two launches over
// workgroups of 2048 slots: the first counts its slots per group, and in the second every
// workgroup adds up all the counts itself, which saves a launch between them, and writes its share
// of the lists; only where the counts are many (over 64 Ki words) does a third kernel scan them once in
// between.
//
// Measured (us): 32 slots of 8 groups 3.5, 512 of 64 5.6, 1600 of 64 6.2, 4096 of 16 7.2; 16384 of 8 4.7 + 6.8,
// 131072 of 128 5.0 + 10.6. With the third kernel, whose one workgroup walks all the counts twice, whole calls:
// 131072 of 1024 62, 200000 of 1024 85, 4 Mi of 128 1200. (With shuffles for the scans and the lists one after another: 5.1, 7.6, 8.0,
// 8.3; 7.2 and 15.3 for the second launches.)
#include "w4a16_device.hpp"
#include "w4a16_routed.hpp"

namespace w4a16 {

namespace {

struct RouteParams {
  const int32_t* ids;
  int32_t* plan;
  RouteLayout r;
  int bits;      // of the largest group number E (the slots of no group)
  bool scanned;  // hist holds each block's first rows, and the plan its offsets and lists
};

template <int B>
struct WaveSlots {
  int g[B], rank[B];  // group (-1 past the end); earlier slots of it in the wave
};

// The wave's share of the block's slots: each lane's groups and their ranks within the wave, and
// in cnt[0..E] (LDS, zeroed) the wave's slots per group.
template <int B>
__device__ __forceinline__ void count_wave(const RouteParams& p, int first, int batches, int lane,
                                           int* cnt, WaveSlots<B>& ws) {
  const int E = p.r.E;
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const int i = first + b * 64 + lane;
    ws.g[b] = -1;
    if (b < batches && i < p.r.S) {
      const uint32_t id = (uint32_t)p.ids[i];
      ws.g[b] = id < (uint32_t)E ? (int)id : E;
    }
  }
#pragma unroll
  for (int b = 0; b < B; ++b) {
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

// v of the lane that a DPP control names, 0 where it names none or the row is masked off
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or_0(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
// exclusive sums over the wave's lanes (DPP: a shuffle goes through LDS, six in a row for each scan)
__device__ __forceinline__ int wave_exclusive(int v, int& total) {
  int s = v;
  s += dpp_or_0<0x111, 0xF>(s);  // one lane to the right in its row of sixteen, then 2, 4, 8
  s += dpp_or_0<0x112, 0xF>(s);
  s += dpp_or_0<0x114, 0xF>(s);
  s += dpp_or_0<0x118, 0xF>(s);
  s += dpp_or_0<0x142, 0xA>(s);  // lane 15 of rows 0 and 2 to rows 1 and 3
  s += dpp_or_0<0x143, 0xC>(s);  // lane 31 to rows 2 and 3
  total = __builtin_amdgcn_readlane(s, 63);
  return s - v;
}

// One wave: out[g] = exclusive sum of ceil(tot[g] / rows) over g = 0..E, out[E + 1] the sum
__device__ __forceinline__ void scan_groups(const int* tot, int* out, int E, int rows, int lane) {
  int carry = 0;
  for (int g0 = 0; g0 <= E; g0 += 64) {
    const int g = g0 + lane;
    int total;
    const int n = g <= E ? (tot[g] + rows - 1) / rows : 0;
    const int s = wave_exclusive(n, total);
    if (g <= E) out[g] = carry + s;
    carry += total;
  }
  if (lane == 0) out[E + 1] = carry;
}

// scan[0..E+1]: the groups' first rows and S; scan + (j + 1) (E + 2): their first tiles in list j
__device__ __forceinline__ void scan_all(const int* tot, int* scan, int E, int W) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int j = wave; j <= kTileLists; j += W)
    scan_groups(tot, scan + j * (E + 2), E, j ? kTileRows[j - 1] : 1, lane);
  __syncthreads();
}

// tile list j of the plan from the scans, by threads `thread` of `threads`
__device__ __forceinline__ void write_list(const RouteParams& p, const int* scan, int j, int thread, int threads) {
  const int E = p.r.E;
  const int* first = scan + (j + 1) * (E + 2);
  int32_t* const list = p.plan + p.r.tiles[j];
  const int n = first[E + 1], tile_rows = kTileRows[j];
  if (thread == 0) list[0] = n;
  for (int i = thread; i < n; i += threads) {
    int lo = 0, hi = E;  // the last group whose first tile is at or before i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= i)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int row = scan[lo] + (i - first[lo]) * tile_rows;
    *reinterpret_cast<int4*>(list + 4 + 4 * i) = int4{lo, row, min(row + tile_rows, scan[lo + 1]), 0};
  }
}

template <int B>
__device__ __forceinline__ void scatter_wave(const RouteParams& p, int first, int batches, int lane,
                                             const int* base, const WaveSlots<B>& ws) {
  const int E = p.r.E;
#pragma unroll
  for (int b = 0; b < B; ++b) {
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

// WHOLE: one workgroup sorts every slot. COUNT and SCATTER: a workgroup of several; COUNT fills the
// block's row of hist, SCATTER places its slots. W waves of at most B 64-slot batches.
enum { WHOLE = 0, COUNT = 1, SCATTER = 2 };
template <int PASS, int W, int B>
__global__ __launch_bounds__(64 * W) void route_kernel(RouteParams p) {
  extern __shared__ int lds[];
  const int E = p.r.E, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int PER = 64 * W / kTileLists;  // threads of a tile list
  int* const cnt = lds;                  // [W][E + 1]
  int* const tot = cnt + W * (E + 1);    // [E + 1]: the block's (SCATTER: all blocks') slots per group
  int* const base = tot + (E + 1);       // [E + 1]: SCATTER: slots of the group in earlier blocks
  int* const scan = base + (E + 1);      // [kTileLists + 1][E + 2]
  for (int i = threadIdx.x; i < W * (E + 1); i += 64 * W) cnt[i] = 0;
  __syncthreads();
  // the waves take equal shares of the block's slots, in whole batches
  const int s0 = blockIdx.x * (64 * W * B);
  const int n = min(64 * W * B, p.r.S - s0);
  const int batches = (n + 64 * W - 1) / (64 * W);
  const int first = s0 + wave * batches * 64;
  WaveSlots<B> ws;
  count_wave(p, first, batches, lane, cnt + wave * (E + 1), ws);
  __syncthreads();
  // cnt[w][g] -> the slots of group g in earlier waves
  for (int g = threadIdx.x; g <= E; g += 64 * W) {
    int s = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int v = cnt[w * (E + 1) + g];
      cnt[w * (E + 1) + g] = s;
      s += v;
    }
    if constexpr (PASS == COUNT)
      p.plan[p.r.hist + blockIdx.x * (E + 1) + g] = s;
    else
      tot[g] = s;
  }
  if constexpr (PASS == COUNT) return;
  __syncthreads();
  if constexpr (PASS == WHOLE) {
    scan_all(tot, scan, E, W);
    for (int g = threadIdx.x; g <= E; g += 64 * W) p.plan[g] = scan[g];
    write_list(p, scan, threadIdx.x / PER, threadIdx.x % PER, PER);
  } else {
    const int32_t* const hist = p.plan + p.r.hist;
    if (p.scanned) {
      for (int g = threadIdx.x; g <= E; g += 64 * W) scan[g] = hist[blockIdx.x * (E + 1) + g];
      __syncthreads();
    } else {
      // every block's counts, over all blocks and over those before this one: the threads of a group
      // take the blocks in turn and add with LDS atomics (whole numbers, so in any order)
      for (int g = threadIdx.x; g <= E; g += 64 * W) tot[g] = base[g] = 0;
      __syncthreads();
      const int parts = max(1, 64 * W / (E + 1));
      for (int i = threadIdx.x; i < parts * (E + 1); i += 64 * W) {
        const int part = i / (E + 1), g = i - part * (E + 1);
        int all = 0, before = 0;
#pragma unroll 8
        for (int b = part; b < p.r.blocks; b += parts) {
          const int v = hist[b * (E + 1) + g];
          all += v;
          before += b < (int)blockIdx.x ? v : 0;
        }
        atomicAdd(tot + g, all);
        atomicAdd(base + g, before);
      }
      __syncthreads();
      scan_all(tot, scan, E, W);
      if (blockIdx.x == 0)
        for (int g = threadIdx.x; g <= E; g += 64 * W) p.plan[g] = scan[g];
      write_list(p, scan, threadIdx.x / PER, blockIdx.x * PER + threadIdx.x % PER, p.r.blocks * PER);
      __syncthreads();
      for (int g = threadIdx.x; g <= E; g += 64 * W) scan[g] += base[g];
      __syncthreads();
    }
  }
  for (int i = threadIdx.x; i < W * (E + 1); i += 64 * W) cnt[i] += scan[i % (E + 1)];
  __syncthreads();
  scatter_wave(p, first, batches, lane, cnt + wave * (E + 1), ws);
}

// Between COUNT and SCATTER where the counts are many: hist[b][g] becomes block b's first row of group g
constexpr int kScanWaves = 16;
__global__ __launch_bounds__(64 * kScanWaves) void route_scan_kernel(RouteParams p) {
  extern __shared__ int lds[];
  const int E = p.r.E;
  int* const tot = lds;
  int* const scan = lds + (E + 1);
  int32_t* const hist = p.plan + p.r.hist;
  for (int g = threadIdx.x; g <= E; g += 64 * kScanWaves) {
    int s = 0;
#pragma unroll 8
    for (int b = 0; b < p.r.blocks; ++b) s += hist[b * (E + 1) + g];
    tot[g] = s;
  }
  __syncthreads();
  scan_all(tot, scan, E, kScanWaves);
  for (int g = threadIdx.x; g <= E; g += 64 * kScanWaves) p.plan[g] = scan[g];
  constexpr int PER = 64 * kScanWaves / kTileLists;
  write_list(p, scan, threadIdx.x / PER, threadIdx.x % PER, PER);
  for (int g = threadIdx.x; g <= E; g += 64 * kScanWaves) {
    int s = scan[g];
    for (int b = 0; b < p.r.blocks; ++b) {
      const int v = hist[b * (E + 1) + g];
      hist[b * (E + 1) + g] = s;
      s += v;
    }
  }
}

template <int PASS, int W, int B>
void launch_pass(const RouteParams& p, hipStream_t s) {
  const int E = p.r.E;
  const size_t words = (size_t)(W + 2) * (E + 1) + (size_t)(kTileLists + 1) * (E + 2);
  hipLaunchKernelGGL((route_kernel<PASS, W, B>), dim3(p.r.blocks), dim3(64 * W), words * 4, s, p);
}

}  // namespace

hipError_t launch_route(const int32_t* ids, const RouteLayout& r, int32_t* plan, hipStream_t s) {
  RouteParams p;
  p.ids = ids;
  p.plan = plan;
  p.r = r;
  p.bits = 0;
  while ((r.E >> p.bits) != 0) ++p.bits;
  p.scanned = false;
  if (r.S <= 512) {
    launch_pass<WHOLE, 4, 2>(p, s);
  } else if (r.blocks == 1) {
    launch_pass<WHOLE, 16, kRouteWholeSlots / 1024>(p, s);
  } else {
    launch_pass<COUNT, 16, kRouteBlockSlots / 1024>(p, s);
    if ((long long)r.blocks * (r.E + 1) > (1 << 16)) {
      p.scanned = true;
      const size_t words = (size_t)(r.E + 1) + (size_t)(kTileLists + 1) * (r.E + 2);
      hipLaunchKernelGGL(route_scan_kernel, dim3(1), dim3(64 * kScanWaves), words * 4, s, p);
    }
    launch_pass<SCATTER, 16, kRouteBlockSlots / 1024>(p, s);
  }
  return hipGetLastError();
}

}  // namespace w4a16
