// w4a16_lora.hip - low-rank adapters of many requests beside a projection all rows share:
//
//   out[m] = y[m] + s[a] (x[m] A[a]^T) B[a]^T,  a = ids[m]   (out[m] = y[m] where a is none)
//
// with x[M][K], A[L][R][K], B[L][N][R] of the activation type and y the projection's output.
// A workgroup takes a tile of rows with one adapter, so at decode the adapters' bytes
// R (K + N) bound the call, at prefill those of x, y and out.
//
// Tiles. Up to 96 rows, workgroup b looks at row b: if the row is the first, 17th, 33rd.. of its
// adapter, the tile is that row and the next fifteen of the adapter, found with one ballot
// per 64 ids; else it leaves. That saves the sort's launch (5 us; at 256 rows the workgroups
// that leave cost more: 33 us against 16 + 5 at 8192x8192 rank 64). More rows, or a plan in
// hand, take the plan's tile lists.
//
// Two launches, or one where t is cheap. The first forms t = x A^T, at most R values a row: a
// workgroup takes a tile of rows and a slice of K, its waves parts of the slice, added through
// LDS in a fixed order; the slices' fp32 sums go to the workspace. The second adds the slices in
// order and multiplies by B.
//
// t in 16-bit MFMA operands. Rounding t once would cost as much as rounding the product, so t
// is split into parts of the activation type, t = t0 + t1 (+ t2), each the rounding of what
// the ones before left, and the parts' products with B add in fp32. bf16 parts hold 16 bits of
// each t (24 in three parts, where out is fp32). fp16 parts of a large or small t could leave
// the type's range, so a row is first scaled by the power of two that brings its largest |t|
// into [1, 2), and the scale goes back into s: they hold 22 bits of that largest t, and of a smaller one
// what is above 2^-25 of it. A workgroup splits its rows' t once, in LDS, for all its columns.
//
// Operands of the second product. B is the A operand (16 columns n of the output) and t the B
// operand (16 rows m), so a lane ends with four consecutive n of one row. A wave's 16 x 64 product is
// turned through its own LDS, so that y and out are accessed by whole 128-byte runs of a row.
//
// Measured: one row, 4096x4096 rank 16 fp16 9.8 us (one launch; two took 14.0); 96 rows with 64
// adapters, 4096x14336 rank 32 bf16 18 us (62 MB; first product 7.7, second 11.7 at 5.5 TB/s); 4096 rows
// with 9 adapters, 8192x8192 rank 64 bf16 60 us (208 MB; sort 7.2, first product 18.2, then the second).
#include <limits.h>

#include <type_traits>

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
constexpr int expand_waves(bool one) { return one ? kShrinkWaves : 4; }  // of the second product
constexpr int kRankChunk = 64;   // ranks per workgroup of the first product
constexpr int kMaxSlices = 16;
constexpr int kSetSteps = 4;     // 32-deep steps of a register set in the first product
constexpr int kSelfRows = 96;    // most rows whose tiles the workgroups find themselves
constexpr int kTileMax = 64;     // most rows of a tile

struct LoraParams {
  const uint16_t *x, *a, *b;
  const void* y;
  void* out;
  const float* scaling;
  const int32_t* ids;  // where the tiles are found here, else NULL
  GroupTiles groups;   // else
  float* part;         // [slices][M][R], by row of x
  int M, K, N, L, R;
  int slices, steps;   // K slices; 32-deep steps per slice
  int tile_rows;
  int strips;          // 64-column strips per wave of the second product
  int col_groups;      // workgroups per tile of it
};

// This workgroup's tile: the rows of x (in LDS, complete after the caller's barrier), their number
// and their adapter (L: none). False if it has none.
__device__ __forceinline__ bool find_tile(const LoraParams& p, int tile, int* rows_of, int& rows, int& e) {
  const int lane = threadIdx.x & 63;
  if (p.ids) {
    const int b = tile;
    const uint32_t id = (uint32_t)p.ids[b];
    e = id < (uint32_t)p.L ? (int)id : p.L;
    constexpr int kBatches = (kSelfRows + 63) / 64;
    uint64_t same[kBatches];
    int before = 0;  // rows of this adapter ahead of row b
#pragma unroll
    for (int c = 0; c < kBatches; ++c) {
      const int m = 64 * c + lane;
      const uint32_t other = (uint32_t)p.ids[min(m, p.M - 1)];
      same[c] = __ballot(m < p.M && (other < (uint32_t)p.L ? (int)other : p.L) == e);
      const int left = b - 64 * c;  // rows of this batch ahead of b
      if (left > 0) before += __popcll(left >= 64 ? same[c] : same[c] & ((1ull << left) - 1));
    }
    if (before & 15) return false;
    int at = 0;  // rows of the adapter seen
#pragma unroll
    for (int c = 0; c < kBatches; ++c) {
      const int pos = at + __popcll(same[c] & ((1ull << lane) - 1)) - before;
      if (((same[c] >> lane) & 1) && pos >= 0 && pos < 16 && threadIdx.x < 64) rows_of[pos] = 64 * c + lane;
      at += __popcll(same[c]);
    }
    rows = min(16, at - before);
    return true;
  }
  int p0, end;
  if (!group_tile(p.groups, tile, e, p0, end)) return false;
  rows = min(p.tile_rows, end - p0);
  if ((int)threadIdx.x < rows) rows_of[threadIdx.x] = p.groups.plan[p.groups.token + p0 + threadIdx.x];
  return true;
}

// t of a 16-row tile and up to 16 RT ranks from r0 on, over the 32-deep steps [s0, s1), by kShrinkWaves waves
// (rows_of complete). It ends in red, [kShrinkWaves / 2][RT][4][64], whose first index shrink_sum adds up.
template <int ACT, int RT>
__device__ __forceinline__ void shrink_tile(const LoraParams& p, const int* rows_of, int rows, int e, int r0, int s0,
                                            int s1, float* red) {
  typedef typename ActT<ACT>::type AT;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int koff = 8 * (lane >> 4);
  const uint16_t* ap[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)  // ranks past the last repeat it, never stored
    ap[rt] = p.a + ((size_t)e * p.R + min(r0 + 16 * rt + (lane & 15), p.R - 1)) * p.K + koff;
  const uint16_t* const xp = p.x + (size_t)rows_of[min(lane & 15, rows - 1)] * p.K + koff;  // and so do rows past the tile
  f4_t acc[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) acc[rt] = f4_t{0.f, 0.f, 0.f, 0.f};
  constexpr int U = kSetSteps;  // steps per register set; one set loads while the other multiplies
  struct Regs {
    u4_t x[U], a[U][RT];
  };
  // The slice's sets go to the waves in turn, 512 bytes of a row at a time (less where a wave
  // would get none). The rows of x and of A are K apart, at a power of two K all in one memory
  // channel; with the eight waves 512 bytes apart their loads cover 4 KiB of each row, and so every channel.
  const int all = (s1 - s0 + U - 1) / U;
  const int shift = all >= 2 * kShrinkWaves ? 1 : 0;
  const int full = (all / kShrinkWaves) >> shift;
  const int sets = (full << shift) + min(max(all - ((full * kShrinkWaves + wave) << shift), 0), 1 << shift);
  auto first = [&](int i) __attribute__((always_inline)) {
    return s0 + ((((i >> shift) * kShrinkWaves + wave) << shift) + (i & ((1 << shift) - 1))) * U;
  };
  auto load = [&](Regs& R, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = 32 * min(first(i) + u, s1 - 1);
      R.x[u] = *reinterpret_cast<const u4_t*>(xp + k);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) R.a[u][rt] = *reinterpret_cast<const u4_t*>(ap[rt] + k);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](const Regs& R, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (first(i) + u >= s1) break;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        acc[rt] = mfma16(__builtin_bit_cast(AT, R.x[u]), __builtin_bit_cast(AT, R.a[u][rt]), acc[rt]);
    }
  };
  if (sets > 0) {
    Regs A, B;
    load(A, 0);
    int i = 0;
    for (; i + 2 < sets; i += 2) {
      load(B, i + 1);
      multiply(A, i);
      load(A, i + 2);
      multiply(B, i + 1);
    }
    if (i + 1 < sets) {
      load(B, i + 1);
      multiply(A, i);
      multiply(B, i + 1);
    } else {
      multiply(A, i);
    }
  }
  // The waves' sums, in two rounds through half the LDS that all would take (so that two workgroups
  // share a compute unit): wave w + 4's go to wave w, then the four sums in order. Lane l holds
  // rank l%16 and rows 4 (l/16) + i, i < 4.
  constexpr int H = kShrinkWaves / 2, TILE = RT * 256;
  if (wave >= H) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[(wave - H) * TILE + (rt * 4 + i) * 64 + lane] = acc[rt][i];
  }
  __syncthreads();
  if (wave < H) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float* const at = red + wave * TILE + (rt * 4 + i) * 64 + lane;
        *at = acc[rt][i] + *at;
      }
  }
  __syncthreads();
}
// rank r (of the tile's 16 RT) of row m of it
template <int RT>
__device__ __forceinline__ float shrink_sum(const float* red, int m, int r) {
  const int at = ((r >> 4) * 4 + (m & 3)) * 64 + (m >> 2) * 16 + (r & 15);
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kShrinkWaves / 2; ++w) v += red[w * RT * 256 + at];
  return v;
}

// one K slice of t
template <int ACT, int RT>
__global__ __launch_bounds__(64 * kShrinkWaves) void shrink_kernel(LoraParams p) {
  extern __shared__ __attribute__((aligned(16))) float red[];
  __shared__ int rows_of[kTileMax];
  // consecutive workgroups (on consecutive XCDs) take a tile's slices
  const int tile = blockIdx.x / p.slices, slice = blockIdx.x - tile * p.slices;
  int rows, e;
  if (!find_tile(p, tile, rows_of, rows, e)) return;
  if (e >= p.L) return;  // rows without an adapter
  __syncthreads();
  const int r0 = blockIdx.y * kRankChunk, s0 = slice * p.steps;
  shrink_tile<ACT, RT>(p, rows_of, rows, e, r0, s0, min(s0 + p.steps, p.K / 32), red);
  for (int q = threadIdx.x; q < rows * RT * 16; q += 64 * kShrinkWaves) {
    const int m = q / (RT * 16), r = q - m * (RT * 16);
    if (r0 + r < p.R) p.part[((size_t)slice * p.M + rows_of[m]) * p.R + r0 + r] = shrink_sum<RT>(red, m, r);
  }
}

// workgroup -> item, so that consecutive items run on the same XCD
__device__ __forceinline__ int tile_of(int b, int G) {
  const int q = G >> 3, r = G & 7, x = b & 7;
  return x * q + (x < r ? x : r) + (b >> 3);
}

// t of a 64-row tile over one K slice, for prefill: the same product, but with x and A through
// LDS. Loaded in the MFMA's layout, sixteen lanes touch sixteen rows of x (or of A): a 1 KiB
// load then takes the address unit 64 cycles, and 66 tiles of 64 rows over 8192 columns, rank 64,
// took 27 us. Here a 128-column block of both goes from memory straight into one of
// kStages slots, four rows of 256 bytes per instruction, three blocks ahead of the product. Row
// r of a slot holds its chunks at positions c ^ (r % 16), so a fragment read touches every bank
// once. Two waves share 16 rows, each with half of a block's columns and every rank, and are added
// at the end: alone on its SIMD, a wave of 16 rows left its pipes idle half the time (22 us; with two
// 18.2; the bytes, 75 MB, take 11-14). The slots fill the LDS, so one workgroup runs a compute unit; two with
// two slots each and twice the slices took 20-23 us. A slice's tiles are neighbours on one XCD, where
// they share A (19.5 us without).
constexpr int kStages = 4, kTallWaves = 8;
template <int RT>
constexpr int tall_slot() { return (64 + 16 * RT) * 128; }  // halves

template <int n>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((n & 0xF) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8));
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

__device__ __forceinline__ void copy16_to_lds(const uint16_t* src, uint16_t* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

template <int ACT, int RT>
__global__ __launch_bounds__(64 * kTallWaves) void shrink_tall_kernel(LoraParams p) {
  typedef typename ActT<ACT>::type AT;
  // A wave's loads of a block: eight rows of x, and its share of A's 16 RT ranks (one rank tile's
  // twice, by two waves)
  constexpr int XL = 2, AL = RT > 1 ? RT / 2 : 1, LOADS = XL + AL;
  extern __shared__ __attribute__((aligned(16))) uint16_t ring[];  // [kStages][tall_slot]
  __shared__ int rows_of[kTileMax];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int item = tile_of(blockIdx.x, p.groups.bound * p.slices);
  const int slice = item / p.groups.bound, tile = item - slice * p.groups.bound;
  int rows, e;
  if (!find_tile(p, tile, rows_of, rows, e)) return;
  if (e >= p.L) return;  // rows without an adapter
  const int r0 = blockIdx.y * kRankChunk;
  const int strip = wave & 3, half = wave >> 2;
  __syncthreads();
  // instruction j covers four rows; lane l row l/16 of them, position l%16. Rows and ranks past the last
  // repeat it, never stored; chunks past a ragged K repeat its last, never multiplied.
  const uint16_t* src[LOADS];
  int chunk[LOADS];
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    const int r = j < XL ? 4 * (wave * XL + j) + (lane >> 4) : 4 * ((wave * AL + j - XL) % (4 * RT)) + (lane >> 4);
    chunk[j] = 8 * ((lane & 15) ^ (r & 15));
    src[j] = j < XL ? p.x + (size_t)rows_of[min(r, rows - 1)] * p.K
                   : p.a + ((size_t)e * p.R + min(r0 + r, p.R - 1)) * p.K;
  }
  auto load = [&](int kb, int slot) __attribute__((always_inline)) {
    uint16_t* const base = ring + slot * tall_slot<RT>();
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      uint16_t* const dst = base + (j < XL ? 4 * (wave * XL + j) : 64 + 4 * ((wave * AL + j - XL) % (4 * RT))) * 128;
      copy16_to_lds(src[j] + min(128 * kb + chunk[j], p.K - 8), dst);
    }
  };
  f4_t acc[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) acc[rt] = f4_t{0.f, 0.f, 0.f, 0.f};
  const int b0 = slice * p.steps / 4, b1 = min(b0 + p.steps / 4, (p.K + 127) / 128);  // steps: whole blocks
  const int nb = b1 - b0;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i)
    if (i < nb) load(b0 + i, i);
  for (int i = 0; i < nb; ++i) {
    // block i has landed: only the loads of the up to two blocks after it may be in flight
    const int later = nb - 1 - i;
    if (later >= 2)
      wait_loads<2 * LOADS>();
    else if (later == 1)
      wait_loads<LOADS>();
    else
      wait_loads<0>();
    __builtin_amdgcn_s_barrier();  // every wave's part of it, and every wave is done with block i - 1
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
    if (i + kStages - 1 < nb) load(b0 + i + kStages - 1, (i + kStages - 1) % kStages);
    const uint16_t* const base = ring + (i % kStages) * tall_slot<RT>();
    const int row = lane & 15;
    auto step = [&](int s) __attribute__((always_inline)) {
      const int at = ((4 * s + (lane >> 4)) ^ row) * 8;
      const u4_t xv = *reinterpret_cast<const u4_t*>(base + (16 * strip + row) * 128 + at);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const u4_t av = *reinterpret_cast<const u4_t*>(base + (64 + 16 * rt + row) * 128 + at);
        acc[rt] = mfma16(__builtin_bit_cast(AT, xv), __builtin_bit_cast(AT, av), acc[rt]);
      }
    };
    const int left = p.K - 128 * (b0 + i);
    if (left >= 128) {  // without branches the steps' reads are all in flight together
#pragma unroll
      for (int s = 0; s < 2; ++s) step(2 * half + s);
    } else {
      for (int s = 2 * half; s < 2 * half + 2 && 32 * s < left; ++s) step(s);
    }
  }
  // the second halves of the blocks, through LDS
  __syncthreads();  // every wave is done with the slots
  f4_t* const other = reinterpret_cast<f4_t*>(ring) + strip * RT * 64 + lane;
  if (half == 1)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) other[rt * 64] = acc[rt];
  __syncthreads();
  if (half == 1) return;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) acc[rt] += other[rt * 64];
  // lane l holds rank l%16 of each tile and rows 4 (l/16) + i, i < 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = 16 * strip + 4 * (lane >> 4) + i;
    if (m >= rows) continue;
    float* const part = p.part + ((size_t)slice * p.M + rows_of[m]) * p.R + r0;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      if (r0 + 16 * rt + (lane & 15) < p.R) part[16 * rt + (lane & 15)] = acc[rt][i];
  }
}

// Sixteen bytes of a row of y or out per lane and access: kPer columns; a 16 x 64 tile takes
// kAccesses of them, access h rows kRows h .. of the tile
template <int YT>
struct Cols {
  static constexpr int kPer = YT == T_F32 ? 4 : 8, kLanes = 64 / kPer, kRows = 64 / kLanes, kAccesses = 16 / kRows;
};
// STREAM: past the caches
template <int YT, bool STREAM>
__device__ __forceinline__ u4_t load_cols(const void* base, size_t at) {
  const u4_t* const v = reinterpret_cast<const u4_t*>(static_cast<const char*>(base) + at * (YT == T_F32 ? 4 : 2));
  if constexpr (STREAM) return __builtin_nontemporal_load(v);
  return *v;
}
template <int YT, bool STREAM>
__device__ __forceinline__ void store_cols(void* base, size_t at, u4_t v) {
  u4_t* const to = reinterpret_cast<u4_t*>(static_cast<char*>(base) + at * (YT == T_F32 ? 4 : 2));
  if constexpr (STREAM)
    __builtin_nontemporal_store(v, to);
  else
    *to = v;
}
// v + back * d for an access's columns, rounded once to the type
template <int YT>
__device__ __forceinline__ u4_t add_cols(u4_t v, const float* d, float back) {
  u4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t bits = v[i];  // a vector's element is no object of its own to a bit cast
    if constexpr (YT == T_F32) {
      const float sum = __builtin_fmaf(back, d[i], __builtin_bit_cast(float, bits));
      r[i] = __builtin_bit_cast(uint32_t, sum);
    } else if constexpr (YT == T_F16) {
      const h2_t y = as_h2(bits);
      const float lo = __builtin_fmaf(back, d[2 * i], (float)y[0]), hi = __builtin_fmaf(back, d[2 * i + 1], (float)y[1]);
      r[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)lo) | (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)hi) << 16;
    } else {
      const float lo = __builtin_fmaf(back, d[2 * i], __builtin_bit_cast(float, bits << 16));
      const float hi = __builtin_fmaf(back, d[2 * i + 1], __builtin_bit_cast(float, bits & 0xFFFF0000u));
      r[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)lo) | (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16;
    }
  }
  return r;
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

template <int ACT, int YT>
constexpr int parts_of() { return ACT == ACT_BF16 && YT == T_F32 ? 3 : 2; }
// halves between a row's parts in LDS: eight more than its ranks, so that the 16-byte reads of
// eight rows fall in different banks
constexpr int part_stride(int RS) { return 32 * RS + 8; }

// floats between rows of a wave's 16 x 64 product in LDS
constexpr int kTurnStride = 68;
constexpr size_t turn_bytes() { return 16 * kTurnStride * 4; }

// RS: 32-rank steps. TALL: tiles of up to 64 rows, one strip a wave, whose y is all in flight before
// t is split; else tiles of 16 rows, several strips, the next one's B and y in flight.
// RT > 0: t is formed here too, 16 RT ranks by every workgroup of a tile for itself (no slices, one launch).
// STREAM (of TALL): y and out past the caches.
template <int ACT, int YT, int RS, bool TALL, int RT = 0, bool STREAM = false>
__global__ __launch_bounds__(64 * expand_waves(RT > 0)) void expand_kernel(LoraParams p) {
  typedef typename ActT<ACT>::type AT;
  constexpr bool ONE = RT > 0;
  typedef Cols<YT> Y;
  constexpr int PARTS = parts_of<ACT, YT>(), STRIDE = part_stride(RS), NH = Y::kAccesses, W = expand_waves(ONE);
  extern __shared__ __attribute__((aligned(16))) uint16_t tp[];  // [tile rows][PARTS][STRIDE], then the waves' own
  __shared__ int rows_of[kTileMax];
  __shared__ float backs[kTileMax];
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // consecutive workgroups take a tile's columns: neighbours in memory, and each XCD's share of a
  // matrix B is an eighth
  const int tile = blockIdx.x / p.col_groups, cg = blockIdx.x - tile * p.col_groups;
  int rows, e;
  if (!find_tile(p, tile, rows_of, rows, e)) return;
  // this wave's strips of 64 columns: n_first, n_first + step, ... below n_end
  constexpr int step = 64 * W;
  const int n_first = cg * p.strips * step + wave * 64;
  const int n_end = min(p.N, (cg + 1) * p.strips * step);
  const int yrow = lane / Y::kLanes, ycol = (lane % Y::kLanes) * Y::kPer;  // N is a multiple of 16: an access is all in or out
  if (e >= p.L) {  // no adapter: out is y
    if (p.out == p.y) return;
    __syncthreads();
    for (int n0 = n_first; n0 < n_end; n0 += step)
      for (int m = yrow; m < rows; m += Y::kRows) {
        const size_t at = (size_t)rows_of[m] * p.N + n0 + ycol;
        if (n0 + ycol < p.N) store_cols<YT, STREAM>(p.out, at, load_cols<YT, STREAM>(p.y, at));
      }
    return;
  }
  char* const own = reinterpret_cast<char*>(tp) + (size_t)p.tile_rows * PARTS * STRIDE * 2;
  float* const turn = reinterpret_cast<float*>(own + wave * turn_bytes());
  const uint16_t* const b = p.b + (size_t)e * p.N * p.R;
  auto load_b = [&](u4_t (&v)[4][RS], int n0) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = min(n0 + 16 * q + (lane & 15), p.N - 1);
#pragma unroll
      for (int rs = 0; rs < RS; ++rs) {
        const int r = 32 * rs + 8 * g;  // R is a multiple of 8
        v[q][rs] = r < p.R ? *reinterpret_cast<const u4_t*>(b + (size_t)n * p.R + r) : u4_t{0, 0, 0, 0};
      }
    }
  };
  auto load_y = [&](u4_t (&v)[NH], int n0, int m0) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < NH; ++h)
      if (n0 + ycol < p.N)
        v[h] = load_cols<YT, STREAM>(p.y, (size_t)rows_of[min(m0 + Y::kRows * h + yrow, rows - 1)] * p.N + n0 + ycol);
  };
  constexpr int TILES = TALL ? kTileMax / 16 : 1;
  u4_t bv[4][RS], yv[TILES][NH];
  load_b(bv, n_first);
  const float scaling = p.scaling[e];
  __syncthreads();  // rows_of
#pragma unroll
  for (int k = 0; k < TILES; ++k)
    if (16 * k < rows) load_y(yv[k], n_first, 16 * k);
  __shared__ __attribute__((aligned(16))) float red[ONE ? kShrinkWaves / 2 * RT * 256 : 1];
  if constexpr (ONE) shrink_tile<ACT, ONE ? RT : 1>(p, rows_of, rows, e, 0, 0, p.K / 32, red);
  // the rows' t: 4 RS threads a row, eight ranks each
  constexpr int C = 4 * RS;
  for (int q = threadIdx.x; q < ((rows + 15) & ~15) * C; q += 64 * W) {
    const int row = q / C, r = 8 * (q - row * C);
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = 0.f;
    if constexpr (ONE) {
      if (r < p.R)
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = shrink_sum<ONE ? RT : 1>(red, row, r + i);
    } else if (r < p.R) {
      const float* src = p.part + (size_t)rows_of[min(row, rows - 1)] * p.R + r;
      const size_t next = (size_t)p.M * p.R;
      for (int s0 = 0; s0 < p.slices; s0 += 4) {
        f4_t lo[4], hi[4];  // four slices' loads in flight
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float* v = src + min(s0 + s, p.slices - 1) * next;
          lo[s] = *reinterpret_cast<const f4_t*>(v);
          hi[s] = *reinterpret_cast<const f4_t*>(v + 4);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            t[i] += s0 + s < p.slices ? lo[s][i] : 0.f;
            t[4 + i] += s0 + s < p.slices ? hi[s][i] : 0.f;
          }
      }
    }
    float back = scaling;
    if constexpr (ACT == ACT_F16) {
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(t[i]));
#pragma unroll
      for (int o = 1; o < C; o <<= 1) big = fmaxf(big, __shfl_xor(big, o));
      // 2^-e of the row's largest value, from its exponent bits (kept off the ends of the range)
      const int ex = min(max((int)(__builtin_bit_cast(uint32_t, big) >> 23), 27), 227);
      const float down = __builtin_bit_cast(float, (uint32_t)(254 - ex) << 23);
      back *= __builtin_bit_cast(float, (uint32_t)ex << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] *= down;
    }
    AT part[PARTS];
    split8<ACT, PARTS>(t, part);
#pragma unroll
    for (int s = 0; s < PARTS; ++s)
      *reinterpret_cast<u4_t*>(tp + (row * PARTS + s) * STRIDE + r) = __builtin_bit_cast(u4_t, part[s]);
    if (r == 0) backs[row] = back;
  }
  __syncthreads();
  // one 16 x 64 tile: the product turned through LDS, so that y and out are accessed by whole runs of a
  // row (lane l holds row l%16 and columns 16 q + 4 (l/16) .. + 3 of it; straight from there, sixteen lanes would
  // access sixteen rows)
  auto add_tile = [&](const u4_t (&y)[NH], int n0, int m0) __attribute__((always_inline)) {
    f4_t acc[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int rs = 0; rs < RS; ++rs)
#pragma unroll
      for (int s = 0; s < PARTS; ++s) {
        const u4_t t = *reinterpret_cast<const u4_t*>(tp + ((m0 + (lane & 15)) * PARTS + s) * STRIDE + 32 * rs + 8 * g);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[q] = mfma16(__builtin_bit_cast(AT, bv[q][rs]), __builtin_bit_cast(AT, t), acc[q]);
      }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<f4_t*>(turn + (lane & 15) * kTurnStride + 16 * q + 4 * g) = acc[q];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const int r = Y::kRows * h + yrow, m = m0 + r;
      float d[Y::kPer];
#pragma unroll
      for (int i = 0; i < Y::kPer; i += 4)
        *reinterpret_cast<f4_t*>(d + i) = *reinterpret_cast<const f4_t*>(turn + r * kTurnStride + ycol + i);
      if (m < rows && n0 + ycol < p.N)
        store_cols<YT, STREAM>(p.out, (size_t)rows_of[m] * p.N + n0 + ycol, add_cols<YT>(y[h], d, backs[m]));
    }
    __builtin_amdgcn_wave_barrier();
  };
  // One strip; with MORE the next strip's B and y load meanwhile. Loads under a branch would make the
  // compiler wait for all that are in flight, so the last strip is a pass of its own.
  auto strip = [&](int n0, auto more) __attribute__((always_inline)) {
    constexpr bool MORE = decltype(more)::value, AHEAD = MORE && RS <= 2;
    u4_t next[NH], bn[4][RS];
    if constexpr (AHEAD) load_b(bn, n0 + step);
    if constexpr (MORE) load_y(next, n0 + step, 0);
#pragma unroll
    for (int k = 0; k < TILES; ++k)
      if (16 * k < rows) add_tile(yv[k], n0, 16 * k);
    if constexpr (MORE) {
#pragma unroll
      for (int h = 0; h < NH; ++h) yv[0][h] = next[h];
      if constexpr (AHEAD) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int rs = 0; rs < RS; ++rs) bv[q][rs] = bn[q][rs];
      } else {
        load_b(bv, n0 + step);
      }
    }
  };
  int n0 = n_first;
  if constexpr (!TALL)
    for (; n0 + step < n_end; n0 += step) strip(n0, std::true_type{});
  if (n0 < n_end) strip(n0, std::false_type{});
}

// tiles found by the workgroups themselves: few rows, no plan
bool self_tiles(int M, bool planned) { return !planned && M <= kSelfRows; }

struct LoraGeometry {
  int list;  // tile list
  int slices, steps, strips;
  bool one;  // both products in one launch
};

LoraGeometry lora_geometry(int M, int K, int N, int L, int R, bool self) {
  LoraGeometry g;
  // One launch where every workgroup can afford its tile's t: an adapter's A of at most 256 KiB, read by all the
  // workgroups of a tile of 512 columns (from L2), 16 MiB of such reads in all.
  g.one = self && R <= kRankChunk && (long long)R * K <= (1 << 17) &&
          (long long)M * ceil_div(N, 64 * expand_waves(true)) * R * K <= (1 << 23);
  // by the adapters that can have rows: with many loaded and few in use the mean is low, and 16-row tiles are taken
  // for what 64-row tiles would do (4096 rows of 9 adapters, 8192x8192 rank 64: 62 us with 9 loaded, 86 with 64, 128 with 128)
  const int groups = L < M ? L : M;
  g.list = M / (groups > 0 ? groups : 1) >= 48 ? 2 : 0;
  // tiles to expect: full ones, and about one part-filled for every second adapter
  const long long tiles = M / kTileRows[g.list] + (groups + 1) / 2;
  const long long cus = device_cu_count();
  // slices of K until the tiles fill the compute units, at least four steps a wave
  const int steps = K / 32;
  int slices = (int)(cus / ((tiles > 0 ? tiles : 1) * ceil_div(R, kRankChunk)));
  const int most = steps / (4 * kShrinkWaves);
  if (slices > most) slices = most;
  if (slices > kMaxSlices) slices = kMaxSlices;
  if (slices < 1) slices = 1;
  g.steps = ceil_div(ceil_div(steps, slices), kSetSteps) * kSetSteps;  // whole sets, whole 128-column blocks
  g.slices = ceil_div(steps, g.steps);
  // strips per wave (each saves the others' search for rows and splitting of t) while two workgroups
  // a compute unit are left
  const long long wgs = tiles * ceil_div(N, 64 * expand_waves(false));
  g.strips = g.list ? 1 : (int)(wgs / (2 * cus));
  if (g.strips > 8) g.strips = 8;
  if (g.strips < 1 || g.one) g.strips = 1;
  return g;
}

template <int ACT>
void launch_shrink(const LoraParams& p, bool tall, dim3 grid, hipStream_t s) {
  if (tall) {
    const dim3 block(64 * kTallWaves);
    if (p.R <= 16)
      hipLaunchKernelGGL((shrink_tall_kernel<ACT, 1>), grid, block, kStages * tall_slot<1>() * 2, s, p);
    else if (p.R <= 32)
      hipLaunchKernelGGL((shrink_tall_kernel<ACT, 2>), grid, block, kStages * tall_slot<2>() * 2, s, p);
    else
      hipLaunchKernelGGL((shrink_tall_kernel<ACT, 4>), grid, block, kStages * tall_slot<4>() * 2, s, p);
    return;
  }
  const dim3 block(64 * kShrinkWaves);
  const size_t lds = (size_t)kShrinkWaves / 2 * 256 * 4;  // per rank tile
  if (p.R <= 16)
    hipLaunchKernelGGL((shrink_kernel<ACT, 1>), grid, block, lds, s, p);
  else if (p.R <= 32)
    hipLaunchKernelGGL((shrink_kernel<ACT, 2>), grid, block, 2 * lds, s, p);
  else
    hipLaunchKernelGGL((shrink_kernel<ACT, 4>), grid, block, 4 * lds, s, p);
}

template <int ACT, int YT>
constexpr size_t expand_lds(int tile_rows, int RS, bool one) {
  return (size_t)tile_rows * parts_of<ACT, YT>() * part_stride(RS) * 2 + expand_waves(one) * turn_bytes();
}

template <int ACT, int YT, int RS>
void launch_expand_rs(const LoraParams& p, dim3 grid, hipStream_t s) {
  const dim3 block(64 * expand_waves(false));
  const size_t lds = expand_lds<ACT, YT>(p.tile_rows, RS, false);
  if (p.tile_rows > 16 && (size_t)p.M * p.N * (YT == T_F32 ? 4 : 2) >= kStreamBytes)
    hipLaunchKernelGGL((expand_kernel<ACT, YT, RS, true, 0, true>), grid, block, lds, s, p);
  else if (p.tile_rows > 16)
    hipLaunchKernelGGL((expand_kernel<ACT, YT, RS, true>), grid, block, lds, s, p);
  else
    hipLaunchKernelGGL((expand_kernel<ACT, YT, RS, false>), grid, block, lds, s, p);
}

template <int ACT, int YT>
void launch_one(const LoraParams& p, dim3 grid, hipStream_t s) {
  const dim3 block(64 * expand_waves(true));
  const size_t lds = expand_lds<ACT, YT>(16, p.R <= 32 ? 1 : 2, true);
  if (p.R <= 16)
    hipLaunchKernelGGL((expand_kernel<ACT, YT, 1, false, 1>), grid, block, lds, s, p);
  else if (p.R <= 32)
    hipLaunchKernelGGL((expand_kernel<ACT, YT, 1, false, 2>), grid, block, lds, s, p);
  else
    hipLaunchKernelGGL((expand_kernel<ACT, YT, 2, false, 4>), grid, block, lds, s, p);
}

template <int ACT, int YT>
void launch_expand(const LoraParams& p, dim3 grid, hipStream_t s) {
  if (p.R <= 32)
    launch_expand_rs<ACT, YT, 1>(p, grid, s);
  else if (p.R <= 64)
    launch_expand_rs<ACT, YT, 2>(p, grid, s);
  else if (p.R <= 128)
    launch_expand_rs<ACT, YT, 4>(p, grid, s);
  else
    launch_expand_rs<ACT, YT, 8>(p, grid, s);
}

}  // namespace

bool lora_fits(int M, int K, int N, int L, int R) {
  if (M > kMaxSlots) return false;
  // the last block of K and the last workgroup's columns (up to eight strips of four waves) end past them
  if (K > INT_MAX - 127 || N > INT_MAX - 2047) return false;
  for (int planned = 0; planned < 2; ++planned) {
    const bool self = self_tiles(M, planned != 0);
    const LoraGeometry g = lora_geometry(M, K, N, L, R, self);
    const long long tiles = self ? M : tile_bound(M, L, g.list);
    const long long first = tiles * g.slices * 64 * kShrinkWaves;
    const long long second = tiles * ceil_div(N, 64 * expand_waves(g.one) * g.strips) * 64 * expand_waves(g.one);
    if (first >= (1LL << 32) || second >= (1LL << 32)) return false;
  }
  return true;
}

size_t lora_workspace_bytes(int M, int K, int N, int L, int R, bool planned) {
  const bool self = self_tiles(M, planned);
  const LoraGeometry g = lora_geometry(M, K, N, L, R, self);
  if (g.one) return 0;
  const size_t plan = planned || self ? 0 : align256((size_t)route_layout(M, 1, L).words * 4);
  return plan + align256((size_t)g.slices * M * R * 4);
}

hipError_t launch_lora(const LoraArgs& a) {
  const bool self = self_tiles(a.M, a.plan != nullptr);
  LoraGeometry g = lora_geometry(a.M, a.K, a.N, a.L, a.R, self);
  char* ws = static_cast<char*>(a.workspace);
  LoraParams p;
  p.ids = nullptr;
  p.groups = GroupTiles{};
  int tiles = a.M;  // of a launch
  if (self) {
    p.ids = a.ids;
    g.list = 0;
  } else {
    const RouteLayout r = route_layout(a.M, 1, a.L);
    p.groups.plan = a.plan;
    if (!a.plan) {
      int32_t* plan = reinterpret_cast<int32_t*>(ws);
      ws += align256((size_t)r.words * 4);
      const hipError_t e = launch_route(a.ids, r, plan, a.stream);
      if (e != hipSuccess) return e;
      p.groups.plan = plan;
    }
    p.groups.E = r.E;
    p.groups.token = r.token;
    p.groups.list = r.tiles[g.list];
    p.groups.bound = tiles = tile_bound(r.S, r.E, g.list);
  }
  p.x = static_cast<const uint16_t*>(a.x);
  p.a = static_cast<const uint16_t*>(a.lora_a);
  p.b = static_cast<const uint16_t*>(a.lora_b);
  p.y = a.y;
  p.out = a.out;
  p.scaling = a.scaling;
  p.part = reinterpret_cast<float*>(ws);
  p.M = a.M;
  p.K = a.K;
  p.N = a.N;
  p.L = a.L;
  p.R = a.R;
  p.slices = g.slices;
  p.steps = g.steps;
  p.tile_rows = kTileRows[g.list];
  p.strips = g.strips;
  p.col_groups = ceil_div(a.N, 64 * expand_waves(g.one) * g.strips);
  const dim3 egrid(tiles * p.col_groups);
  if (g.one) {
    if (a.act == ACT_F16)
      a.ydtype == T_F32 ? launch_one<ACT_F16, T_F32>(p, egrid, a.stream) : launch_one<ACT_F16, T_F16>(p, egrid, a.stream);
    else
      a.ydtype == T_F32 ? launch_one<ACT_BF16, T_F32>(p, egrid, a.stream) : launch_one<ACT_BF16, T_BF16>(p, egrid, a.stream);
    return hipGetLastError();
  }
  const dim3 sgrid(tiles * g.slices, ceil_div(a.R, kRankChunk));
  if (a.act == ACT_F16)
    launch_shrink<ACT_F16>(p, g.list != 0, sgrid, a.stream);
  else
    launch_shrink<ACT_BF16>(p, g.list != 0, sgrid, a.stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.act == ACT_F16)
    a.ydtype == T_F32 ? launch_expand<ACT_F16, T_F32>(p, egrid, a.stream) : launch_expand<ACT_F16, T_F16>(p, egrid, a.stream);
  else
    a.ydtype == T_F32 ? launch_expand<ACT_BF16, T_F32>(p, egrid, a.stream) : launch_expand<ACT_BF16, T_BF16>(p, egrid, a.stream);
  return hipGetLastError();
}

}  // namespace w4a16
