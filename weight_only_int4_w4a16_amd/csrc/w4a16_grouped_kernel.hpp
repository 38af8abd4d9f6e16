// w4a16_grouped_kernel.hpp - W4A16 products of sorted rows with their groups' weights, few rows
// a group: a template over the formats, instantiated per activation type in
// w4a16_grouped_{f16,bf16}.hip.
//
//   out[p] = x[row(p)] * W_hat[e]  for p in [offsets[e], offsets[e + 1])
//
// With a few rows per expert the call is bound by the weight bytes of the experts that have rows:
// each must cross HBM once, at full rate, whichever experts were chosen, and nothing of the
// choice is known on the host. So the grid covers the most row tiles the slots can make
// (w4a16_route's list of 16-row tiles) and a workgroup takes its group and rows from the list;
// those past its end leave at once.
//
// Work split. A workgroup owns 16 MT rows by four 16-column strips over all of K, its waves take
// contiguous k-block slices (as in the decode kernel) and their partial tiles are added through
// LDS in wave order. Row tiles of one group and column tile are neighbours on one XCD, so a
// second tile of the same group finds the codes in that L2.
//
// A tile has up to MT sixteens of rows, and the kernel a whole body for each number of them: the
// workgroup takes the one that its rows need, so that a part-filled tile costs no MFMAs, fragment
// reads or sums for rows that it has not (8 experts of 14336x4096 at a mean of 8 rows in 64-row tiles
// 61 -> 46 us, of 4096x14336 at 32 rows 91 -> 71). Branches per sixteen inside one body cost registers for
// all paths at once, and spilled.
//
// Operands. v_mfma_f32_16x16x32: word j of a lane's 16-byte chunk of a packed block is its B
// operand for k-step j. The A operand's sixteen rows go through LDS: read from memory in its
// layout, sixteen lanes at a time would touch sixteen rows' cache lines (a 1 KiB load then
// takes 64 cycles of the compute unit's address unit instead of 16), so each wave copies its
// block of x, four rows of 256 bytes per instruction and only those rows that the tile has,
// straight into a slot of its own. The slot is read into registers before the next block's copy
// and codes are issued, which then travel while this block is multiplied: no barriers, one slot.
// Row r of a slot holds its sixteen 16-byte chunks at positions c ^ (r % 16), so that a
// fragment read touches every bank once.
//
// bf16 weights. The vector instructions that form W_hat, not HBM, would bound the call (21 per
// eight weights at the decode kernels' way), so (q - z) s is one fma of the biased code: with v = 1024 + q
// (exact in fp16), fma(v, s, -(1024 + z) s) is exact: both products have at most 19 significant
// bits. 17 instructions. The constants cost two multiplications per strip and scale group.
#pragma once

#include <type_traits>

#include "w4a16_device.hpp"
#include "w4a16_routed.hpp"

namespace w4a16 {
namespace grouped {

enum Fmt { FMT_ASYM = 0, FMT_SYM = 1, FMT_NF4 = 2 };

template <int ACT>
struct ActT;
template <>
struct ActT<ACT_F16> { typedef h8_t type; };
template <>
struct ActT<ACT_BF16> { typedef b8_t type; };

struct GroupedParams {
  const uint16_t* x;
  GroupTiles groups;
  int K, N;
  const u4_t* packed;
  const uint16_t* scales;
  const uint32_t* qzeros;
  const uint16_t* codebook;
  void* out;
  int out_dtype;
  int KC, NT, NG, half;
  int slice;  // k-blocks per wave
  int col_tiles;
};

// workgroup -> tile, so that consecutive tiles run on the same XCD
__device__ __forceinline__ int tile_of(int b, int G) {
  const int q = G >> 3, r = G & 7, x = b & 7;
  return x * q + (x < r ? x : r) + (b >> 3);
}

constexpr int kStrips = 4;
constexpr int kWaves = 4;

// (q - z) s of one packed word in bf16 by one fma per weight; c1024 = -(1024 + z) s,
// c64 = -(64 + z) s
__device__ __forceinline__ b8_t dequant_word_bf16_fma(uint32_t w, float s, float c1024, float c64) {
  const uint32_t w8 = w >> 8;
  const h2_t d[4] = {as_h2(and_or(w, 0x000F000Fu, 0x64006400u)), as_h2(and_or(w, 0x00F000F0u, 0x54005400u)),
                     as_h2(and_or(w8, 0x000F000Fu, 0x64006400u)), as_h2(and_or(w8, 0x00F000F0u, 0x54005400u))};
  b8_t r;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float c = p & 1 ? c64 : c1024;
    r[2 * p] = (__bf16)__builtin_fmaf((float)d[p][0], s, c);
    r[2 * p + 1] = (__bf16)__builtin_fmaf((float)d[p][1], s, c);
  }
  return r;
}

// What the words of one strip and scale group share
struct GroupScale {
  uint32_t raw, z;
  float s, c1024, c64;
};
template <int ACT, int FMT>
__device__ __forceinline__ GroupScale group_scale(uint32_t raw, uint32_t z) {
  GroupScale g;
  g.raw = raw;
  g.z = z;
  if constexpr (FMT == FMT_NF4) {
    g.s = (float)__builtin_bit_cast(_Float16, (uint16_t)raw);
  } else if constexpr (ACT == ACT_BF16) {
    g.s = __builtin_bit_cast(float, raw << 16);
    g.c1024 = -((float)(1024u + z) * g.s);
    g.c64 = -((float)(64u + z) * g.s);
  }
  return g;
}

template <int ACT, int FMT>
__device__ __forceinline__ typename ActT<ACT>::type dequant_word(uint32_t w, const GroupScale& g, const uint32_t* ptab) {
  if constexpr (FMT == FMT_NF4) {
    // the levels in the pair table's order; the activations are put in the same order
    const h8_t c = nf4_levels_f16_pairs(w, ptab);
    if constexpr (ACT == ACT_F16) {
      const h2_t a2 = as_h2(g.raw * 0x00010001u);
      h8_t r;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const h2_t d = h2_t{c[2 * p], c[2 * p + 1]} * a2;
        r[2 * p] = d[0];
        r[2 * p + 1] = d[1];
      }
      return r;
    } else {
      // c * a is exact in fp32; as fma(c, a, +0) the multiplication takes the fp16 level as it is
      b8_t r;
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = (__bf16)__builtin_fmaf((float)c[i], g.s, 0.0f);
      return r;
    }
  } else if constexpr (ACT == ACT_F16) {
    return dequant_word_f16(w, make_zero_f16(g.z), as_h2(g.raw * 0x00010001u));
  } else {
    return dequant_word_bf16_fma(w, g.s, g.c1024, g.c64);
  }
}

// f(n), n a constant: the sixteens of rows that a tile of up to MT of them has
template <int MT, typename F>
__device__ __forceinline__ void for_active(int rows, F&& f) {
  if constexpr (MT == 1) {
    f(std::integral_constant<int, 1>{});
  } else {
    if (rows <= 16 * (MT - 1))
      for_active<MT - 1>(rows, f);
    else
      f(std::integral_constant<int, MT>{});
  }
}

constexpr int slot_halves(int MT) { return 16 * MT * 128; }
// floats between rows of a partial tile: four rows written at once then fall in different banks
constexpr int kRedStride = 16 * kStrips + 4;
// a wave's LDS: its slot, later its partial tile
constexpr size_t wave_lds(int MT) {
  return (size_t)16 * MT * kRedStride * 4 > (size_t)slot_halves(MT) * 2 ? (size_t)16 * MT * kRedStride * 4 : (size_t)slot_halves(MT) * 2;
}

// four consecutive elements of the output
__device__ __forceinline__ void store_quad(void* out, size_t at, f4_t v, int out_dtype) {
  if (out_dtype == 2) {
    *reinterpret_cast<f4_t*>(static_cast<float*>(out) + at) = v;
    return;
  }
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = v[i];
    h[i] = out_dtype == 0 ? __builtin_bit_cast(uint16_t, (_Float16)f) : __builtin_bit_cast(uint16_t, (__bf16)f);
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
      uint2{(uint32_t)h[0] | (uint32_t)h[1] << 16, (uint32_t)h[2] | (uint32_t)h[3] << 16};
}

// every load of the wave has landed
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xF << 8));
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
}
// and every LDS read
__device__ __forceinline__ void wait_lds() {
  __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
}

// Waves a SIMD is to hold: as many as leave the registers unspilled (scale groups of 32 hold
// more of them)
constexpr int waves_per_simd(int MT, int GPC) { return (MT == 1 ? 4 : MT == 2 ? 3 : 2) - (GPC == 4 ? 1 : 0); }

// GLU: the first two strips are gate strips, the others the matching up strips, and the output
// is h = SiLU(gate) * up, [S][N / 2].
template <int ACT, int GPC, int FMT, int MT, bool GLU, int W>
__device__ __forceinline__ void grouped_tile(const GroupedParams& p, uint16_t* lds, uint32_t* ptab, int tn, int e,
                                             int p0, int rows) {
  typedef typename ActT<ACT>::type AT;
  constexpr bool ZEROS = FMT == FMT_ASYM;
  constexpr int SW = kStrips, OS = GLU ? SW / 2 : SW;  // strips, output strips

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = p.K, N = p.N, KC = p.KC;
  const int width = GLU ? N >> 1 : N;  // of an output row
  const int shift = 4 * (lane & 7);
  uint16_t* const slot = lds + wave * (wave_lds(MT) / 2);
  const int kc0 = min(wave * p.slice, KC), kc1 = min(kc0 + p.slice, KC);
  const int ocol0 = tn * OS * 16, ocols = min(OS * 16, width - ocol0);
  struct Codes {
    u4_t b[SW];
    uint32_t s[SW][GPC], z[SW][GPC];
  };
  const u4_t* const wbase = p.packed + (size_t)e * p.NT * KC * 64;
  const uint16_t* const sbase = p.scales + (size_t)e * p.NG * N;
  const uint32_t* const zbase = ZEROS ? p.qzeros + (size_t)e * p.NG * (N >> 3) : nullptr;
  const __amdgpu_buffer_rsrc_t srs = make_rsrc(sbase, (uint32_t)p.NG * N * 2);
  const __amdgpu_buffer_rsrc_t zrs = make_rsrc(ZEROS ? (const void*)zbase : (const void*)sbase, (uint32_t)p.NG * (N >> 3) * 4);
  // strip s of the tile, clamped in bounds for loads (never stored past the last one)
  auto strip = [&](int s) __attribute__((always_inline)) {
    return GLU ? min(tn * OS + (s < OS ? s : s - OS), p.half - 1) + (s < OS ? 0 : p.half) : min(tn * SW + s, p.NT - 1);
  };
  auto load_codes = [&](Codes& R, int kc) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < SW; ++s)
      R.b[s] = __builtin_nontemporal_load(wbase + ((size_t)strip(s) * KC + kc) * 64 + lane);
#pragma unroll
    for (int s = 0; s < SW; ++s) {
#pragma unroll
      for (int gi = 0; gi < GPC; ++gi) {
        const int g = min(kc * GPC + gi, p.NG - 1);
        R.s[s][gi] = __builtin_amdgcn_raw_buffer_load_b16(srs, (lane & 15) * 2, (g * N + strip(s) * 16) * 2, 0);
        if constexpr (ZEROS)
          R.z[s][gi] = __builtin_amdgcn_raw_buffer_load_b32(zrs, ((lane & 15) >> 3) * 4, (g * (N >> 3) + strip(s) * 2) * 4, 0);
      }
    }
  };
  Codes R;
  if (kc0 < kc1) load_codes(R, kc0);
  // The copies of x: instruction j of a block covers rows 4j .. 4j + 3, lane l row 4j + l/16 and
  // position l%16, which holds chunk (l%16) ^ (row%16). Chunks past a ragged K read out of range (zeros).
  const __amdgpu_buffer_rsrc_t xrs = p.groups.tokens
      ? make_rsrc(p.x, (uint32_t)p.groups.tokens * (uint32_t)K * 2u)
      : make_rsrc(p.x + (size_t)p0 * K, (uint32_t)rows * (uint32_t)K * 2u);
  // lane l: the row of x of the tile's row l (its last one past the end)
  int src = min(lane, rows - 1);
  if (p.groups.tokens) src = p.groups.plan[p.groups.token + p0 + src];
  uint32_t xoff[4 * MT];
#pragma unroll
  for (int j = 0; j < 4 * MT; ++j) {
    const int row = 4 * j + (lane >> 4);
    xoff[j] = ((uint32_t)__shfl(src, row) * (uint32_t)K + ((lane & 15) ^ (row & 15)) * 8) * 2u;
  }
  auto copy_x = [&](int kc) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4 * MT; ++j) {
      if (j && 4 * j >= rows) break;
      const int chunk = (lane & 15) ^ ((4 * j + (lane >> 4)) & 15);
      buffer_copy16_to_lds(xrs, kc * 128 + chunk * 8 < K ? xoff[j] : kOutOfRange, kc * 256, slot + j * 512);
    }
  };
  if constexpr (FMT == FMT_NF4) {
    nf4_pair_table_fill(ptab, p.codebook);
    __syncthreads();
  }
  f4_t acc[MT][SW];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int s = 0; s < SW; ++s) acc[mt][s] = f4_t{0.f, 0.f, 0.f, 0.f};
  if (kc0 < kc1) copy_x(kc0);
  for (int kc = kc0; kc < kc1; ++kc) {
    wait_loads();  // this block's codes and copies
    u4_t a[4][MT];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int row = 16 * mt + (lane & 15);
        a[j][mt] = *reinterpret_cast<const u4_t*>(slot + row * 128 + (((4 * j + (lane >> 4)) ^ (row & 15)) * 8));
      }
    wait_lds();  // the slot is free
    const Codes C = R;
    if (kc + 1 < kc1) {
      load_codes(R, kc + 1);
      copy_x(kc + 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (FMT == FMT_NF4) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) a[j][mt] = act8_to_pair_order(a[j][mt]);
    }
    GroupScale gs[SW][GPC];
#pragma unroll
    for (int s = 0; s < SW; ++s)
#pragma unroll
      for (int gi = 0; gi < GPC; ++gi)
        gs[s][gi] = group_scale<ACT, FMT>(C.s[s][gi], ZEROS ? (C.z[s][gi] >> shift) & 0xFu : 8u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kc * 128 + 32 * j >= K) break;
#pragma unroll
      for (int s = 0; s < SW; ++s) {
        const AT w = dequant_word<ACT, FMT>(C.b[s][j], gs[s][j * GPC / 4], ptab);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[mt][s] = mfma16(__builtin_bit_cast(AT, a[j][mt]), w, acc[mt][s]);
      }
    }
  }
  // The partial tiles over the waves' slots (each wave is done with its own), row by row: lane l
  // holds column l%16 of each strip and rows 16 mt + 4 (l/16) + i, i < 4
  float* const red = reinterpret_cast<float*>(lds);
  constexpr int TILE = wave_lds(MT) / 4;  // floats per wave
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int s = 0; s < SW; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[wave * TILE + (16 * mt + 4 * (lane >> 4) + i) * kRedStride + 16 * s + (lane & 15)] = acc[mt][s][i];
  __syncthreads();
  constexpr int QUADS = OS * 4;  // of columns in a row
  for (int q = threadIdx.x; q < rows * QUADS; q += 64 * W) {
    const int r = q / QUADS, c = 4 * (q % QUADS);
    if (c >= ocols) continue;  // whole quads: the width is a multiple of 16
    const float* const at = red + r * kRedStride + c;
    f4_t v = *reinterpret_cast<const f4_t*>(at), u = {0.f, 0.f, 0.f, 0.f};
    if constexpr (GLU) u = *reinterpret_cast<const f4_t*>(at + OS * 16);
#pragma unroll
    for (int w = 1; w < W; ++w) {
      v += *reinterpret_cast<const f4_t*>(at + w * TILE);
      if constexpr (GLU) u += *reinterpret_cast<const f4_t*>(at + w * TILE + OS * 16);
    }
    if constexpr (GLU) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = v[i] / (1.0f + __expf(-v[i])) * u[i];
    }
    store_quad(p.out, (size_t)(p0 + r) * width + ocol0 + c, v, p.out_dtype);
  }
}

template <int ACT, int GPC, int FMT, int MT, bool GLU, int W>
__global__ __launch_bounds__(64 * W, waves_per_simd(MT, GPC)) void grouped_kernel(GroupedParams p) {
  constexpr int OS = GLU ? kStrips / 2 : kStrips;
  extern __shared__ __attribute__((aligned(16))) uint16_t lds[];  // [waves][wave_lds(MT)]
  __shared__ uint32_t ptab[FMT == FMT_NF4 ? kNf4PairEntries : 1];
  const int item = tile_of(blockIdx.x, p.groups.bound * p.col_tiles);
  const int tn = item / p.groups.bound;
  int e, p0, end;
  if (!group_tile(p.groups, item - tn * p.groups.bound, e, p0, end)) return;
  const int rows = end - p0;
  const int width = GLU ? p.N >> 1 : p.N;
  if (e >= p.groups.E) {  // the slots of no group: their rows are zeros
    zero_tile(p.out, p.out_dtype, p0, rows, width, tn * OS * 16, OS * 16);
    return;
  }
  for_active<MT>(rows, [&](auto active) __attribute__((always_inline)) {
    grouped_tile<ACT, GPC, FMT, decltype(active)::value, GLU, W>(p, lds, ptab, tn, e, p0, rows);
  });
}

// ---------------------------------------------------------------------------------------
// The same product with the waves side by side: a wave owns four strips over all of K, a
// workgroup 256 columns, and x is shared. Nothing is added between waves, a wave's fixed work is spread
// over four times the blocks, and x costs a quarter of the copies and LDS, so that more waves
// fit; but the workgroups are a quarter as many, which only fills the chip with enough tiles.
//
// Two slots of x: at block i every wave waits for its own codes and copies of it, a barrier
// makes all copies visible and frees the other slot, and block i + 1's loads go out before block i is multiplied.
// ---------------------------------------------------------------------------------------
constexpr int cols_waves_per_simd(int MT, int GPC) { return (MT == 4 ? 3 : 4) - (GPC == 4 ? 1 : 0); }
// the slots, later one 16-row partial tile a wave
constexpr size_t cols_lds(int MT) {
  const size_t ring = 2 * (size_t)slot_halves(MT) * 2, turn = (size_t)kWaves * 16 * kRedStride * 4;
  return ring > turn ? ring : turn;
}

template <int ACT, int GPC, int FMT, int MT, bool GLU>
__device__ __forceinline__ void grouped_cols_tile(const GroupedParams& p, uint16_t* lds, uint32_t* ptab, int tn, int e,
                                                  int p0, int rows) {
  typedef typename ActT<ACT>::type AT;
  constexpr bool ZEROS = FMT == FMT_ASYM;
  constexpr int SW = kStrips, OS = GLU ? SW / 2 : SW;  // strips of a wave, output strips

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = p.K, N = p.N, KC = p.KC;
  const int width = GLU ? N >> 1 : N;  // of an output row
  const int shift = 4 * (lane & 7);
  const int s0 = (tn * kWaves + wave) * OS;  // the wave's first (gate) strip
  const u4_t* const wbase = p.packed + (size_t)e * p.NT * KC * 64;
  const uint16_t* const sbase = p.scales + (size_t)e * p.NG * N;
  const uint32_t* const zbase = ZEROS ? p.qzeros + (size_t)e * p.NG * (N >> 3) : nullptr;
  const __amdgpu_buffer_rsrc_t srs = make_rsrc(sbase, (uint32_t)p.NG * N * 2);
  const __amdgpu_buffer_rsrc_t zrs = make_rsrc(ZEROS ? (const void*)zbase : (const void*)sbase, (uint32_t)p.NG * (N >> 3) * 4);
  // strip s of the wave, clamped in bounds for loads (never stored past the last one)
  auto strip = [&](int s) __attribute__((always_inline)) {
    return GLU ? min(s0 + (s < OS ? s : s - OS), p.half - 1) + (s < OS ? 0 : p.half) : min(s0 + s, p.NT - 1);
  };
  struct Codes {
    u4_t b[SW];
    uint32_t s[SW][GPC], z[SW][GPC];
  };
  auto load_codes = [&](Codes& R, int kc) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < SW; ++s)
      R.b[s] = __builtin_nontemporal_load(wbase + ((size_t)strip(s) * KC + kc) * 64 + lane);
#pragma unroll
    for (int s = 0; s < SW; ++s) {
#pragma unroll
      for (int gi = 0; gi < GPC; ++gi) {
        const int g = min(kc * GPC + gi, p.NG - 1);
        R.s[s][gi] = __builtin_amdgcn_raw_buffer_load_b16(srs, (lane & 15) * 2, (g * N + strip(s) * 16) * 2, 0);
        if constexpr (ZEROS)
          R.z[s][gi] = __builtin_amdgcn_raw_buffer_load_b32(zrs, ((lane & 15) >> 3) * 4, (g * (N >> 3) + strip(s) * 2) * 4, 0);
      }
    }
  };
  Codes R;
  load_codes(R, 0);
  // instruction i of wave w copies rows 16 i + 4 w .. + 3 of the tile, laid out as above
  const __amdgpu_buffer_rsrc_t xrs = p.groups.tokens
      ? make_rsrc(p.x, (uint32_t)p.groups.tokens * (uint32_t)K * 2u)
      : make_rsrc(p.x + (size_t)p0 * K, (uint32_t)rows * (uint32_t)K * 2u);
  const int crow = 4 * wave + (lane >> 4), cchunk = (lane & 15) ^ (crow & 15);
  uint32_t xoff[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    int src = min(16 * i + crow, rows - 1);
    if (p.groups.tokens) src = p.groups.plan[p.groups.token + p0 + src];
    xoff[i] = ((uint32_t)src * (uint32_t)K + cchunk * 8) * 2u;
  }
  auto copy_x = [&](int kc) __attribute__((always_inline)) {
    uint16_t* const slot = lds + (kc & 1) * slot_halves(MT) + wave * 512;
    const bool in = kc * 128 + cchunk * 8 < K;  // chunks past a ragged K read out of range (zeros)
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (16 * i + 4 * wave >= rows) break;
      buffer_copy16_to_lds(xrs, in ? xoff[i] : kOutOfRange, kc * 256, slot + i * 2048);
    }
  };
  copy_x(0);
  if constexpr (FMT == FMT_NF4) nf4_pair_table_fill(ptab, p.codebook);  // complete at the first barrier

  f4_t acc[MT][SW];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int s = 0; s < SW; ++s) acc[mt][s] = f4_t{0.f, 0.f, 0.f, 0.f};
  for (int kc = 0; kc < KC; ++kc) {
    wait_loads();
    __syncthreads();
    const Codes C = R;
    if (kc + 1 < KC) {
      load_codes(R, kc + 1);
      copy_x(kc + 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    const uint16_t* const slot = lds + (kc & 1) * slot_halves(MT);
    GroupScale gs[SW][GPC];
#pragma unroll
    for (int s = 0; s < SW; ++s)
#pragma unroll
      for (int gi = 0; gi < GPC; ++gi)
        gs[s][gi] = group_scale<ACT, FMT>(C.s[s][gi], ZEROS ? (C.z[s][gi] >> shift) & 0xFu : 8u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kc * 128 + 32 * j >= K) break;
      u4_t a[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int row = 16 * mt + (lane & 15);
        a[mt] = *reinterpret_cast<const u4_t*>(slot + row * 128 + (((4 * j + (lane >> 4)) ^ (row & 15)) * 8));
        if constexpr (FMT == FMT_NF4) a[mt] = act8_to_pair_order(a[mt]);
      }
#pragma unroll
      for (int s = 0; s < SW; ++s) {
        const AT w = dequant_word<ACT, FMT>(C.b[s][j], gs[s][j * GPC / 4], ptab);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[mt][s] = mfma16(__builtin_bit_cast(AT, a[mt]), w, acc[mt][s]);
      }
    }
  }
  // Each 16 rows through the wave's part of LDS and out by whole runs of a row. Lane l holds column
  // l%16 of each strip and rows 4 (l/16) + i, i < 4.
  __syncthreads();  // every wave is done with the slots
  float* const turn = reinterpret_cast<float*>(lds) + wave * 16 * kRedStride;
  constexpr int QUADS = OS * 4;  // of the wave's output columns
  const int c = 4 * (lane % QUADS), col = s0 * 16 + c;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    if (16 * mt >= rows) break;
#pragma unroll
    for (int s = 0; s < SW; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) turn[(4 * (lane >> 4) + i) * kRedStride + 16 * s + (lane & 15)] = acc[mt][s][i];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r0 = 0; r0 < 16; r0 += 64 / QUADS) {
      const int r = r0 + lane / QUADS, m = 16 * mt + r;
      const float* const at = turn + r * kRedStride + c;
      f4_t v = *reinterpret_cast<const f4_t*>(at);
      if constexpr (GLU) {
        const f4_t u = *reinterpret_cast<const f4_t*>(at + OS * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = v[i] / (1.0f + __expf(-v[i])) * u[i];
      }
      if (m < rows && col < width) store_quad(p.out, (size_t)(p0 + m) * width + col, v, p.out_dtype);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int ACT, int GPC, int FMT, int MT, bool GLU>
__global__ __launch_bounds__(64 * kWaves, cols_waves_per_simd(MT, GPC)) void grouped_cols_kernel(GroupedParams p) {
  constexpr int OS = GLU ? kStrips / 2 : kStrips;
  extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
  __shared__ uint32_t ptab[FMT == FMT_NF4 ? kNf4PairEntries : 1];
  const int item = tile_of(blockIdx.x, p.groups.bound * p.col_tiles);
  const int tn = item / p.groups.bound;
  int e, p0, end;
  if (!group_tile(p.groups, item - tn * p.groups.bound, e, p0, end)) return;
  const int rows = end - p0;
  const int width = GLU ? p.N >> 1 : p.N;
  if (e >= p.groups.E) {  // the slots of no group: their rows are zeros
    zero_tile(p.out, p.out_dtype, p0, rows, width, tn * kWaves * OS * 16, kWaves * OS * 16);
    return;
  }
  for_active<MT>(rows, [&](auto active) __attribute__((always_inline)) {
    grouped_cols_tile<ACT, GPC, FMT, decltype(active)::value, GLU>(p, lds, ptab, tn, e, p0, rows);
  });
}

struct GroupedGeometry {
  int MT;
  int waves;  // that share K; 0: waves side by side
};

template <int ACT, int GPC, int FMT, int MT>
hipError_t launch_mt(const GroupedParams& p, const GroupedGeometry& g, bool glu, hipStream_t s) {
  const dim3 grid(p.groups.bound * p.col_tiles), block(64 * kWaves);
  if constexpr (MT == 4) {
    if (g.waves == 0) {  // side by side
      if (glu)
        hipLaunchKernelGGL((grouped_cols_kernel<ACT, GPC, FMT, MT, true>), grid, block, cols_lds(MT), s, p);
      else
        hipLaunchKernelGGL((grouped_cols_kernel<ACT, GPC, FMT, MT, false>), grid, block, cols_lds(MT), s, p);
      return hipGetLastError();
    }
  }
  if constexpr (MT == 1) {
    if (g.waves == 8) {
      if (glu)
        hipLaunchKernelGGL((grouped_kernel<ACT, GPC, FMT, MT, true, 8>), grid, dim3(512), 8 * wave_lds(MT), s, p);
      else
        hipLaunchKernelGGL((grouped_kernel<ACT, GPC, FMT, MT, false, 8>), grid, dim3(512), 8 * wave_lds(MT), s, p);
      return hipGetLastError();
    }
  }
  if (glu)
    hipLaunchKernelGGL((grouped_kernel<ACT, GPC, FMT, MT, true, kWaves>), grid, block, kWaves * wave_lds(MT), s, p);
  else
    hipLaunchKernelGGL((grouped_kernel<ACT, GPC, FMT, MT, false, kWaves>), grid, block, kWaves * wave_lds(MT), s, p);
  return hipGetLastError();
}

template <int ACT, int GPC, int FMT>
hipError_t launch_fmt(const GroupedParams& p, const GroupedGeometry& g, bool glu, hipStream_t s) {
  switch (g.MT) {
    case 1: return launch_mt<ACT, GPC, FMT, 1>(p, g, glu, s);
    case 2: return launch_mt<ACT, GPC, FMT, 2>(p, g, glu, s);
    default: return launch_mt<ACT, GPC, FMT, 4>(p, g, glu, s);
  }
}

template <int ACT, int GPC>
hipError_t launch_gpc(const GroupedParams& p, const GroupedGeometry& g, bool nf4, bool glu, hipStream_t s) {
  if (nf4) return launch_fmt<ACT, GPC, FMT_NF4>(p, g, glu, s);
  if (p.qzeros) return launch_fmt<ACT, GPC, FMT_ASYM>(p, g, glu, s);
  return launch_fmt<ACT, GPC, FMT_SYM>(p, g, glu, s);
}

template <int ACT>
hipError_t launch_few(const GroupedParams& p, const GroupedGeometry& g, int group_size, bool nf4, bool glu,
                      hipStream_t s) {
  switch (group_size) {
    case 128: return launch_gpc<ACT, 1>(p, g, nf4, glu, s);
    case 64: return launch_gpc<ACT, 2>(p, g, nf4, glu, s);
    default: return launch_gpc<ACT, 4>(p, g, nf4, glu, s);
  }
}

}  // namespace grouped
}  // namespace w4a16
