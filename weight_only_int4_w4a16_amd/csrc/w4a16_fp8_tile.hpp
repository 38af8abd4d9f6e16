// w4a16_fp8_tile.hpp - products of e4m3 codes for many rows: tiles of the output by a workgroup, bound by arithmetic.
//
//   out[m][n] = sum over blocks of 128 k of  sx[kb][m] sw[n / 128][kb]  sum_k x[m][k] w[n][k]
//
// The inner sum of a block, 16 x 16 outputs at a time, comes from the matrix cores in one of two ways; it is
// multiplied by the block's two scales and added to the running sums in fp32, one fma an output and block. The
// weight is the A operand, so a lane holds four consecutive n of one row m and one scale factor serves all four.
//
// Results of 16 bits: one v_mfma_f32_16x16x128_f8f6f4. These instructions (the 16x16x32 form too) line products up with
// the largest of them and drop what lies more than about 17 bits below it: a block's sum is off by at most 2^-10 of its
// largest product, which on normal operands is 1.5e-5 of the result: an eighth of an fp16 rounding's mean, a
// hundredth of a bf16's. Independent MFMAs of this form reach 3.7 PFLOP/s on MI355X, with their fmas 3.3, with
// v_mfma_f32_32x32x64_f8f6f4 4.0 and 3.4: the smaller form needs one instruction a block instead of two that wait
// for each other, and four registers for the block's sum instead of sixteen.
//
// Results of 32 bits, and h that is quantized here (EXACT): every e4m3 is an fp16 number, so the fragments are
// widened in registers (one instruction for two codes) and four v_mfma_f32_16x16x32_f16 sum a block in full
// fp32 (1e-8 of the result on the same operands), at half the rate: 1.7 PFLOP/s with the fmas.
//
// Rates reached: 2048 rows of 8192x28672 in bf16 416 to 430 us, 2.3 PFLOP/s, in fp32 800, 1.2 PFLOP/s. With codes of all
// zeros the first takes 324 us: the chip lowers its clock under full load, so that past this point a product's time is its
// energy, and fewer waits do not shorten it (the widened product by v_mfma_f32_32x32x16_f16: 14 % fewer cycles, 1 % less
// time; v_mfma_f32_32x32x64_f8f6f4, with half the operand reads: 6 % more). The blocks' scales are 50 us of the first.
//
// Tiles. Both operands go from memory straight to LDS (buffer_load_dwordx4 ... lds), one or two blocks of k ahead of the
// MFMAs, rows of 128 bytes whose 16-byte chunk c lies at position c ^ (row % 8), so that the fragment reads
// of eight rows use every bank once. A lane's 32 bytes of a row are chunks l/16 and l/16 + 4: the same k for both operands,
// in whatever order. Rows of the weight past its end repeat the last one and are never stored; chunks past K, and rows of
// x past the tile's end, are read out of range and land as zeros. The block's scales of the tile's rows (and of its
// weights' rows) take one 4-byte copy a lane.
#pragma once

#include <type_traits>

#include "w4a16_fp8.hpp"

namespace w4a16 {
namespace fp8 {

typedef int i8v_t __attribute__((ext_vector_type(8)));
typedef int i4v_t __attribute__((ext_vector_type(4)));

enum Mode { DENSE = 0, GROUPED = 1, BY_GROUP = 2 };

struct TileParams {
  const uint8_t* x;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  void* out;
  float* out_scales;
  int out_dtype;
  int M, N, K, KB;
  int ldk, xs_ld;
  int up_blocks;     // GLU: blocks of a half
  int tiles_m, tiles_n;
  // tiles of up to 64 rows, over 0: column tile tn starts its blocks of k at the tn-th, so that workgroups side by side do
  // not ask the same channels of memory for rows that lie a power of two apart
  int turn;
  bool once;         // the weight is read past the caches
  // DENSE: the launch takes `count` tiles from the first on; or, with first over 0, the tiles of twice its height from there
  // on in halves (tiles_m counts those)
  int count, first;
  int slice;         // DENSE: blocks of k of a workgroup; slice blockIdx.y's sums go to out + blockIdx.y M N (fp32)
  int scale_rows;    // rows of out_scales' blocks
  bool pair;         // DENSE, tiles of up to 64 rows: two groups of waves share a tile's blocks of k
  GroupTiles groups;
};

// workgroup -> tile, so that consecutive tiles run on the same XCD
__device__ __forceinline__ int tile_of(int b, int G) {
  const int q = G >> 3, r = G & 7, x = b & 7;
  return x * q + (x < r ? x : r) + (b >> 3);
}

// until n loads, and so many reads of LDS, are left in flight
template <int n, int reads = 15>
__device__ __forceinline__ void wait_loads() {
  static_assert(n >= 0 && n < 64 && reads >= 0 && reads < 16, "vmcnt holds 0..63, lgkmcnt 0..15 (15: any)");
  __builtin_amdgcn_s_waitcnt((n & 0xF) | ((n >> 4) << 14) | (0x7 << 4) | (reads << 8));
}

__device__ __forceinline__ f4_t mfma_fp8(i8v_t a, i8v_t b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// a block's sum from widened fragments: step s multiplies bytes 8 s .. 8 s + 7 of each lane's 32
typedef _Float16 h2v_t __attribute__((ext_vector_type(2)));
struct Wide {
  h8_t k[4];
};
__device__ __forceinline__ Wide widen(i8v_t f) {
  Wide r;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const h2v_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(f[2 * s], 1.0f, false);
    const h2v_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(f[2 * s], 1.0f, true);
    const h2v_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(f[2 * s + 1], 1.0f, false);
    const h2v_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(f[2 * s + 1], 1.0f, true);
    r.k[s] = h8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
  return r;
}

// a fragment: chunks q and q + 4 (q = lane / 16) of a row of 128 bytes whose chunk c lies at c ^ (row % 8)
__device__ __forceinline__ i8v_t read_fragment(const uint8_t* tile, int row, int q) {
  const uint8_t* p = tile + row * 128;
  const i4v_t a = *reinterpret_cast<const i4v_t*>(p + ((q ^ (row & 7)) << 4));
  const i4v_t b = *reinterpret_cast<const i4v_t*>(p + (((q + 4) ^ (row & 7)) << 4));
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The weight's copies: non-temporal (ONCE) where few rows read a weight that the last-level cache (256 MiB) would not hold for
// the next call anyway (one row of 8192x57344 83.8 -> 75.7 us, of 28672x8192 41.9 -> 37.7). A small one may be found
// there: sixteen rows of 8192x10240 take 18.6 us cold and 18.0 non-temporal, but 15 where the last 252 MB read were three such.
constexpr long long kOnceBytes = 128LL << 20;
template <bool ONCE>
__device__ __forceinline__ void buffer_copy_weight_to_lds(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, void* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, (int)voff, (int)soff, 0, ONCE ? 2 : 0);
}

// 4 bytes per lane from global memory straight into LDS
__device__ __forceinline__ void buffer_copy4_to_lds(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, void* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 4, (int)voff, (int)soff, 0, 0);
}

// WN x WM waves of NT x MT 16 x 16 outputs; ST stages of LDS, of which ST - 1 are filled ahead; ISSUE copies go out before
// each of a block's MT steps; TOUCH: how many blocks ahead a block's lines are brought into L2
template <int WN, int WM, int NT, int MT, int ST, int ISSUE, int TOUCH = 0>
struct Tile {
  static constexpr int kWN = WN, kWM = WM, kNT = NT, kMT = MT, kStages = ST, kIssue = ISSUE, kTouch = TOUCH;
  static constexpr int kBN = WN * NT * 16, kBM = WM * MT * 16;
  static constexpr int kWaves = WN * WM, kThreads = 64 * kWaves;
  static constexpr int kCopiesX = kBM / 8 / kWaves, kCopiesW = kBN / 8 / kWaves;  // 1 KiB copies a wave and block
  static constexpr int kLoads = kCopiesX + kCopiesW + 1;  // and one of scales
  static constexpr int kCodes = (kBN + kBM) * 128;
  static constexpr int kStage = kCodes + kThreads * 4;
  static constexpr size_t kLdsBytes = ST * kStage + (TOUCH ? kThreads * 4 : 0);
  static constexpr int kScalesX = (kBM + 63) / 64 * 64;  // lanes for x's scales: whole waves
  static_assert(kBM % (8 * kWaves) == 0 && kBN % (8 * kWaves) == 0, "each wave copies as many rows of each operand");
  static_assert(kBN + kScalesX <= kThreads, "a lane copies the scale of one row");
  static_assert((ST - 2) * kLoads + 1 < 64, "vmcnt holds 0..63");
  static_assert(MT * ISSUE >= kLoads, "all of a block's copies go out within one");
  static_assert(!TOUCH || (ST == 2 && kBN + kBM == kThreads && (kLoads + ISSUE - 1) / ISSUE < MT), "a lane touches one row");
};

// LOOP: a workgroup takes tiles blockIdx.x, blockIdx.x + gridDim.x, ..., and the first blocks of the next one are on their way
// while it stores the last; else tile blockIdx.x alone. The loop's tiles cost the 256-row ones spills.
// KG: groups of waves that take a tile's blocks of k in turn, each with stages of its own; the second one's sums are added
// to the first one's. With one workgroup on a compute unit, four waves' MFMAs wait for their own reads and copies.
template <class T, bool GLU, bool WROWS, int MODE, bool EXACT, bool LOOP, bool ONCE, int KG = 1>
__global__ __launch_bounds__(T::kThreads* KG) void fp8_tile_kernel(TileParams p) {
  static_assert(KG == 1 || (KG == 2 && MODE == DENSE && !LOOP && T::kTouch == 0), "two groups: of dense tiles");
  constexpr int NT = T::kNT, MT = T::kMT, BN = T::kBN, BM = T::kBM;
  constexpr int OUT = GLU ? BN / 2 : BN;  // columns of out that a tile makes
  constexpr int ST = T::kStages, ISSUE = T::kIssue;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds_all[];
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  const int wave_of_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = wave_of_all % T::kWaves, group = KG > 1 ? wave_of_all / T::kWaves : 0;
  const int tid = wave * 64 + lane;
  uint8_t* const lds8 = lds_all + group * T::kLdsBytes;
  const int wn = wave % T::kWN, wm = wave / T::kWN;
  const int N = p.N;
  const bool gathered = MODE == GROUPED && p.groups.tokens;

  // ---- the tile at hand ----
  int m0 = 0, rows = 0, n0 = 0, kb0 = 0, kb1 = 0, turned = 0;
  size_t out_row = 0;
  __amdgpu_buffer_rsrc_t xrs, wrs, srs;
  uint32_t xoff[T::kCopiesX], woff[T::kCopiesW], soff = 0, toff = 0;
  const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;  // of every copy: its rows start at a multiple of eight
  const bool scale_x = wave < T::kScalesX / 64, touch_x = wave < BM / 64;
  const uint32_t sstep = scale_x ? (uint32_t)p.xs_ld * 4u : WROWS ? (uint32_t)N * 4u : 4u;

  // Copies: instruction j of the wave fills eight tile rows of x, then of the weight, lane l row l/8 and position l%8.
  // Offsets are bytes from the tile's first row (gathered: from the first token's).
  auto set = [&](const uint8_t* w, const float* ws, int tm, int tn) __attribute__((always_inline)) {
    // tile row r of the weight -> its row: GLU tiles hold BN/2 gate rows, then the matching up rows
    auto weight_row = [&](int r) __attribute__((always_inline)) {
      if constexpr (GLU) return min(n0 + r % OUT, N - 1) + (r / OUT) * N;
      else return min(n0 + r, N - 1);
    };
    auto x_row = [&](int r) __attribute__((always_inline)) {
      int src = min(r, rows - 1);
      if constexpr (MODE == GROUPED)
        if (gathered) src = p.groups.plan[p.groups.token + m0 + src];
      return src;
    };
    const uint32_t wrows = (uint32_t)(GLU ? 2 * N - n0 : min(BN, N - n0));
    xrs = make_rsrc(p.x + (gathered ? 0 : (size_t)m0 * p.ldk), (uint32_t)(gathered ? p.groups.tokens : rows) * (uint32_t)p.ldk);
    wrs = make_rsrc(w + (size_t)n0 * p.ldk, wrows * (uint32_t)p.ldk);
    srs = make_rsrc(scale_x ? p.xs : ws, 0x7FFFFFFFu);
#pragma unroll
    for (int j = 0; j < T::kCopiesX; ++j) {
      const int r = 8 * (wave * T::kCopiesX + j) + (lane >> 3);
      xoff[j] = r < rows ? (uint32_t)x_row(r) * (uint32_t)p.ldk + (uint32_t)chunk : kOutOfRange;
    }
#pragma unroll
    for (int j = 0; j < T::kCopiesW; ++j)
      woff[j] = (uint32_t)(weight_row(8 * (wave * T::kCopiesW + j) + (lane >> 3)) - n0) * (uint32_t)p.ldk + (uint32_t)chunk;
    // and a scale: the first waves' lanes take x's rows', the next ones the weight's
    const int r = scale_x ? tid : tid - T::kScalesX;
    if (scale_x) {
      const int src = x_row(r);
      soff = (uint32_t)(gathered ? src : m0 + src) * 4u;
    } else if constexpr (WROWS) {
      soff = (uint32_t)weight_row(r) * 4u;
    } else if constexpr (GLU) {
      soff = (uint32_t)((min(n0 + r % OUT, N - 1) >> 7) + (r / OUT) * p.up_blocks) * (uint32_t)p.KB * 4u;
    } else {
      soff = (uint32_t)(weight_row(r) >> 7) * (uint32_t)p.KB * 4u;
    }
    if (r >= (scale_x ? rows : BN)) soff = kOutOfRange;
    // Lines that are not in L2 yet hold the tiles that share them up for as long as memory takes. So a block's lines
    // are touched some blocks ahead (into LDS that nothing reads), by lane r that of tile row r: of the weight's rows an
    // eighth, of x's a quarter, as about eight and four tiles that run at once on an XCD share them (2048 rows of
    // 8192x28672: 475 -> 424 us; every row by every tile 462).
    if constexpr (T::kTouch > 0) {
      const int i = touch_x ? tid : tid - BM;
      toff = kOutOfRange;
      if (touch_x ? i % 4 == tn % 4 : i % 8 == tm % 8)
        toff = (uint32_t)(touch_x ? x_row(i) : weight_row(i) - n0) * (uint32_t)p.ldk;
    }
  };

  // The next tile that has something to multiply, or false
  int turn = blockIdx.x;
  const int live = MODE == GROUPED ? min(p.groups.plan[p.groups.list], p.tiles_m) : p.tiles_m;
  const int tiles = live * p.tiles_n;
  const int turns = MODE == BY_GROUP && LOOP ? tiles * p.groups.E : MODE != DENSE ? tiles : p.first > 0 ? 2 * (tiles - p.first) : p.count;
  auto next_tile = [&]() __attribute__((always_inline)) -> bool {
    if (turn >= turns) return false;
    do {
      // (by group: each group's tiles go over all XCDs, as groups differ in their rows)
      int e = MODE == BY_GROUP ? LOOP ? turn / tiles : blockIdx.y : 0, half = 0;
      int t = MODE == BY_GROUP ? tile_of(LOOP ? turn - e * tiles : turn, tiles) : tile_of(turn, turns);
      turn += gridDim.x;
      if constexpr (MODE == DENSE) {
        if (p.first > 0) {  // what whole rounds of tiles twice as high have left: the halves of their tiles from the first one on
          half = t & 1;
          t = p.first + (t >> 1);
        }
      }
      const int tm = MODE == DENSE && p.first > 0 ? 2 * (t % live) + half : t % live, tn = t / live;  // neighbours share the weight's rows
      const uint8_t* w = p.w;
      const float* ws = p.ws;
      n0 = tn * OUT;
      m0 = tm * BM;
      int end = p.M;
      kb0 = 0;
      kb1 = p.KB;
      if constexpr (MODE == DENSE) {
        if (m0 >= p.M) continue;
        kb0 = min((int)blockIdx.y * p.slice, p.KB);
        kb1 = min(kb0 + p.slice, p.KB);
        out_row = (size_t)blockIdx.y * p.M;
      }
      if constexpr (MODE == GROUPED) {
        group_tile(p.groups, tm, e, m0, end);
        if (e >= p.groups.E) {  // the slots of no group: their rows are zeros
          if (GLU && OUT == 128 && p.out_dtype == kE4M3) {
            uint8_t* const codes = static_cast<uint8_t*>(p.out);
            const int cols = min(OUT, N - n0);
            for (int i = threadIdx.x; i < (end - m0) * cols; i += T::kThreads)
              codes[(size_t)(m0 + i / cols) * N + n0 + i % cols] = 0;
            for (int i = threadIdx.x; i < end - m0; i += T::kThreads)
              p.out_scales[(size_t)(n0 / 128) * p.scale_rows + m0 + i] = kLeastScale;
          } else {
            zero_tile(p.out, p.out_dtype, m0, end - m0, N, n0, OUT);
          }
          continue;
        }
        w += (size_t)e * (GLU ? 2 : 1) * N * p.ldk;
        ws += (size_t)e * (GLU ? 2 * p.up_blocks : (N + 127) / 128) * p.KB;
      }
      if constexpr (MODE == BY_GROUP) {
        // group e's blocks of k are its 128-row tiles: as many as earlier groups have come before them
        int before = 0;
        for (int g = lane; g < e; g += 64) before += (p.groups.plan[g + 1] - p.groups.plan[g] + 127) / 128;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) before += __shfl_xor(before, o);
        kb0 = __builtin_amdgcn_readfirstlane(before);
        kb1 = kb0 + __builtin_amdgcn_readfirstlane((p.groups.plan[e + 1] - p.groups.plan[e] + 127) / 128);
        out_row = (size_t)e * p.M;
      }
      rows = min(BM, end - m0);
      if constexpr (BM <= 64) {
        const int nb = kb1 - kb0;
        turned = p.turn && nb > 0 ? tn % nb : 0;
      }
      set(w, ws, tm, tn);
      return true;
    } while (LOOP && turn < turns);
    return false;
  };

  // copy j of a block: x's rows, the weight's, the scales
  auto copy = [&](int j, int i, int stage) __attribute__((always_inline)) {
    uint8_t* const dst = lds8 + stage * T::kStage;
    i = i * KG + group;
    const bool live = i < kb1 - kb0;
    int kb = kb0 + i + turned;
    kb = kb >= kb1 ? kb - (kb1 - kb0) : kb;
    const bool in_k = live && kb * 128 + chunk < p.K;
    if (j < T::kCopiesX) {
      buffer_copy16_to_lds(xrs, in_k ? xoff[j] : kOutOfRange, kb * 128,
                           reinterpret_cast<uint16_t*>(dst + (wave * T::kCopiesX + j) * 1024));
    } else if (j < T::kCopiesX + T::kCopiesW) {
      const int c = j - T::kCopiesX;
      buffer_copy_weight_to_lds<ONCE>(wrs, in_k ? woff[c] : kOutOfRange, kb * 128, dst + BM * 128 + (wave * T::kCopiesW + c) * 1024);
    } else {
      buffer_copy4_to_lds(srs, live ? soff : kOutOfRange, live ? kb * sstep : 0u, dst + T::kCodes + wave * 256);
    }
  };
  auto touch = [&](int i) __attribute__((always_inline)) {
    if constexpr (T::kTouch > 0)
      buffer_copy4_to_lds(touch_x ? xrs : wrs, i < kb1 - kb0 ? toff : kOutOfRange, (kb0 + i) * 128, lds8 + ST * T::kStage + wave * 256);
  };
  auto first_copies = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < ST - 1; ++i)
#pragma unroll
      for (int j = 0; j < T::kLoads; ++j) copy(j, i, i);
    touch(ST - 1);
  };

  f4_t acc[NT][MT];

  // first tile row (of the weight) of this wave's 16 outputs nt
  auto nrow = [&](int nt) __attribute__((always_inline)) {
    if constexpr (GLU) return (nt / (NT / 2)) * OUT + wn * (NT / 2) * 16 + (nt % (NT / 2)) * 16;
    else return (wn * NT + nt) * 16;
  };

  // The sums of the last 16 rows multiplied, and their factors: added to the running sums while the next ones'
  // MFMAs run (over the end of a block too)
  f4_t part[NT];
  float fac[2];
  // scales of the weight's blocks (one of the wave's rows stands for all; GLU: one of each half), or of its rows
  float sw[2];
  f4_t swr[WROWS ? NT : 1];
  auto add = [&](int nt, int mt) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f = GLU && nt >= NT / 2 ? fac[1] : fac[0];
      if constexpr (WROWS) f = fac[0] * swr[nt][i];
      acc[nt][mt][i] = __builtin_fmaf(part[nt][i], f, acc[nt][mt][i]);
    }
  };

  // Fragments: chunks q and q + 4 of a row of 128 bytes, which lie at q ^ (row % 8) and its neighbour half a row away. All of
  // a wave's rows have the same row % 8 and lie at constants from its first ones, so a stage takes five addresses, made anew
  // when the reads go on to it (hidden from the compiler, which adds the stage to each read otherwise: 188 instead of 162 vector
  // instructions a block of the 256-row tiles beside the MFMAs; 2048 rows of 8192x28672 426 -> 416 us).
  const uint32_t lane_x = (uint32_t)(wm * MT * 16 + l16) * 128 + ((q ^ (l16 & 7)) << 4);
  const uint32_t lane_w = (uint32_t)(BM + nrow(0) + l16) * 128 + ((q ^ (l16 & 7)) << 4);
  uint32_t x_lo, x_hi, w_lo, w_hi, scale;
  auto turn_to = [&](int stage) __attribute__((always_inline)) {
    const uint32_t base = (uint32_t)(group * (int)T::kLdsBytes + stage * T::kStage);
    x_lo = base + lane_x;
    w_lo = base + lane_w;
    x_hi = x_lo ^ 64;
    w_hi = w_lo ^ 64;
    scale = base + T::kCodes + (wm * MT * 16 + l16) * 4;
    asm volatile("" : "+v"(x_lo), "+v"(x_hi), "+v"(w_lo), "+v"(w_hi), "+v"(scale));
  };
  static_assert(T::kStage % 128 == 0 && T::kLdsBytes % 128 == 0, "the half of a row is a bit of the address");
  auto fragment = [&](uint32_t lo, uint32_t hi, int rows_on) __attribute__((always_inline)) {
    const i4v_t a = *reinterpret_cast<const i4v_t*>(lds_all + lo + rows_on * 128);
    const i4v_t b = *reinterpret_cast<const i4v_t*>(lds_all + hi + rows_on * 128);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto read_b = [&](int mt) __attribute__((always_inline)) { return fragment(x_lo, x_hi, mt * 16); };
  auto read_a = [&](int nt) __attribute__((always_inline)) {
    return fragment(w_lo, w_hi, GLU ? nt / (NT / 2) * OUT + nt % (NT / 2) * 16 : nt * 16);
  };
  auto read_sx = [&](int mt) __attribute__((always_inline)) { return *reinterpret_cast<const float*>(lds_all + scale + mt * 64); };
  i8v_t a[NT];
  auto read_sw = [&](int stage) __attribute__((always_inline)) {
    const float* const wsc = reinterpret_cast<const float*>(lds8 + stage * T::kStage + T::kCodes) + T::kScalesX;
    if constexpr (WROWS) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) swr[nt] = *reinterpret_cast<const f4_t*>(wsc + nrow(nt) + 4 * q);
    } else {
      sw[0] = wsc[nrow(0)];
      if constexpr (GLU) sw[1] = wsc[nrow(NT / 2)];
    }
  };

  // Block i is multiplied while the next ST - 1 travel into the other stages, a few copies at a time between the MFMAs
  // (a burst of them would hold the wave while the address unit takes it in). Before a block's last 16 rows,
  // whose operands are in registers by then, each wave waits for its own copies of the next block; the barrier
  // makes all waves' visible and frees the block's own stage; and the next block's first fragments are read
  // while the last rows are multiplied. Copies past the last block read out of range, so that the count
  // of loads in flight is the same at every step.
  auto meet = [&]() __attribute__((always_inline)) {
    wait_loads<(ST - 2) * T::kLoads + (T::kTouch > 0), 0>();  // (and for its reads of this block: copies may overwrite it now)
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) part[nt] = f4_t{0.f, 0.f, 0.f, 0.f};
    if constexpr (WROWS) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) swr[nt] = part[nt];
    }
    fac[0] = fac[1] = 0.f;
    meet();
    const int nb = (kb1 - kb0 + KG - 1) / KG;  // (a block past the last one is zeros)
    if (nb <= 0) return;
    if constexpr (MODE == GROUPED && T::kWM > 1) {
      // of a tile that its group does not fill, a wave without rows takes part in the copies only (at this rate a
      // product's time is its energy, so that zeros would be multiplied at the others' cost)
      if (wm * MT * 16 >= rows) {
        int stage = 0;
        for (int i = 0; i < nb; ++i) {
          const int free = stage == 0 ? ST - 1 : stage - 1;
#pragma unroll
          for (int j = 0; j < T::kLoads; ++j) copy(j, i + ST - 1, free);
          meet();
          stage = stage == ST - 1 ? 0 : stage + 1;
        }
        return;
      }
    }
    turn_to(0);
    i8v_t b = read_b(0);
    float sx = read_sx(0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) a[nt] = read_a(nt);
    if (!WROWS) read_sw(0);
    Wide aw[EXACT ? NT : 1];
    int stage = 0;
    for (int i = 0; i < nb; ++i) {
      const int free = stage == 0 ? ST - 1 : stage - 1, next = stage == ST - 1 ? 0 : stage + 1;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int j = mt * ISSUE; j < (mt + 1) * ISSUE && j < T::kLoads; ++j) copy(j, i + ST - 1, free);
        if (mt == (T::kLoads + ISSUE - 1) / ISSUE) touch(i + T::kTouch);
        if (mt == MT - 1) meet();
        if (mt == MT - 1) turn_to(next);
        const i8v_t bn = read_b((mt + 1) % MT);
        const float sxn = read_sx((mt + 1) % MT);
        __builtin_amdgcn_sched_barrier(0);  // the reads travel while these rows are multiplied
        const int before = mt == 0 ? MT - 1 : mt - 1;
        f4_t now[NT];
        if constexpr (EXACT) {
          if (mt == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) aw[nt] = widen(a[nt]);
          }
          const Wide bw = widen(b);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) now[nt] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) now[nt] = mfma16(aw[nt].k[s], bw.k[s], now[nt]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            add(nt, before);
            if (mt == MT - 1) a[nt] = read_a(nt);
          }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            now[nt] = mfma_fp8(a[nt], b);
            if (mt == MT - 1) a[nt] = read_a(nt);
            add(nt, before);
          }
        }
        fac[0] = WROWS ? sx : sx * sw[0];
        if constexpr (GLU) fac[1] = sx * sw[1];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) part[nt] = now[nt];
        // rows' scales are read once the last block's have been used
        if (WROWS && mt == 0) read_sw(stage);
        if (!WROWS && mt == MT - 1) read_sw(next);
        b = bn;
        sx = sxn;
        __builtin_amdgcn_sched_barrier(0);
      }
      stage = next;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) add(nt, MT - 1);
  };

  // Each wave turns 16 rows m by its columns at a time through a slice of LDS of its own (in the last stage, which the
  // next tile's first copies do not fill), and stores runs of a row.
  constexpr int COLS = GLU ? NT / 2 * 16 : NT * 16;  // this wave's columns of out
  constexpr int PITCH = COLS + 4;                    // floats: rows start four banks apart
  static_assert(T::kWaves * 16 * PITCH * 4 + T::kWN * BM * 4 <= T::kStage, "the waves' slices and the rows' maxima fit a stage");
  float* const slices = reinterpret_cast<float*>(lds8 + (ST - 1) * T::kStage);
  float* const slice = slices + wave * 16 * PITCH;
  float* const most = slices + T::kWaves * 16 * PITCH;  // [WN][BM], e4m3
  auto store = [&](int m0, int rows, int n0, size_t out_row) __attribute__((always_inline)) {
    const int nw = n0 + wn * COLS;  // this wave's first column
    if constexpr (GLU) {
#pragma unroll
      for (int nt = 0; nt < NT / 2; ++nt)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float g = acc[nt][mt][i], u = acc[nt + NT / 2][mt][i];
            acc[nt][mt][i] = g / (1.0f + __expf(-g)) * u;  // (a reciprocal would be 0 where 1 + exp(-g) passes 2^126)
          }
      if (OUT == 128 && p.out_dtype == kE4M3) {
        // the largest |h| of a row over the tile's 128 columns: this wave's, then all waves' of the row
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t v = 0;
#pragma unroll
          for (int nt = 0; nt < NT / 2; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int n = nw + nt * 16 + 4 * q + i;
              const float h = acc[nt][mt][i];  // (a bit cast of a vector's element itself takes the first one)
              const uint32_t b = __builtin_bit_cast(uint32_t, h) & 0x7FFFFFFFu;
              v = max(v, n < N ? b : 0u);
            }
          v = max(v, (uint32_t)__shfl_xor((int)v, 16));
          v = max(v, (uint32_t)__shfl_xor((int)v, 32));
          if (q == 0) most[wn * BM + (wm * MT + mt) * 16 + l16] = __builtin_bit_cast(float, v);
        }
        __syncthreads();
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r0 = (wm * MT + mt) * 16;
      if (r0 >= rows) break;  // of this wave's rows, so of all its lanes
#pragma unroll
      for (int nt = 0; nt < COLS / 16; ++nt)
        *reinterpret_cast<f4_t*>(slice + l16 * PITCH + nt * 16 + 4 * q) = acc[nt][mt];
      __builtin_amdgcn_wave_barrier();
      // a lane takes eight columns of a row
#pragma unroll
      for (int pass = 0; pass < (16 * COLS / 8 + 63) / 64; ++pass) {
        const int piece = lane + 64 * pass;
        if (16 * COLS / 8 % 64 != 0 && piece >= 16 * COLS / 8) continue;
        const int r = piece / (COLS / 8), c = piece % (COLS / 8) * 8;
        if (r0 + r >= rows) continue;
        const float* src = slice + r * PITCH + c;
        float v[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const f4_t f = *reinterpret_cast<const f4_t*>(src + 4 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[4 * i + j] = f[j];
        }
        const int n = nw + c, some = N - n;
        if (some <= 0) continue;
        const size_t at = (out_row + m0 + r0 + r) * (size_t)N + n;
        if (GLU && OUT == 128 && p.out_dtype == kE4M3) {
          uint32_t b = 0;
#pragma unroll
          for (int w = 0; w < T::kWN; ++w) b = max(b, __builtin_bit_cast(uint32_t, most[w * BM + r0 + r]));
          const float s = fp8_scale(b);
          const Fp8Divisor d = fp8_divisor(s);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = fp8_quotient<2>(v[j], d);
          const uint32_t lo = fp8_pack(v[0], v[1], v[2], v[3]), hi = fp8_pack(v[4], v[5], v[6], v[7]);
          uint8_t* const dst = static_cast<uint8_t*>(p.out) + at;
          if (some >= 8 && N % 8 == 0) {
            *reinterpret_cast<uint2*>(dst) = uint2{lo, hi};
          } else {
            for (int j = 0; j < 8 && j < some; ++j) dst[j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
          }
          if (wn == 0 && c == 0) p.out_scales[(size_t)(n0 / 128) * p.scale_rows + m0 + r0 + r] = s;
          continue;
        }
        fp8_store8(p.out, at, v, some, p.out_dtype);
      }
      __builtin_amdgcn_wave_barrier();
    }
  };

  if constexpr (LOOP) {
    bool multiplied = false;
    int at_m = 0, at_rows = 0, at_n = 0;
    size_t at_row = 0;
    while (true) {
      const bool more = next_tile();
      if (more) first_copies();
      if (multiplied) store(at_m, at_rows, at_n, at_row);
      if (!more) break;
      multiply();
      at_m = m0;
      at_rows = rows;
      at_n = n0;
      at_row = out_row;
      multiplied = true;
      // every wave is done with the stages, and its last copies (of nothing) have landed
      wait_loads<0>();
      __syncthreads();
    }
  } else {
    if (!next_tile()) return;
    first_copies();
    multiply();
    wait_loads<0>();
    __syncthreads();
    if constexpr (KG > 1) {
      f4_t* const sums = reinterpret_cast<f4_t*>(lds_all) + tid;
      static_assert(NT * MT * T::kThreads * 16 <= (ST - 1) * T::kStage, "the sums leave the stage that results are turned in");
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          if (group) sums[(nt * MT + mt) * T::kThreads] = acc[nt][mt];
      __syncthreads();
      if (group) return;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[nt][mt] += sums[(nt * MT + mt) * T::kThreads];
    }
    store(m0, rows, n0, out_row);
  }
}

// Kinds of kernel, by the rows of x of a tile
enum Kind { STREAM = 0, LOW = 1, MID = 2, HALF = 3, WHOLE = 4 };
typedef Tile<4, 1, 2, 2, 3, 3> Low;       // 32 rows, 128 columns
typedef Tile<4, 1, 2, 4, 3, 2> Mid;       // 64, 128
typedef Tile<4, 2, 4, 4, 3, 2> Half;      // 128, 256
typedef Tile<4, 2, 4, 8, 2, 3, 3> Whole;  // 256, 256: dense rows, results of 16 bits (widened fragments would not fit)

template <class T, bool GLU, bool WROWS, int MODE, bool EXACT>
hipError_t launch_tile(const TileParams& p, unsigned grid, int gy, hipStream_t s) {
  constexpr bool LOOP = std::is_same<T, Half>::value;
  const dim3 blocks(grid, gy), threads(T::kThreads), twice(2 * T::kThreads);
  if constexpr (T::kBM <= 64 && !WROWS) {
    if (p.once) {
      if constexpr (MODE == DENSE) {
        if (p.pair) {
          hipLaunchKernelGGL((fp8_tile_kernel<T, GLU, WROWS, MODE, EXACT, LOOP, true, 2>), blocks, twice, 2 * T::kLdsBytes, s, p);
          return hipGetLastError();
        }
      }
      hipLaunchKernelGGL((fp8_tile_kernel<T, GLU, WROWS, MODE, EXACT, LOOP, true>), blocks, threads, T::kLdsBytes, s, p);
      return hipGetLastError();
    }
  }
  if constexpr (T::kBM <= 64 && MODE == DENSE) {
    if (p.pair) {
      hipLaunchKernelGGL((fp8_tile_kernel<T, GLU, WROWS, MODE, EXACT, LOOP, false, 2>), blocks, twice, 2 * T::kLdsBytes, s, p);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((fp8_tile_kernel<T, GLU, WROWS, MODE, EXACT, LOOP, false>), blocks, threads, T::kLdsBytes, s, p);
  return hipGetLastError();
}

template <bool GLU, bool WROWS, int MODE>
hipError_t launch_kind(const TileParams& p, int kind, bool exact, unsigned grid, int gy, hipStream_t s) {
  if (exact || WROWS) {
    switch (kind) {
      case LOW:
        if constexpr (MODE != BY_GROUP) return launch_tile<Low, GLU, WROWS, MODE, true>(p, grid, gy, s);
      case MID: return launch_tile<Mid, GLU, WROWS, MODE, true>(p, grid, gy, s);
      default: return launch_tile<Half, GLU, WROWS, MODE, true>(p, grid, gy, s);
    }
  }
  if constexpr (!WROWS) {  // a weight's gradient has fp32 results only
    switch (kind) {
      case LOW: return launch_tile<Low, GLU, WROWS, MODE, false>(p, grid, gy, s);
      case MID: return launch_tile<Mid, GLU, WROWS, MODE, false>(p, grid, gy, s);
      case HALF: return launch_tile<Half, GLU, WROWS, MODE, false>(p, grid, gy, s);
      default:
        if constexpr (MODE == DENSE) return launch_tile<Whole, GLU, WROWS, MODE, false>(p, grid, gy, s);
    }
  }
  return hipErrorInvalidValue;
}

}  // namespace fp8
}  // namespace w4a16
