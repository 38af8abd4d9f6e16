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
// Tiles. Both operands go from memory straight to LDS (buffer_load_dwordx4 ... lds), one block of k ahead of the
// MFMAs, rows of 128 bytes whose 16-byte chunk c lies at position c ^ (row % 8), so that the fragment reads
// of eight rows use every bank once. A lane's 32 bytes of a row are chunks l/16 and l/16 + 4: the same k for both operands,
// in whatever order. Rows past the tile's end repeat the last one and are never stored; chunks past K are read out of
// range and land as zeros. The block's scales of the tile's rows (and of its weights' rows) take one
// 4-byte copy a lane.
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
  int scale_rows;    // GROUPED with e4m3 out: rows of out_scales' blocks
  GroupTiles groups;
};

// workgroup -> tile, so that consecutive tiles run on the same XCD
__device__ __forceinline__ int tile_of(int b, int G) {
  const int q = G >> 3, r = G & 7, x = b & 7;
  return x * q + (x < r ? x : r) + (b >> 3);
}

template <int n>
__device__ __forceinline__ void wait_loads() {
  static_assert(n >= 0 && n < 64, "vmcnt holds 0..63");
  __builtin_amdgcn_s_waitcnt((n & 0xF) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8));
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

// 4 bytes per lane from global memory straight into LDS
__device__ __forceinline__ void buffer_copy4_to_lds(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, void* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 4, (int)voff, (int)soff, 0, 0);
}

// WN x WM waves of NT x MT 16 x 16 outputs
template <int WN, int WM, int NT, int MT>
struct Tile {
  static constexpr int kWN = WN, kWM = WM, kNT = NT, kMT = MT;
  static constexpr int kBN = WN * NT * 16, kBM = WM * MT * 16;
  static constexpr int kWaves = WN * WM, kThreads = 64 * kWaves;
  static constexpr int kCopies = (kBN + kBM) / 8 / kWaves;  // 1 KiB copies a wave and block
  static constexpr int kCodes = (kBN + kBM) * 128;
  static constexpr int kStage = kCodes + (kBN + kBM) * 4;
  static constexpr size_t kLdsBytes = 2 * kStage;
  static_assert(kBN + kBM == kThreads, "a lane copies the scale of one row");
  static_assert(kBM % (8 * kCopies) == 0 && kBM % 64 == 0, "a wave copies rows of one operand");
};
typedef Tile<4, 2, 4, 8> Large;  // 256 x 256
typedef Tile<2, 2, 4, 4> Small;  // 128 x 128

template <class T, bool GLU, bool WROWS, int MODE, bool EXACT>
__global__ __launch_bounds__(T::kThreads) void fp8_tile_kernel(TileParams p) {
  constexpr int NT = T::kNT, MT = T::kMT, BN = T::kBN, BM = T::kBM;
  constexpr int OUT = GLU ? BN / 2 : BN;  // columns of out that a tile makes
  extern __shared__ __attribute__((aligned(16))) uint8_t lds8[];
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave % T::kWN, wm = wave / T::kWN;
  const int t = tile_of(blockIdx.x, p.tiles_m * p.tiles_n);
  const int tm = t % p.tiles_m, tn = t / p.tiles_m;  // neighbours share the weight's rows
  const int N = p.N, n0 = tn * OUT;
  int m0 = tm * BM, end = p.M, kb0 = 0, kb1 = p.KB, e = 0;
  size_t out_row = 0;
  if constexpr (MODE == GROUPED) {
    if (!group_tile(p.groups, tm, e, m0, end)) return;
    if constexpr (BM > 128) {
      // the list's tiles have 128 rows: every second one of a group stands for itself and the next
      const int first = e < p.groups.E ? p.groups.plan[e] : p.groups.plan[p.groups.E];
      const int last = e < p.groups.E ? p.groups.plan[e + 1] : p.M;
      if ((m0 - first) % BM) return;
      end = min(m0 + BM, last);
    }
    if (e >= p.groups.E) {  // the slots of no group: their rows are zeros
      if constexpr (GLU) {
        if (p.out_dtype == kE4M3) {
          uint8_t* const codes = static_cast<uint8_t*>(p.out);
          const int cols = min(OUT, N - n0);
          for (int i = threadIdx.x; i < (end - m0) * cols; i += T::kThreads)
            codes[(size_t)(m0 + i / cols) * N + n0 + i % cols] = 0;
          for (int i = threadIdx.x; i < end - m0; i += T::kThreads)
            p.out_scales[(size_t)(n0 / 128) * p.scale_rows + m0 + i] = kLeastScale;
          return;
        }
      }
      zero_tile(p.out, p.out_dtype, m0, end - m0, N, n0, OUT);
      return;
    }
    p.w += (size_t)e * (GLU ? 2 : 1) * N * p.ldk;
    p.ws += (size_t)e * (GLU ? 2 * p.up_blocks : (N + 127) / 128) * p.KB;
  }
  if constexpr (MODE == BY_GROUP) {
    // group e's blocks of k are its 128-row tiles: as many as earlier groups have come before them
    e = blockIdx.y;
    int before = 0;
    for (int g = lane; g < e; g += 64) before += (p.groups.plan[g + 1] - p.groups.plan[g] + 127) / 128;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) before += __shfl_xor(before, o);
    kb0 = __builtin_amdgcn_readfirstlane(before);
    kb1 = kb0 + __builtin_amdgcn_readfirstlane((p.groups.plan[e + 1] - p.groups.plan[e] + 127) / 128);
    out_row = (size_t)e * p.M;
  }
  const int rows = min(BM, end - m0);

  // This lane's copies: instruction j of the wave fills eight tile rows (x's first, then the weight's), lane l
  // row l/8 and position l%8. Offsets are bytes from the tile's first row (gathered: from the first token's).
  const bool gathered = MODE == GROUPED && p.groups.tokens;
  // tile row r of the weight -> its row: GLU tiles hold BN/2 gate rows, then the matching up rows
  auto weight_row = [&](int r) __attribute__((always_inline)) {
    if constexpr (GLU) return min(n0 + r % OUT, N - 1) + (r / OUT) * N;
    else return min(n0 + r, N - 1);
  };
  constexpr int WAVES_X = BM / (8 * T::kCopies);  // waves that copy x's rows
  const bool mine_x = wave < WAVES_X;
  const uint8_t* const xbase = p.x + (gathered ? 0 : (size_t)m0 * p.ldk);
  const uint8_t* const wbase = p.w + (size_t)n0 * p.ldk;
  const uint32_t wrows = (uint32_t)(GLU ? 2 * N - n0 : min(BN, N - n0));
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(
      mine_x ? xbase : wbase, mine_x ? (uint32_t)(gathered ? p.groups.tokens : rows) * (uint32_t)p.ldk : wrows * (uint32_t)p.ldk);
  uint32_t off[T::kCopies];
#pragma unroll
  for (int j = 0; j < T::kCopies; ++j) {
    const int r = 8 * (wave * T::kCopies + j) + (lane >> 3);
    int src;
    if (mine_x) {
      src = min(r, rows - 1);
      if constexpr (MODE == GROUPED)
        if (gathered) src = p.groups.plan[p.groups.token + m0 + src];
    } else {
      src = weight_row(r - BM) - n0;
    }
    off[j] = (uint32_t)src * (uint32_t)p.ldk + (uint32_t)(((lane & 7) ^ (r & 7)) * 16);
  }
  const int chunk = (lane & 7) ^ (lane >> 3);  // of every copy: its rows start at a multiple of eight
  // and its scale: thread i that of tile row i
  const bool scale_x = wave < BM / 64;
  uint32_t soff;
  {
    const int r = threadIdx.x;
    if (scale_x) {
      int src = min(r, rows - 1);
      if constexpr (MODE == GROUPED)
        if (gathered) src = p.groups.plan[p.groups.token + m0 + src];
      soff = (uint32_t)(gathered ? src : m0 + src) * 4u;
    } else if constexpr (WROWS) {
      soff = (uint32_t)weight_row(r - BM) * 4u;
    } else if constexpr (GLU) {
      const int rr = r - BM;
      soff = (uint32_t)((min(n0 + rr % OUT, N - 1) >> 7) + (rr / OUT) * p.up_blocks) * (uint32_t)p.KB * 4u;
    } else {
      soff = (uint32_t)(weight_row(r - BM) >> 7) * (uint32_t)p.KB * 4u;
    }
  }
  const __amdgpu_buffer_rsrc_t srs = make_rsrc(scale_x ? p.xs : p.ws, 0x7FFFFFFFu);
  const uint32_t sstep = scale_x ? (uint32_t)p.xs_ld * 4u : WROWS ? (uint32_t)N * 4u : 4u;

  auto copy = [&](int kb, int stage) __attribute__((always_inline)) {
    uint8_t* const dst = lds8 + stage * T::kStage;
    const bool in_k = kb * 128 + chunk * 16 < p.K;
#pragma unroll
    for (int j = 0; j < T::kCopies; ++j)
      buffer_copy16_to_lds(rs, in_k ? off[j] : kOutOfRange, kb * 128,
                           reinterpret_cast<uint16_t*>(dst + (wave * T::kCopies + j) * 1024));
    buffer_copy4_to_lds(srs, soff, kb * sstep, dst + T::kCodes + wave * 256);
  };

  f4_t acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f4_t{0.f, 0.f, 0.f, 0.f};

  // first tile row (of the weight) of this wave's 16 outputs nt
  auto nrow = [&](int nt) __attribute__((always_inline)) {
    if constexpr (GLU) return (nt / (NT / 2)) * OUT + wn * (NT / 2) * 16 + (nt % (NT / 2)) * 16;
    else return (wn * NT + nt) * 16;
  };

  auto compute = [&](int stage) __attribute__((always_inline)) {
    const uint8_t* const xt = lds8 + stage * T::kStage;
    const uint8_t* const wt = xt + BM * 128;
    const float* const xsc = reinterpret_cast<const float*>(xt + T::kCodes);
    const float* const wsc = xsc + BM;
    typename std::conditional<EXACT, Wide, i8v_t>::type a[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const i8v_t f = read_fragment(wt, nrow(nt) + l16, q);
      if constexpr (EXACT) a[nt] = widen(f);
      else a[nt] = f;
    }
    // block scales: one of the wave's rows stands for all (GLU: one of each half)
    float sw[2];
    f4_t swr[WROWS ? NT : 1];
    if constexpr (WROWS) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) swr[nt] = *reinterpret_cast<const f4_t*>(wsc + nrow(nt) + 4 * q);
    } else {
      sw[0] = wsc[nrow(0)];
      sw[1] = GLU ? wsc[nrow(NT / 2)] : sw[0];
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = (wm * MT + mt) * 16 + l16;
      const i8v_t b = read_fragment(xt, r, q);
      const float sx = xsc[r];
      f4_t part[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) part[nt] = f4_t{0.f, 0.f, 0.f, 0.f};
      if constexpr (EXACT) {
        const Wide bw = widen(b);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) part[nt] = mfma16(a[nt].k[s], bw.k[s], part[nt]);
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) part[nt] = mfma_fp8(a[nt], b);
      }
      const float f0 = WROWS ? sx : sx * sw[0], f1 = GLU ? sx * sw[1] : f0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f = nt < NT / 2 ? f0 : f1;
          if constexpr (WROWS) f = sx * swr[nt][i];
          acc[nt][mt][i] = __builtin_fmaf(part[nt][i], f, acc[nt][mt][i]);
        }
    }
  };

  // Block i is multiplied while block i + 1 travels into the other stage. Each wave waits for its own copies; the
  // barrier makes all waves' visible and frees the stage of block i - 1.
  const int nb = kb1 - kb0;
  if (nb > 0) copy(kb0, 0);
  for (int i = 0; i < nb; ++i) {
    wait_loads<0>();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
    if (i + 1 < nb) copy(kb0 + i + 1, (i + 1) & 1);
    compute(i & 1);
  }

  // ---- epilogue ----
  // Each wave turns 16 rows m by its columns at a time through a slice of LDS of its own, and stores runs of a row.
  constexpr int COLS = GLU ? NT / 2 * 16 : NT * 16;  // this wave's columns of out
  constexpr int PITCH = COLS + 4;                    // floats: rows start four banks apart
  static_assert(T::kWaves * 16 * PITCH * 4 <= (int)T::kLdsBytes, "the waves' slices fit where the tiles were");
  const int nw = n0 + wn * COLS;                     // its first column
  wait_loads<0>();
  __syncthreads();
  float* const slice = reinterpret_cast<float*>(lds8) + wave * 16 * PITCH;
  float* const most = reinterpret_cast<float*>(lds8) + T::kWaves * 16 * PITCH;  // [WN][BM], e4m3
  if constexpr (GLU) {
#pragma unroll
    for (int nt = 0; nt < NT / 2; ++nt)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float g = acc[nt][mt][i], u = acc[nt + NT / 2][mt][i];
          acc[nt][mt][i] = g / (1.0f + __expf(-g)) * u;
        }
    if (p.out_dtype == kE4M3) {
      static_assert(T::kWaves * 16 * PITCH * 4 + T::kWN * BM * 4 <= (int)T::kLdsBytes, "and the rows' maxima");
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
    for (int piece = lane; piece < 16 * COLS / 8; piece += 64) {
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
      if (GLU && p.out_dtype == kE4M3) {
        uint32_t b = 0;
#pragma unroll
        for (int w = 0; w < T::kWN; ++w) b = max(b, __builtin_bit_cast(uint32_t, most[w * BM + r0 + r]));
        const float s = fp8_scale(b);
        const Fp8Divisor d = fp8_divisor(s);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = fp8_quotient(v[j], d);
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
      if (p.out_dtype == 2) {
        float* const dst = static_cast<float*>(p.out) + at;
        if (some >= 8 && N % 4 == 0) {
          *reinterpret_cast<f4_t*>(dst) = f4_t{v[0], v[1], v[2], v[3]};
          *reinterpret_cast<f4_t*>(dst + 4) = f4_t{v[4], v[5], v[6], v[7]};
        } else {
          for (int j = 0; j < 8 && j < some; ++j) dst[j] = v[j];
        }
      } else if (some >= 8 && N % 8 == 0) {
        if (p.out_dtype == 0) {
          h8_t o;
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = (_Float16)v[j];
          *reinterpret_cast<h8_t*>(static_cast<_Float16*>(p.out) + at) = o;
        } else {
          b8_t o;
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = (__bf16)v[j];
          *reinterpret_cast<b8_t*>(static_cast<__bf16*>(p.out) + at) = o;
        }
      } else {
        for (int j = 0; j < 8 && j < some; ++j) store_out(p.out, at + j, v[j], p.out_dtype);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace fp8
}  // namespace w4a16
