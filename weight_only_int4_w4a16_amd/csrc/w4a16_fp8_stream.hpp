// w4a16_fp8_stream.hpp - products of e4m3 codes for few rows, bound by the weight's bytes: each must cross HBM once, at
// full rate.
//
// A workgroup owns 16 NT rows of the weight and up to 16 MT rows of x; its W waves take contiguous slices of k and their
// partial sums are added through LDS in wave order. Each wave streams its slice through a ring of D slots of its own
// in LDS, one block of 128 k a slot (both operands' codes and x's scales): copies go from memory straight to LDS, so that
// what is in flight takes no registers, eight lanes read 128 consecutive bytes of a row (fragments read from memory
// would touch sixteen rows' lines with every sixteen lanes), and as only the wave that fills a slot reads it, its own
// load counter orders the two and no barrier is needed. Copies past the slice read out of range: no memory is touched.
//
// Codes are widened to fp16 in registers (exactly) and multiplied by v_mfma_f32_16x16x32_f16, which sums in full
// fp32: at these sizes neither bounds the call.
#pragma once

#include "w4a16_fp8_tile.hpp"

namespace w4a16 {
namespace fp8 {

struct StreamParams {
  const uint8_t* x;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  void* out;
  int out_dtype;
  int M, N, K, KB;
  int ldk, xs_ld;
  int up_blocks;  // GLU: blocks of a half
  int slice;      // blocks of k a wave
  bool once;      // the weight is read past the caches
  const void* values;  // XC 0: x itself, of 16 bits
  int values_dtype;
  int tiles_n, tiles_m;
};

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// XC: 1 KiB copies of x a block (eight rows each), or 0 where each workgroup quantizes x itself (two rows at most)
template <int NT, int XC, int D>
struct Stream {
  static constexpr int MT = XC == 4 ? 2 : 1;  // times sixteen rows of x
  static constexpr int kSlot = NT * 2048 + (XC ? XC * 1024 + 256 : 0);
  static constexpr int kLoads = 2 * NT + (XC ? XC + 1 : 0);  // a slot's copies
  static constexpr int kWave = D * kSlot;         // bytes of LDS a wave
  static_assert((D - 1) * kLoads < 64, "vmcnt holds 0..63");
  static constexpr int kSums = NT * MT * 256;     // floats a wave
  static constexpr size_t ring_bytes(int W) {
    const size_t ring = (size_t)W * kWave, sums = (size_t)W * kSums * 4;
    return ring > sums ? ring : sums;
  }
  // groups: of x that a wave quantizes (its blocks of k by the rows)
  static constexpr size_t lds_bytes(int W, int groups) { return ring_bytes(W) + W * group_bytes(groups); }
  // their codes and scales, 16-byte aligned
  static constexpr __host__ __device__ size_t group_bytes(int groups) { return ((size_t)groups * (128 + 4) + 15) & ~(size_t)15; }
};

template <int NT, int XC, int D, int W, bool GLU, bool ONCE>
__global__ __launch_bounds__(64 * W) void fp8_stream_kernel(StreamParams p) {
  typedef Stream<NT, XC, D> S;
  static_assert(!GLU || NT % 2 == 0, "a SwiGLU workgroup holds gate rows and the matching up rows");
  static_assert(XC == 0 || XC == 1 || XC == 2 || XC == 4, "up to two, eight, 16 or 32 rows of x");
  constexpr int MT = S::MT;
  constexpr int OUT = (GLU ? NT / 2 : NT) * 16;  // columns of out a workgroup makes
  extern __shared__ __attribute__((aligned(16))) uint8_t lds8[];
  const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = tile_of(blockIdx.x, p.tiles_m * p.tiles_n);
  const int tm = t % p.tiles_m, tn = t / p.tiles_m;  // neighbours share the weight's rows
  const int N = p.N, n0 = tn * OUT, KB = p.KB;
  const int m0 = tm * 16 * MT, rows = min(16 * MT, p.M - m0);
  const int kb0 = min(wave * p.slice, KB), nb = min(p.slice, KB - kb0);
  uint8_t* const ring = lds8 + wave * S::kWave;

  // Copies: instruction j fills eight rows of a slot (the weight's 16 NT, then x's), lane l row l/8 and position
  // l%8, which holds chunk (l%8) ^ (row % 8). Offsets are bytes from the tile's first row.
  const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
  const uint32_t wrows = (uint32_t)(GLU ? 2 * N - n0 : min(OUT, N - n0));
  const __amdgpu_buffer_rsrc_t wrs = make_rsrc(p.w + (size_t)n0 * p.ldk, wrows * (uint32_t)p.ldk);
  const __amdgpu_buffer_rsrc_t xrs = make_rsrc(p.x + (size_t)m0 * p.ldk, (uint32_t)rows * (uint32_t)p.ldk);
  uint32_t woff[2 * NT], xoff[XC ? XC : 1];
#pragma unroll
  for (int j = 0; j < 2 * NT; ++j) {
    const int r = 8 * j + (lane >> 3);
    const int src = GLU ? min(r % OUT, N - 1 - n0) + (r / OUT) * N : min(r, N - 1 - n0);
    woff[j] = (uint32_t)src * (uint32_t)p.ldk + (uint32_t)chunk;
  }
#pragma unroll
  for (int j = 0; j < XC; ++j) {  // rows past the tile's are zeros
    const int r = 8 * j + (lane >> 3);
    xoff[j] = r < rows ? (uint32_t)r * (uint32_t)p.ldk + (uint32_t)chunk : kOutOfRange;
  }
  // x's scales: lane l that of row l (the last copy of a slot)
  const __amdgpu_buffer_rsrc_t srs = make_rsrc(p.xs, 0x7FFFFFFFu);
  const uint32_t soff = lane < rows ? (uint32_t)(m0 + lane) * 4u : kOutOfRange;

  auto copy = [&](int i) __attribute__((always_inline)) {  // block i of the slice, into slot i % D
    uint8_t* const dst = ring + (i % D) * S::kSlot;
    const int kb = kb0 + i;
    const bool in_k = i < nb && kb * 128 + chunk < p.K;
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j)
      buffer_copy_weight_to_lds<ONCE>(wrs, in_k ? woff[j] : kOutOfRange, kb * 128, dst + j * 1024);
#pragma unroll
    for (int j = 0; j < XC; ++j)
      buffer_copy16_to_lds(xrs, in_k ? xoff[j] : kOutOfRange, kb * 128,
                           reinterpret_cast<uint16_t*>(dst + NT * 2048 + j * 1024));
    if constexpr (XC > 0) buffer_copy4_to_lds(srs, i < nb ? soff : kOutOfRange, kb * p.xs_ld * 4, dst + NT * 2048 + XC * 1024);
  };

  // the blocks' scales of the weight, one for all the workgroup's rows (GLU: of each half): lane l holds block l's
  // of each 64
  const float* const ws0 = p.ws + (size_t)(n0 >> 7) * KB + kb0;
  const float* const ws1 = GLU ? ws0 + (size_t)p.up_blocks * KB : ws0;
  float wsc0 = lane < nb ? ws0[lane] : 0.f, wsc1 = GLU && lane < nb ? ws1[lane] : 0.f;
  // XC 0: the wave's groups of x, block by block and row by row, four at a time by sixteen lanes each; the first sixteen
  // are asked for before the weight
  const int groups = nb * rows, g16 = lane >> 4;
  uint8_t* const codes = lds8 + S::ring_bytes(W) + wave * S::group_bytes(p.slice * p.M);
  float* const code_scales = reinterpret_cast<float*>(codes + (size_t)p.slice * p.M * 128);
  u4_t asked[4];
  auto ask = [&](int g) __attribute__((always_inline)) {
    const int b = g / rows, k = (kb0 + b) * 128 + l16 * 8;
    return g < groups && k < p.K ? *reinterpret_cast<const u4_t*>(static_cast<const uint16_t*>(p.values) + (size_t)(m0 + g - b * rows) * p.K + k)
                                 : u4_t{0u, 0u, 0u, 0u};
  };
  auto quantize = [&](int g, u4_t v, auto dtype) __attribute__((always_inline)) {
    typedef Eight<decltype(dtype)::value> E;
    E e;
    e.v = v;
    uint32_t w = e.magnitude(0);
#pragma unroll
    for (int i = 1; i < E::kWords; ++i) w = E::larger(w, e.magnitude(i));
    const float s = fp8_scale(max_of_16_lanes(E::largest_bits(w)));
    const Fp8Divisor d = fp8_divisor(s);
    float c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = fp8_quotient<decltype(dtype)::value>(e.value(j), d);
    if (g < groups) {
      *reinterpret_cast<uint2*>(codes + g * 128 + l16 * 8) = uint2{fp8_pack(c[0], c[1], c[2], c[3]), fp8_pack(c[4], c[5], c[6], c[7])};
      if (l16 == 0) code_scales[g] = s;
    }
  };
  if constexpr (XC == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) asked[j] = ask(4 * j + g16);
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < D; ++i) copy(i);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (XC == 0) {
    auto all = [&](auto dtype) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * j < groups) quantize(4 * j + g16, asked[j], dtype);
      for (int g = 16; g < groups; g += 4) quantize(g + g16, ask(g + g16), dtype);
    };
    if (p.values_dtype == 0) all(std::integral_constant<int, 0>{});
    else all(std::integral_constant<int, 1>{});
    __builtin_amdgcn_wave_barrier();
  }

  f4_t acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f4_t{0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < nb; ++i) {
    if (i && i % 64 == 0) {
      wsc0 = i + lane < nb ? ws0[i + lane] : 0.f;
      if constexpr (GLU) wsc1 = i + lane < nb ? ws1[i + lane] : 0.f;
    }
    wait_loads<(D - 1) * S::kLoads>();  // slot i has landed: D - 1 slots' copies came after its own
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
    const float sw0 = lane_value(wsc0, i & 63), sw1 = GLU ? lane_value(wsc1, i & 63) : sw0;
    const uint8_t* const wt = ring + (i % D) * S::kSlot;
    const uint8_t* const xt = wt + NT * 2048;
    const float* const xsc = reinterpret_cast<const float*>(xt + XC * 1024);
    Wide a[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) a[nt] = widen(read_fragment(wt, nt * 16 + l16, q));
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      // (eight rows' copy: the other lanes read the same rows again, for columns that are not stored)
      i8v_t bf;
      float sx;
      if constexpr (XC == 0) {  // the codes lie in k order; lanes past the rows repeat the last one
        const int g = i * rows + min(l16, rows - 1);
        const i4v_t lo = *reinterpret_cast<const i4v_t*>(codes + g * 128 + q * 16);
        const i4v_t hi = *reinterpret_cast<const i4v_t*>(codes + g * 128 + q * 16 + 64);
        bf = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        sx = code_scales[g];
      } else {
        bf = read_fragment(xt, mt * 16 + (XC == 1 ? l16 & 7 : l16), q);
        sx = xsc[mt * 16 + l16];
      }
      const Wide b = widen(bf);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f4_t part = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 4; ++s) part = mfma16(a[nt].k[s], b.k[s], part);
        const float f = sx * (GLU && nt >= NT / 2 ? sw1 : sw0);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[nt][mt][r] = __builtin_fmaf(part[r], f, acc[nt][mt][r]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    copy(i + D);
  }

  // ---- the waves' sums, in wave order ----
  // [16 MT rows][16 NT columns] a wave, over its own ring (no copy of a slice is in flight into another's)
  wait_loads<0>();
  __syncthreads();
  float* const red = reinterpret_cast<float*>(lds8);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
      *reinterpret_cast<f4_t*>(red + wave * S::kSums + (mt * 16 + l16) * (NT * 16) + nt * 16 + 4 * q) = acc[nt][mt];
  __syncthreads();
  constexpr int PIECES = OUT / 4;  // of a row
  for (int piece = threadIdx.x; piece < rows * PIECES; piece += 64 * W) {
    const int r = piece / PIECES, c = piece % PIECES * 4, some = N - n0 - c;
    if (some <= 0) continue;
    f4_t v = f4_t{0.f, 0.f, 0.f, 0.f}, u = v;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float* src = red + w * S::kSums + r * (NT * 16) + c;
      v += *reinterpret_cast<const f4_t*>(src);
      if constexpr (GLU) u += *reinterpret_cast<const f4_t*>(src + OUT);
    }
    if constexpr (GLU) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = v[j] / (1.0f + __expf(-v[j])) * u[j];
    }
    const size_t at = (size_t)(m0 + r) * N + n0 + c;
    if (some >= 4 && N % 4 == 0) {
      if (p.out_dtype == 2) {
        *reinterpret_cast<f4_t*>(static_cast<float*>(p.out) + at) = v;
      } else if (p.out_dtype == 0) {
        typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
        *reinterpret_cast<h4_t*>(static_cast<_Float16*>(p.out) + at) = h4_t{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
      } else {
        typedef __bf16 b4_t __attribute__((ext_vector_type(4)));
        *reinterpret_cast<b4_t*>(static_cast<__bf16*>(p.out) + at) = b4_t{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
      }
    } else {
      for (int j = 0; j < 4 && j < some; ++j) store_out(p.out, at + j, v[j], p.out_dtype);
    }
  }
}

}  // namespace fp8
}  // namespace w4a16
