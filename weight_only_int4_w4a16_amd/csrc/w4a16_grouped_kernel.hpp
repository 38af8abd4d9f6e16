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
// Work split. A workgroup owns 16 rows by SW 16-column strips over all of K, its waves take
// contiguous k-block slices (as in the decode kernel) and their partial tiles are added through LDS in
// wave order. Row tiles of one group and column tile are neighbours on one XCD, so a second
// tile of the same group finds the codes in that L2.
//
// Operands. v_mfma_f32_16x16x32: word j of a lane's 16-byte chunk of a packed block is its B
// operand for k-step j, and its A operand is 16 bytes of row l%16, loaded from global memory
// (L2: every workgroup of a tile reads the same rows): staging x in LDS would cost a barrier
// and as much LDS traffic as the loads it saves. Rows past the tile's last one read out of
// range, which costs no traffic and gives zeros.
#pragma once

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

template <int ACT, int FMT>
__device__ __forceinline__ typename ActT<ACT>::type dequant_word(uint32_t w, uint32_t sraw, uint32_t zq,
                                                                 const uint32_t* ptab) {
  if constexpr (FMT == FMT_NF4) {
    if constexpr (ACT == ACT_F16)
      return dequant_word_nf4_f16_tab(w, ptab, as_h2(sraw * 0x00010001u));
    else
      return dequant_word_nf4_bf16_tab(w, ptab, (float)__builtin_bit_cast(_Float16, (uint16_t)sraw));
  } else if constexpr (ACT == ACT_F16) {
    return dequant_word_f16(w, make_zero_f16(zq), as_h2(sraw * 0x00010001u));
  } else {
    return dequant_word_bf16(w, make_zero_f32(zq, __builtin_bit_cast(float, sraw << 16)));
  }
}

constexpr int kMaxWaves = 8;

// GLU: the first SW / 2 strips are gate strips, the others the matching up strips, and the
// output is h = SiLU(gate) * up, [S][N / 2].
template <int ACT, int GPC, int FMT, int SW, bool GLU>
__global__ __launch_bounds__(64 * kMaxWaves) void grouped_kernel(GroupedParams p) {
  typedef typename ActT<ACT>::type AT;
  constexpr bool ZEROS = FMT == FMT_ASYM;
  constexpr int OS = GLU ? SW / 2 : SW;  // output strips
  extern __shared__ __attribute__((aligned(16))) float red[];  // [waves][SW][4][64]
  __shared__ uint32_t ptab[FMT == FMT_NF4 ? kNf4PairEntries : 1];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int t = tile_of(blockIdx.x, p.groups.bound * p.col_tiles);
  const int tn = t / p.groups.bound;
  int e, p0, end;
  if (!group_tile(p.groups, t - tn * p.groups.bound, e, p0, end)) return;
  const int rows = min(16, end - p0);
  const int K = p.K, N = p.N, KC = p.KC;
  const int width = GLU ? N >> 1 : N;  // of an output row
  const int ocol0 = tn * OS * 16;
  const int ocols = min(OS * 16, width - ocol0);
  if (e >= p.groups.E) {  // the slots of no group: their rows are zeros
    zero_tile(p.out, p.out_dtype, p0, rows, width, ocol0, OS * 16);
    return;
  }
  if constexpr (FMT == FMT_NF4) {
    nf4_pair_table_fill(ptab, p.codebook);
    __syncthreads();
  }

  // strip s of this tile, clamped in bounds for loads (never stored past the last one)
  auto strip = [&](int s) __attribute__((always_inline)) {
    return GLU ? min(tn * OS + (s < OS ? s : s - OS), p.half - 1) + (s < OS ? 0 : p.half)
               : min(tn * SW + s, p.NT - 1);
  };
  const u4_t* const wbase = p.packed + (size_t)e * p.NT * KC * 64;
  const uint16_t* const sbase = p.scales + (size_t)e * p.NG * N;
  const uint32_t* const zbase = ZEROS ? p.qzeros + (size_t)e * p.NG * (N >> 3) : nullptr;
  const __amdgpu_buffer_rsrc_t srs = make_rsrc(sbase, (uint32_t)p.NG * N * 2);
  const __amdgpu_buffer_rsrc_t zrs = make_rsrc(ZEROS ? (const void*)zbase : (const void*)sbase, (uint32_t)p.NG * (N >> 3) * 4);
  const int shift = 4 * (lane & 7);

  // this lane's row of the tile: byte offset of its 16-byte chunk of k-step 0
  const int arow = lane & 15;
  uint32_t aoff = kOutOfRange;
  if (arow < rows)
    aoff = (uint32_t)(p.groups.tokens ? p.groups.plan[p.groups.order + p0 + arow] / p.groups.topk : arow) *
               (uint32_t)K * 2u + (lane >> 4) * 16u;
  const __amdgpu_buffer_rsrc_t xrs = p.groups.tokens
      ? make_rsrc(p.x, (uint32_t)p.groups.tokens * (uint32_t)K * 2u)
      : make_rsrc(p.x + (size_t)p0 * K, (uint32_t)rows * (uint32_t)K * 2u);

  struct Regs {
    u4_t b[SW], a[4];
    uint32_t s[SW][GPC], z[SW][GPC];
  };
  auto load = [&](Regs& R, int kc) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < SW; ++s)
      R.b[s] = __builtin_nontemporal_load(wbase + ((size_t)strip(s) * KC + kc) * 64 + lane);
#pragma unroll
    for (int j = 0; j < 4; ++j)  // steps past a ragged K are not multiplied
      R.a[j] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(xrs, aoff, min(kc * 128 + 32 * j, K - 32) * 2, 0));
#pragma unroll
    for (int s = 0; s < SW; ++s) {
      const int col = strip(s) * 16 + (lane & 15);
#pragma unroll
      for (int gi = 0; gi < GPC; ++gi) {
        const int g = min(kc * GPC + gi, p.NG - 1);
        R.s[s][gi] = __builtin_amdgcn_raw_buffer_load_b16(srs, col * 2, g * N * 2, 0);
        if constexpr (ZEROS) R.z[s][gi] = __builtin_amdgcn_raw_buffer_load_b32(zrs, (col >> 3) * 4, g * (N >> 3) * 4, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  f4_t acc[SW];
#pragma unroll
  for (int s = 0; s < SW; ++s) acc[s] = f4_t{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Regs& R, int kc) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kc * 128 + 32 * j >= K) break;
      const int gi = j * GPC / 4;
#pragma unroll
      for (int s = 0; s < SW; ++s) {
        const uint32_t zq = ZEROS ? (R.z[s][gi] >> shift) & 0xFu : 8u;
        acc[s] = mfma16(__builtin_bit_cast(AT, R.a[j]), dequant_word<ACT, FMT>(R.b[s][j], R.s[s][gi], zq, ptab), acc[s]);
      }
    }
  };
  const int kc0 = min(wave * p.slice, KC), kc1 = min(kc0 + p.slice, KC);
  if (kc0 < kc1) {
    Regs A, B;
    load(A, kc0);
    for (int kc = kc0; kc < kc1; kc += 2) {
      load(B, min(kc + 1, kc1 - 1));
      compute(A, kc);
      load(A, min(kc + 2, kc1 - 1));
      if (kc + 1 < kc1) compute(B, kc + 1);
    }
  }
  // lane l holds column l%16 of each strip and rows 4 (l/16) + i, i < 4
#pragma unroll
  for (int s = 0; s < SW; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[((wave * SW + s) * 4 + i) * 64 + lane] = acc[s][i];
  __syncthreads();
  for (int q = threadIdx.x; q < rows * OS * 16; q += blockDim.x) {
    const int r = q / (OS * 16), c = q - r * (OS * 16);
    if (c >= ocols) continue;
    const int at = ((c >> 4) * 4 + (r & 3)) * 64 + (r >> 2) * 16 + (c & 15);
    float v = 0.f, u = 0.f;
    for (int w = 0; w < waves; ++w) {
      v += red[w * SW * 256 + at];
      if constexpr (GLU) u += red[w * SW * 256 + at + OS * 256];
    }
    if constexpr (GLU) v = v / (1.0f + __expf(-v)) * u;
    store_out(p.out, (size_t)(p0 + r) * width + ocol0 + c, v, p.out_dtype);
  }
}

struct GroupedGeometry {
  int SW, waves;
};

template <int ACT, int GPC, int FMT, int SW>
hipError_t launch_sw(const GroupedParams& p, const GroupedGeometry& g, bool glu, hipStream_t s) {
  const dim3 grid(p.groups.bound * p.col_tiles), block(64 * g.waves);
  const size_t lds = (size_t)g.waves * SW * 256 * 4;
  if (glu)
    hipLaunchKernelGGL((grouped_kernel<ACT, GPC, FMT, SW, true>), grid, block, lds, s, p);
  else
    hipLaunchKernelGGL((grouped_kernel<ACT, GPC, FMT, SW, false>), grid, block, lds, s, p);
  return hipGetLastError();
}

template <int ACT, int GPC, int FMT>
hipError_t launch_fmt(const GroupedParams& p, const GroupedGeometry& g, bool glu, hipStream_t s) {
  return g.SW == 4 ? launch_sw<ACT, GPC, FMT, 4>(p, g, glu, s) : launch_sw<ACT, GPC, FMT, 2>(p, g, glu, s);
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
