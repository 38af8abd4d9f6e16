// w4a16_fp8_quantize.hip - values of 16 or 32 bits to e4m3 codes with a scale for each 128 (or block of 128 x 128).
//
// All forms read every value once and write its code once; they are bound by those bytes (at decode sizes by
// one launch). The largest magnitude of a group is taken from the bits of |v|, which order as the values do and put
// infinities and NaNs above them.
#include <type_traits>

#include "w4a16_fp8.hpp"

namespace w4a16 {

namespace {

typedef u2_t u2_any_t __attribute__((aligned(1)));
typedef u4_t u4_byte_t __attribute__((aligned(1)));

// ---- rows ----
// Sixteen lanes hold a group of 128, eight values each; a wave takes four groups of R rows, all of whose loads are
// in flight at once, and writes a block's scales of its rows as consecutive words. Four waves take rows below each other.
constexpr int kRowWaves = 4;
template <int DT, int R>
__global__ __launch_bounds__(64 * kRowWaves) void fp8_rows_kernel(const void* __restrict__ x, int M, int K,
                                                                  uint8_t* __restrict__ codes,
                                                                  float* __restrict__ scales, int chunks) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int chunk = blockIdx.x % chunks;
  const int m0 = (int)(blockIdx.x / chunks) * (kRowWaves * R) + wave * R;
  const int kb = chunk * 4 + (lane >> 4), li = lane & 15;
  const int k = kb * 128 + li * 8;
  const bool in_k = k < K;  // K is a multiple of 8: a lane's values are in the row, or none
  Eight<DT> v[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (in_k && m0 + r < M) v[r].load(x, (size_t)(m0 + r) * K + k);
    else v[r].clear();
  }
  float mine = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    uint32_t w = v[r].magnitude(0);
#pragma unroll
    for (int i = 1; i < Eight<DT>::kWords; ++i) w = Eight<DT>::larger(w, v[r].magnitude(i));
    const float s = fp8_scale(max_of_16_lanes(Eight<DT>::largest_bits(w)));
    const Fp8Divisor d = fp8_divisor(s);
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = fp8_quotient<DT>(v[r].value(j), d);
    if (in_k && m0 + r < M)
      *reinterpret_cast<u2_t*>(codes + (size_t)(m0 + r) * K + k) =
          u2_t{fp8_pack(q[0], q[1], q[2], q[3]), fp8_pack(q[4], q[5], q[6], q[7])};
    if (li == r) mine = s;
  }
  if (li < R && m0 + li < M && kb * 128 < K) scales[(size_t)kb * M + m0 + li] = mine;
}

// ---- columns (and rows in the same pass), and blocks of a weight ----
// A workgroup takes 128 x 128 values, a thread eight rows by eight columns of them. Column scales: the threads above
// each other join their maxima through LDS; block scales: all threads do; row scales: the sixteen lanes side by side. The
// transposed codes go through LDS, eight rows of a column (8 bytes) a store: column c's store t lies at slot t ^ (c / 8),
// so that the sixteen threads side by side use every bank once, and leave as whole 16-byte pieces of a column.
// 14336x4096 in fp32 both ways 70 us (5.0 TB/s, a copy's rate); columns of 4096x14336 in bf16 40 us (4.4 TB/s),
// with the rows 59 (4.0); of 4099x2885 13 us (2.7 TB/s): all workgroups run at once, so that reads and writes do not overlap.
constexpr int kTileThreads = 256;

struct Fp8TileParams {
  const void* x;
  int M, K;
  uint8_t* codes;    // as they lie (blocks, and rows)
  float* scales;     // of the blocks or columns
  float* row_scales;
  uint8_t* codes_t;  // transposed, or NULL
  float* scales_t;   // blocks only
  size_t pitch;      // bytes between columns of codes_t
  int limit;         // columns of codes_t that are written: a tile's from 128 (its number) up to here
  int tiles_k;
  const int32_t* list;  // the plan's 128-row tiles, or NULL
  int groups;
};

enum Form { COLUMNS = 0, BLOCKS_OF_ALL = 1, COLUMNS_AND_ROWS = 2 };

template <int DT, int FORM>
__global__ __launch_bounds__(kTileThreads) void fp8_tile_kernel(Fp8TileParams p) {
  typedef Eight<DT> E;
  constexpr bool BLOCKS = FORM == BLOCKS_OF_ALL;
  __shared__ __attribute__((aligned(16))) uint8_t lds[128 * 128];
  uint32_t* const red = reinterpret_cast<uint32_t*>(lds);  // [16][16 * kWords], before the codes
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int tk = blockIdx.x % p.tiles_k, tm = blockIdx.x / p.tiles_k;
  int row0 = tm * 128, end = p.M;
  if (p.list) {
    const int4 t = *reinterpret_cast<const int4*>(p.list + 4 + 4 * tm);
    if (tm >= p.list[0] || t.x >= p.groups) return;
    row0 = t.y;
    end = t.z;
  }
  const int c = tk * 128 + tx * 8, some = p.K - c;
  E v[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int row = row0 + ty * 8 + r;
    if (row < end && some >= 8) v[r].load(p.x, (size_t)row * p.K + c);
    else v[r].clear();
  }
  if (FORM != COLUMNS_AND_ROWS && some > 0 && some < 8) {  // (there K is a multiple of 16)
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int row = row0 + ty * 8 + r;
      if (row >= end) continue;
      if constexpr (DT != 2) {  // (of fp32 it would cost a wave of occupancy: 14336x4096 70.6 -> 75.5 us)
        if (p.K >= 8) {  // the row's last eight, down to the ones asked for
          v[r].load(p.x, (size_t)row * p.K + p.K - 8);
          v[r].drop(8 - some);
          continue;
        }
      }
      v[r].load_some(p.x, (size_t)row * p.K + c, some);
    }
  }
  constexpr int WORDS = E::kWords;
  if constexpr (FORM == COLUMNS_AND_ROWS) {
    float mine = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      uint32_t w = v[r].magnitude(0);
#pragma unroll
      for (int i = 1; i < WORDS; ++i) w = E::larger(w, v[r].magnitude(i));
      const float s = fp8_scale(max_of_16_lanes(E::largest_bits(w)));
      const Fp8Divisor d = fp8_divisor(s);
      float q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = fp8_quotient<DT>(v[r].value(j), d);
      const int row = row0 + ty * 8 + r;
      if (row < end && some > 0)
        *reinterpret_cast<u2_t*>(p.codes + (size_t)row * p.K + c) = u2_t{fp8_pack(q[0], q[1], q[2], q[3]), fp8_pack(q[4], q[5], q[6], q[7])};
      if (tx == r) mine = s;
    }
    if (tx < 8 && row0 + ty * 8 + tx < end) p.row_scales[(size_t)tk * p.M + row0 + ty * 8 + tx] = mine;
  }
  uint32_t most[WORDS];
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    most[w] = v[0].magnitude(w);
#pragma unroll
    for (int r = 1; r < 8; ++r) most[w] = E::larger(most[w], v[r].magnitude(w));
  }
  Fp8Divisor d[BLOCKS ? 1 : 8];
  if constexpr (BLOCKS) {
    uint32_t one = most[0];
#pragma unroll
    for (int w = 1; w < WORDS; ++w) one = E::larger(one, most[w]);
    one = max_of_16_lanes(E::largest_bits(one));
    if (tx == 0) red[ty] = one;
    __syncthreads();
    one = red[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) one = max(one, red[i]);
    const float s = fp8_scale(one);
    d[0] = fp8_divisor(s);
    if (threadIdx.x == 0) {
      const int tiles_m = (p.M + 127) / 128;
      p.scales[(size_t)tm * p.tiles_k + tk] = s;
      if (p.scales_t) p.scales_t[(size_t)tk * tiles_m + tm] = s;
    }
  } else {
#pragma unroll
    for (int w = 0; w < WORDS; w += 4)
      *reinterpret_cast<u4_t*>(red + ty * 16 * WORDS + tx * WORDS + w) = u4_t{most[w], most[w + 1], most[w + 2], most[w + 3]};
    __syncthreads();
#pragma unroll
    for (int i = 1; i < 16; ++i)
#pragma unroll
      for (int w = 0; w < WORDS; w += 4) {
        const u4_t o = *reinterpret_cast<const u4_t*>(red + ((ty + i) & 15) * 16 * WORDS + tx * WORDS + w);
#pragma unroll
        for (int j = 0; j < 4; ++j) most[w + j] = E::larger(most[w + j], o[j]);
      }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = fp8_scale(E::float_bits(most[j / E::kPerWord], j % E::kPerWord));
      d[j] = fp8_divisor(s);
      if (ty == 0 && j < some) p.scales[(size_t)tm * p.K + c + j] = s;
    }
  }
  __syncthreads();
  uint32_t lo[8], hi[8];  // a column's eight codes
  if constexpr (BLOCKS) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {  // a row's eight codes
      float q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = fp8_quotient<DT>(v[r].value(j), d[0]);
      const int row = row0 + ty * 8 + r;
      lo[r] = fp8_pack(q[0], q[1], q[2], q[3]);
      hi[r] = fp8_pack(q[4], q[5], q[6], q[7]);
      if (row < end && some > 0) {
        uint8_t* const dst = p.codes + (size_t)row * p.K + c;
        if (some >= 8) {
          *reinterpret_cast<u2_any_t*>(dst) = u2_t{lo[r], hi[r]};
        } else {
          for (int j = 0; j < some; ++j) dst[j] = (uint8_t)((j < 4 ? lo[r] : hi[r]) >> (8 * (j & 3)));
        }
      }
    }
    if (!p.codes_t) return;
    // rows of codes to columns: two 4 x 4 byte transposes for each half of the rows
    uint32_t tlo[8], thi[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t* src = h ? hi : lo;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const uint32_t a = src[4 * part], b = src[4 * part + 1], cc = src[4 * part + 2], e = src[4 * part + 3];
        const uint32_t ab0 = perm_b32(b, a, 0x05010400u), ab1 = perm_b32(b, a, 0x07030602u);
        const uint32_t ce0 = perm_b32(e, cc, 0x05010400u), ce1 = perm_b32(e, cc, 0x07030602u);
        uint32_t* dst = part ? thi : tlo;
        dst[4 * h + 0] = perm_b32(ce0, ab0, 0x05040100u);
        dst[4 * h + 1] = perm_b32(ce0, ab0, 0x07060302u);
        dst[4 * h + 2] = perm_b32(ce1, ab1, 0x05040100u);
        dst[4 * h + 3] = perm_b32(ce1, ab1, 0x07060302u);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) lo[j] = tlo[j], hi[j] = thi[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float q[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) q[r] = fp8_quotient<DT>(v[r].value(j), d[j]);
      lo[j] = fp8_pack(q[0], q[1], q[2], q[3]);
      hi[j] = fp8_pack(q[4], q[5], q[6], q[7]);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<u2_t*>(lds + (tx * 8 + j) * 128 + ((ty ^ tx) & 15) * 8) = u2_t{lo[j], hi[j]};
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 128 * 8 / kTileThreads; ++i) {
    const int piece = threadIdx.x + i * kTileThreads;
    const int col = piece >> 3, part = piece & 7, cx = col >> 3;
    const u4_t q = *reinterpret_cast<const u4_t*>(lds + col * 128 + ((part ^ (cx >> 1)) & 7) * 16);
    u4_t o = cx & 1 ? u4_t{q[2], q[3], q[0], q[1]} : q;
    const int at = tm * 128 + part * 16, n = p.limit - at;
    if (!BLOCKS && end - row0 < 128) {  // behind the last row: zeros, also where the column's scale is NaN
      const int rows = end - row0 - part * 16;
#pragma unroll
      for (int w = 0; w < 4; ++w) o[w] &= rows >= 4 * w + 4 ? ~0u : rows <= 4 * w ? 0u : (1u << 8 * (rows - 4 * w)) - 1u;
    }
    if (tk * 128 + col >= p.K || n <= 0) continue;
    uint8_t* const dst = p.codes_t + (size_t)(tk * 128 + col) * p.pitch + at;
    if (n >= 16) {
      *reinterpret_cast<u4_byte_t*>(dst) = o;
    } else {
      for (int j = 0; j < n; ++j) dst[j] = (uint8_t)(o[j >> 2] >> (8 * (j & 3)));
    }
  }
}

// Four groups of a row to a wave. Two rows a wave for many: 4096x14336 in bf16 35.7 us with one, 30.9 with two (5.7 TB/s), 33.0
// with four, 34.3 with eight; 4096x4096 12.7, 12.2, 13.4, 15.3; 4096x2048 7.5, 7.7, 8.6, 10.0; 16x8192 2.6, 3.0, 3.6, 4.8.
struct RowsShape {
  size_t chunks, rows, workgroups;  // chunks of a row; rows a wave
};
RowsShape rows_shape(int M, int K) {
  RowsShape r;
  r.chunks = (fp8_blocks(K) + 3) / 4;
  r.rows = (size_t)M * r.chunks >= 32768 ? 2 : 1;
  r.workgroups = r.chunks * (((size_t)M + kRowWaves * r.rows - 1) / (kRowWaves * r.rows));
  return r;
}

template <int DT>
void launch_rows(const void* x, int M, int K, uint8_t* codes, float* scales, hipStream_t s) {
  const RowsShape r = rows_shape(M, K);
  const dim3 grid((unsigned)r.workgroups), threads(64 * kRowWaves);
  if (r.rows == 2) hipLaunchKernelGGL((fp8_rows_kernel<DT, 2>), grid, threads, 0, s, x, M, K, codes, scales, (int)r.chunks);
  else hipLaunchKernelGGL((fp8_rows_kernel<DT, 1>), grid, threads, 0, s, x, M, K, codes, scales, (int)r.chunks);
}

template <int FORM>
void launch_tiles(const Fp8TileParams& p, int tiles_m, int dtype, hipStream_t s) {
  const dim3 grid((unsigned)((size_t)tiles_m * p.tiles_k)), threads(kTileThreads);
  if (dtype == 0) hipLaunchKernelGGL((fp8_tile_kernel<0, FORM>), grid, threads, 0, s, p);
  else if (dtype == 1) hipLaunchKernelGGL((fp8_tile_kernel<1, FORM>), grid, threads, 0, s, p);
  else if constexpr (FORM != COLUMNS_AND_ROWS) hipLaunchKernelGGL((fp8_tile_kernel<2, FORM>), grid, threads, 0, s, p);
}

}  // namespace

bool fp8_rows_fit(int M, int K) { return rows_shape(M, K).workgroups * 64 * kRowWaves < (1ULL << 32); }
bool fp8_tiles_fit(int M, int K) { return fp8_blocks(M) * fp8_blocks(K) * kTileThreads < (1ULL << 32); }

hipError_t launch_fp8_rows(const void* x, int M, int K, int dtype, uint8_t* codes, float* scales, hipStream_t s) {
  if (dtype == 0) launch_rows<0>(x, M, K, codes, scales, s);
  else if (dtype == 1) launch_rows<1>(x, M, K, codes, scales, s);
  else launch_rows<2>(x, M, K, codes, scales, s);
  return hipGetLastError();
}

hipError_t launch_fp8_columns(const void* x, int M, int K, int dtype, uint8_t* codes, size_t pitch, float* scales,
                              uint8_t* row_codes, float* row_scales, const RouteLayout* r, const int32_t* plan,
                              hipStream_t s) {
  Fp8TileParams p{};
  p.x = x;
  p.M = M;
  p.K = K;
  p.scales = scales;
  p.codes_t = codes;
  p.pitch = pitch;
  p.limit = (int)pitch;
  p.tiles_k = (int)fp8_blocks(K);
  int tiles = (int)fp8_blocks(M);
  if (r) {
    p.list = plan + r->tiles[kTileLists - 1];
    p.groups = r->E;
    tiles = tile_bound(r->S, r->E, kTileLists - 1);
  }
  if (row_codes) {
    p.codes = row_codes;
    p.row_scales = row_scales;
    launch_tiles<COLUMNS_AND_ROWS>(p, tiles, dtype, s);
  } else {
    launch_tiles<COLUMNS>(p, tiles, dtype, s);
  }
  return hipGetLastError();
}

hipError_t launch_fp8_weight(const void* w, int N, int K, int dtype, uint8_t* codes, float* scales, uint8_t* codes_t,
                             float* scales_t, hipStream_t s) {
  Fp8TileParams p{};
  p.x = w;
  p.M = N;
  p.K = K;
  p.codes = codes;
  p.scales = scales;
  p.codes_t = codes_t;
  p.scales_t = scales_t;
  p.pitch = (size_t)N;
  p.limit = N;
  p.tiles_k = (int)fp8_blocks(K);
  launch_tiles<BLOCKS_OF_ALL>(p, (int)fp8_blocks(N), dtype, s);
  return hipGetLastError();
}

}  // namespace w4a16
