// w4a16_fp8.hip - which kernel takes a product of e4m3 codes, and its launch geometry.
#include <stdlib.h>

#include "w4a16_fp8_stream.hpp"

namespace w4a16 {

using namespace fp8;

namespace fp8 {
// The kernels' instantiations, one source for each kind of product (w4a16_fp8_{dense,glu,grouped,grouped_glu,columns}.hip)
#define W4A16_FP8_EXTERN(NAME) hipError_t NAME(const TileParams& p, int kind, bool exact, unsigned grid, int gy, hipStream_t s)
W4A16_FP8_EXTERN(launch_dense);
W4A16_FP8_EXTERN(launch_glu);
W4A16_FP8_EXTERN(launch_grouped_plain);
W4A16_FP8_EXTERN(launch_grouped_glu);
W4A16_FP8_EXTERN(launch_columns);
W4A16_FP8_EXTERN(launch_by_group);
hipError_t launch_stream(const StreamParams& p, int NT, int XC, int W, bool glu, unsigned grid, hipStream_t s);
}  // namespace fp8

namespace {

// ---- after a product: sums of its slices of k, and h to codes ----
// Sixteen lanes take 128 columns of a row, eight each; the partial sums [S][M][width] are added in slice order. GLU: width is
// 2 N, gate columns first. Bound by the partial sums' bytes.
template <bool GLU>
__global__ __launch_bounds__(256) void fp8_finish_kernel(const float* __restrict__ part, int S, int M, int N, void* out,
                                                         int out_dtype, float* __restrict__ out_scales, int chunks) {
  const int lane = threadIdx.x & 63, item = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int m = item / chunks, n = (item - m * chunks) * 512 + lane * 8;
  if (m >= M) return;
  const size_t width = GLU ? 2 * (size_t)N : N, slice = (size_t)M * width;
  const int some = N - n;
  float v[8], u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = u[j] = 0.f;
  auto add = [&](const float* row, float (&sum)[8]) __attribute__((always_inline)) {
    if (some >= 8) {
      const f4_t a = *reinterpret_cast<const f4_any_t*>(row), b = *reinterpret_cast<const f4_any_t*>(row + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += a[j], sum[4 + j] += b[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < some) sum[j] += row[j];
    }
  };
  if (some > 0)
    for (int s = 0; s < S; ++s) {
      const float* row = part + s * slice + (size_t)m * width + n;
      add(row, v);
      if constexpr (GLU) add(row + N, u);
    }
  if constexpr (GLU) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] / (1.0f + __expf(-v[j])) * u[j];
  }
  const size_t at = (size_t)m * N + n;
  if (out_dtype == kE4M3) {
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) most = max(most, j < some ? __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu : 0u);
    const float sc = fp8_scale(max_of_16_lanes(most));
    const Fp8Divisor d = fp8_divisor(sc);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fp8_quotient<2>(v[j], d);
    if (some > 0) {  // N is a multiple of 16
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(out) + at) = uint2{fp8_pack(v[0], v[1], v[2], v[3]), fp8_pack(v[4], v[5], v[6], v[7])};
      if ((lane & 15) == 0) out_scales[(size_t)(n >> 7) * M + m] = sc;
    }
  } else {
    fp8_store8(out, at, v, some, out_dtype);
  }
}

hipError_t launch_finish(const float* part, int S, int M, int N, bool glu, void* out, int out_dtype, float* out_scales,
                         hipStream_t s) {
  const int chunks = ceil_div(N, 512);
  const dim3 grid((unsigned)(((size_t)M * chunks + 3) / 4));
  if (glu) hipLaunchKernelGGL(fp8_finish_kernel<true>, grid, dim3(256), 0, s, part, S, M, N, out, out_dtype, out_scales, chunks);
  else hipLaunchKernelGGL(fp8_finish_kernel<false>, grid, dim3(256), 0, s, part, S, M, N, out, out_dtype, out_scales, chunks);
  return hipGetLastError();
}

// ---- which kernel ----

constexpr int kRows[] = {16, 32, 64, 128, 256};  // rows of x of a kind's tile (STREAM, LOW, MID, HALF, WHOLE)
constexpr int kCols[] = {16, 128, 128, 256, 256};

// W4A16_FP8_ROWS=16|32|64|128|256 pins the row tile (for benchmarking one against another); read once
// per process.
int forced_kind() {
  static const int forced = [] {
    const char* v = getenv("W4A16_FP8_ROWS");
    if (!v) return -1;
    for (int j = 0; j < 5; ++j)
      if (atoi(v) == kRows[j]) return j;
    return -1;
  }();
  return forced;
}

struct Plan {
  int kind;
  int S;     // slices of k, added by a second kernel
  int pair;  // 2: two groups of waves share a workgroup's slice
};

// us of a product on tiles of a kind with k in S slices: 3 and, for each round of workgroups, the blocks of k by what
// one takes, and 1.5 more a round; at least the weight's bytes at 5.6 TB/s; and the slices' sums, written and read at
// 4 TB/s with another launch. What a block takes was measured on 1024x4096 to 8192x32768, 24 to 2048 rows, S 1 to
// 12, cold weights: `one` with few workgroups, `full` with one on every compute unit, `pair` with two on each (the kinds
// of which two fit), or in later rounds. With two groups of waves to a workgroup (pair) each takes every second block, at
// the pair's time (333 rows of 2896x5001 in fp32, 240 tiles of 64 rows: 27.7 us with one group, 23.8 with two).
struct BlockTimes {
  double one, full, pair;
};
constexpr BlockTimes kBlock[2][5] = {{{}, {0.42, 0.52, 0.85}, {0.50, 0.66, 0.83}, {0.82, 0.95, 1.02}, {1.60, 1.68, 1.70}},
                                     {{}, {0.56, 0.66, 0.95}, {0.78, 0.92, 1.15}, {1.60, 1.75, 1.82}, {}}};
// whether a product's last round of tiles runs as halves of them, all at once
bool halved(int kind, int S, long long tiles, long long cus) {
  const long long left = tiles % cus;
  return kind == WHOLE && S == 1 && tiles > cus && left && 2 * left <= cus;
}
double model_us(int kind, int S, int pair, int M, int N, int KB, bool exact, long long cus) {
  const long long wgs = (long long)ceil_div(M, kRows[kind]) * ceil_div(N, kCols[kind]) * S;
  const int steps = ceil_div(ceil_div(KB, S), pair);
  const BlockTimes& b = kBlock[exact][kind];
  const long long slots = kind <= MID ? 2 * cus : cus;
  double t = 3;
  if (pair > 1) {
    t += 1 + (double)((wgs + cus - 1) / cus) * steps * b.pair + 1.5 * (double)((wgs - 1) / cus);
  } else if (wgs <= cus) {
    t += steps * (b.one + (b.full - b.one) * wgs / cus);
  } else {
    double rounds = (double)((wgs + slots - 1) / slots);
    if (halved(kind, S, wgs, cus)) rounds -= 0.4;
    t += rounds * steps * b.pair + 1.5 * (rounds - 1);
  }
  const double memory = 3 + (double)N * KB * 128 / 5.6e6;
  if (t < memory) t = memory;
  if (S > 1) t += 4.5 + 2.0 * S * M * N * 4 / 4e6;
  return t;
}

// us of 17 to 32 rows by the sixteen-row products' kernel, eight waves to a workgroup and one workgroup to a compute
// unit: a round of 16 or 32 columns by what each of a wave's blocks takes (20 rows of 4096x4096: 7.6 us, by tiles 11.7;
// of 2048x7168 7.5 and 10.5; of 8192x8192 18.4 and 20.7; of 4096x14336 20.9 and 17.8). N: columns of out
double stream32_us(int N, int KB, bool glu, long long cus, int& NT) {
  const auto us = [&](int cols, double block) {
    const long long rounds = (ceil_div(N, cols) + cus - 1) / cus;
    return 3 + rounds * ceil_div(KB, 8) * block + 1.5 * (rounds - 1);
  };
  const double narrow = glu ? 1e30 : us(16, 1.05), two = us(glu ? 16 : 32, 1.95);
  NT = narrow <= two ? 1 : 2;
  return narrow <= two ? narrow : two;
}

// Whether so many tiles leave at most an eighth of the chip idle. Of three to sixteen rows such a weight is read faster by
// tiles of 32 rows, which ask for 128 of its rows at once (16 rows of 8192x28672 37.7 us, by sixteen columns 45.3; of
// 8192x57344 72.4 and 77.1; of 4096x28672 25.1 and 27.9; but with 192 tiles, 8192x24576, 36.9 and 33.3, and with 320,
// 8192x40960, 59.6 and 52.0). One row or two are quantized on the way by the other kernel.
bool fills(long long tiles, long long cus) { return 8 * tiles >= 7 * ((tiles + cus - 1) / cus) * cus; }

Plan choose(int M, int N, int K, bool glu, bool exact, bool w_rows = false) {
  // N: columns that are multiplied (GLU: both halves)
  const int KB = (int)fp8_blocks(K);
  if (forced_kind() >= 0 && !(exact && forced_kind() == WHOLE) && !(w_rows && forced_kind() == STREAM)) return Plan{forced_kind(), 1, 1};
  if (M <= 2 && !w_rows) return Plan{STREAM, 1, 1};
  const long long cus = device_cu_count();
  if (M <= 16 && !w_rows) return Plan{fills(ceil_div(N, 128), cus) ? LOW : STREAM, 1, 1};
  const bool sliced = !glu || (N / 2) % 128 == 0;  // sums of both halves as plain columns: their blocks follow each other
  Plan best{MID, 1, 1};
  double least = 1e30;
  if (M <= 32 && !w_rows) {
    int NT;
    least = stream32_us(glu ? N / 2 : N, KB, glu, cus, NT);
    best = Plan{STREAM, 1, 1};
  }
  for (int kind = LOW; kind <= (exact ? HALF : WHOLE); ++kind)
    for (int S = 1; S <= (sliced ? 12 : 1); ++S) {
      if (S > 1 && KB < 4 * S) break;
      for (int pair = 1; pair <= (kind <= MID && KB >= 4 * S ? 2 : 1); ++pair) {
        const double t = model_us(kind, S, pair, M, N, KB, exact, cus);
        if (t < least * 0.999) {
          least = t;
          best = Plan{kind, S, pair};
        }
      }
    }
  return best;
}

// The plan of a dense product, by its columns of out: what sizes its scratch, makes its operands and launches it all ask this
Plan plan_of(int M, int N, int K, bool glu, int out_dtype, bool w_rows = false) {
  return choose(M, glu ? 2 * N : N, K, glu, out_dtype >= 2, w_rows);
}

TileParams tile_params(const Fp8Args& a) {
  TileParams p{};
  p.x = a.x;
  p.xs = a.xs;
  p.w = a.w;
  p.ws = a.ws;
  p.out = a.out;
  p.out_scales = a.out_scales;
  p.out_dtype = a.out_dtype;
  p.M = a.M;
  p.N = a.N;
  p.K = a.K;
  p.KB = p.slice = (int)fp8_blocks(a.K);
  p.ldk = a.ldk;
  p.xs_ld = a.xs_ld;
  p.up_blocks = (int)fp8_blocks(a.N);
  p.scale_rows = a.M;
  p.once = (long long)p.N * (a.glu ? 2 : 1) * p.K >= kOnceBytes;
  return p;
}

void set_tiles(TileParams& p, int kind, bool glu, int tiles_m) {
  p.tiles_m = tiles_m;
  p.tiles_n = ceil_div(p.N, glu ? kCols[kind] / 2 : kCols[kind]);
  p.count = p.tiles_m * p.tiles_n;
  // blocks of k in turn where the workgroups fill the chip (64 rows of 8192x57344 96.6 -> 87.7 us, of 4096x32768 35.8 -> 32.1;
  // of 4096x14336, 112 workgroups, 24.1 -> 25.0)
  p.turn = 4LL * p.tiles_m * p.tiles_n >= 3 * device_cu_count();
}

// Sixteen-row products: eight waves share k where the workgroups are few (up to two a compute unit), else four;
// 32 columns a workgroup where 16 would make many, and for more than eight rows over a deep K, whose x no
// cache near the compute unit holds. us by (columns, waves), 16/4, 16/8, 32/4, 32/8, one row and sixteen rows:
//   4096x4096   8.5, 6.2, 9.7, 7.3;   8.2, 6.2, 10.4, 7.9    8192x10240  18.6, 19.2, 20.7, 24.2;  20.1, 22.1, 22.4, 25.3
//   4096x14336  13.6, 15.1, 13.8, 16.9;  15.7, 17.0, 14.7, 17.8    14336x4096  24.8, 15.3, 28.5, 18.0;  23.5, 14.8, 30.7, 19.7
//   28672x8192  53.4, 42.0, 57.6, 42.0;  51.1, 50.0, 64.1, 42.8
void stream_shape(int M, int N, int K, bool glu, long long cus, int& NT, int& W) {
  const long long tiles = ceil_div(N, 16);
  NT = glu || tiles > 3 * cus || (M > 8 && K > 16384) ? 2 : 1;
  W = ceil_div(N, glu ? 16 : 16 * NT) <= 2 * cus ? 8 : 4;
}

hipError_t launch_rows16(const TileParams& t, bool glu, const void* values, int values_dtype, hipStream_t s) {
  StreamParams p{};
  p.x = t.x;
  p.xs = t.xs;
  p.w = t.w;
  p.ws = t.ws;
  p.out = t.out;
  p.out_dtype = t.out_dtype;
  p.M = t.M;
  p.N = t.N;
  p.K = t.K;
  p.KB = t.KB;
  p.ldk = t.ldk;
  p.xs_ld = t.xs_ld;
  p.up_blocks = t.up_blocks;
  p.once = t.once;
  p.values = values;
  p.values_dtype = values_dtype;
  int NT, W;
  const int XC = values ? 0 : t.M > 16 ? 4 : t.M > 8 ? 2 : 1;
  p.tiles_m = ceil_div(t.M, XC == 4 ? 32 : 16);
  stream_shape(t.M, t.N, t.K, glu, device_cu_count(), NT, W);
  if (XC == 4) stream32_us(t.N, t.KB, glu, device_cu_count(), NT), W = 8;
  p.tiles_n = ceil_div(t.N, glu ? 8 * NT : 16 * NT);
  p.slice = ceil_div(t.KB, W);
  const unsigned grid = (unsigned)((size_t)p.tiles_m * p.tiles_n);
  return launch_stream(p, NT, XC, W, glu, grid, s);
}

// Workgroups of a launch of so many tiles: with one a compute unit, each takes its share of the tiles in turn
unsigned workgroups(int kind, long long tiles) {
  const long long cus = device_cu_count();
  return (unsigned)(kind == HALF && tiles > cus ? cus : tiles);
}

bool grid_fits(long long tiles_m, int N, int kind, bool glu, int S) {
  const long long cols = kind == STREAM ? 16 : kCols[kind] / (glu ? 2 : 1);
  return tiles_m * ((N + cols - 1) / cols) * 512 * S < (1LL << 32);
}

// h of a swiglu product in e4m3 is quantized by the HALF tiles themselves (128 columns of h each); else from fp32
bool by_finish(int kind, int S, int out_dtype) { return S > 1 || (out_dtype == kE4M3 && kind != HALF); }

}  // namespace

namespace {
// the grid of the second kernel
bool finish_fits(int M, int N) { return (long long)M * ceil_div(N, 512) < (1LL << 25); }
}  // namespace

bool fp8_fits(int M, int N, int K, bool glu, int out_dtype, bool w_rows) {
  // offsets within a tile's operands, and of scales, in 31 bits; fewer than 2^32 threads
  const long long wrows = glu ? 2LL * N : 256;
  if ((long long)K >= (1LL << 23) || wrows * K >= (1LL << 31)) return false;
  if ((long long)fp8_blocks(K) * M * 4 >= (1LL << 31) || (long long)(fp8_blocks(N) + 1) * 2 * fp8_blocks(K) * 4 >= (1LL << 31))
    return false;
  // on any tile
  if ((long long)ceil_div(M, 16) * ceil_div(glu ? 2 * N : N, 16) * 512 * 12 < (1LL << 32) && finish_fits(M, N)) return true;
  const Plan c = plan_of(M, N, K, glu, out_dtype, w_rows);
  return grid_fits(ceil_div(M, kRows[c.kind]), N, c.kind, glu, c.S) && (!by_finish(c.kind, c.S, out_dtype) || finish_fits(M, N));
}

// One or two rows of 16 bits: each workgroup quantizes the groups that its waves multiply, which saves a launch and its
// scratch. More rows' groups would take as long as the weight does to arrive.
bool fp8_takes_values(int M, int N, int K, bool glu, int out_dtype) {
  if (M > 2 || M < 1 || plan_of(M, N, K, glu, out_dtype).kind != STREAM) return false;
  int NT, W;
  stream_shape(M, N, K, glu, device_cu_count(), NT, W);
  return ceil_div((int)fp8_blocks(K), W) * M <= 64;
}

size_t fp8_scratch_bytes(int M, int N, int K, bool glu, int out_dtype, bool w_rows) {
  const Plan c = plan_of(M, N, K, glu, out_dtype, w_rows);
  if (c.S > 1) return align256((size_t)c.S * M * (glu ? 2 * (size_t)N : N) * 4);
  return by_finish(c.kind, c.S, out_dtype) ? align256((size_t)M * N * 4) : 0;
}

const char* fp8_name(int M, int N, int K, bool glu) {
  const Plan c = choose(M, glu ? 2 * N : N, K, glu, false);
  static const char* const names[2][5] = {
      {"w4a16_fp8_16", "w4a16_fp8_32x128", "w4a16_fp8_64x128", "w4a16_fp8_128x256", "w4a16_fp8_256x256"},
      {"w4a16_fp8_32", "w4a16_fp8_32x128_splitk", "w4a16_fp8_64x128_splitk", "w4a16_fp8_128x256_splitk", "w4a16_fp8_256x256_splitk"}};
  return names[c.kind == STREAM ? M > 16 : c.S > 1][c.kind];
}

hipError_t launch_fp8(const Fp8Args& a) {
  const bool exact = a.out_dtype >= 2;
  const Plan c = plan_of(a.M, a.N, a.K, a.glu, a.out_dtype, a.w_rows);
  if (a.values && c.kind != STREAM) return hipErrorInvalidValue;  // (tiles read codes)
  TileParams p = tile_params(a);
  const bool finish = by_finish(c.kind, c.S, a.out_dtype);
  if (finish) {
    p.out = a.scratch;
    p.out_dtype = 2;
  }
  hipError_t e;
  if (c.kind == STREAM) {
    e = launch_rows16(p, a.glu, a.values, a.values_dtype, a.stream);
  } else {
    const bool glu = a.glu && c.S == 1;
    if (a.glu && !glu) p.N = 2 * a.N;
    const int kind = c.kind;
    set_tiles(p, kind, glu, ceil_div(a.M, kRows[kind]));
    p.slice = ceil_div(p.KB, c.S);
    p.pair = c.pair > 1;
    const auto launch = a.w_rows ? launch_columns : glu ? launch_glu : fp8::launch_dense;
    const long long tiles = (long long)p.tiles_m * p.tiles_n, cus = device_cu_count(), left = tiles % cus;
    if (halved(kind, c.S, tiles, cus)) {
      // the last round fills half the chip at most: its tiles run as halves, all at once
      p.first = (int)(tiles - left);
      TileParams whole = p;
      whole.first = 0;
      whole.count = p.first;
      e = launch(whole, WHOLE, exact, workgroups(WHOLE, p.first), 1, a.stream);
      if (e != hipSuccess) return e;
      e = launch(p, HALF, exact, workgroups(HALF, 2 * left), 1, a.stream);
    } else {
      e = launch(p, kind, exact, c.S > 1 ? (unsigned)tiles : workgroups(kind, tiles), c.S, a.stream);
    }
  }
  if (e != hipSuccess || !finish) return e;
  return launch_finish(a.scratch, c.S, a.M, a.N, a.glu && c.S > 1, a.out, a.out_dtype, a.out_scales, a.stream);
}

// ---- grouped ----

namespace {

// The rows of each group are known on the device only, so the tile goes by their mean over the groups that can have rows.
// us of 32, 64 and 128 rows a tile, plain results in bf16, random groups: 16 groups of 2048x1408 with a mean of 24 13.3,
// 12.3, 13.8; of 48 12.9, 12.8, 15.2; of 96 19.5, 16.1, 17.4; of 128 23.6, 20.8, 19.2; of 384 54.7, 44.9, 35.7. 8 groups of
// 4096x2048: 14.5, 14.8, 17.3; 16.5, 15.8, 19.0; 26.8, 20.5, 21.4; 33.8, 28.7, 22.8; 72.6, 56.2, 45.5 (tiles of 256 rows 62.3:
// a group's last tile is half empty more often, and nothing hides its first blocks). The kernel of sixteen rows is
// slower for the fewest rows too (32 tokens through two of 8 experts of 4096x14336: 254 us, tiles of 32 rows 226).
int choose_grouped(const RouteLayout& r) {
  if (forced_kind() >= 0) return forced_kind() < LOW ? LOW : forced_kind() > HALF ? HALF : forced_kind();
  const int groups = r.E < r.S ? r.E : r.S;
  const int mean = r.S / (groups > 0 ? groups : 1);
  return mean <= 24 ? LOW : mean <= 100 ? MID : HALF;
}

// (the plan's lists have 16, 32, 64 and 128 rows a tile: LOW's is list LOW, and so on)

GroupTiles group_tiles(const RouteLayout& r, const int32_t* plan, bool gather, int list) {
  GroupTiles t;
  t.plan = plan;
  t.E = r.E;
  t.token = r.token;
  t.list = r.tiles[list];
  t.bound = tile_bound(r.S, r.E, list);
  t.tokens = gather ? r.S / r.topk : 0;
  return t;
}

}  // namespace

bool fp8_grouped_fits(const RouteLayout& r, int N, int K, bool glu, int out_dtype) {
  const long long wrows = glu ? 2LL * N : 256;
  if ((long long)K >= (1LL << 23) || wrows * K >= (1LL << 31)) return false;
  if ((long long)fp8_blocks(K) * r.S * 4 >= (1LL << 31) || (long long)(fp8_blocks(N) + 1) * 2 * fp8_blocks(K) * 4 >= (1LL << 31))
    return false;
  const int kind = choose_grouped(r);
  if (by_finish(kind, 1, out_dtype) && !finish_fits(r.S, N)) return false;
  return grid_fits(tile_bound(r.S, r.E, kind), N, kind, glu, 1);
}

size_t fp8_grouped_scratch_bytes(const RouteLayout& r, int N, int out_dtype) {
  if (!by_finish(choose_grouped(r), 1, out_dtype)) return 0;
  return align256((size_t)r.S * N * 4);
}

hipError_t launch_fp8_grouped(const Fp8Args& a, const RouteLayout& r, const int32_t* plan, bool gather) {
  const bool exact = a.out_dtype >= 2;
  const int kind = choose_grouped(r);
  TileParams p = tile_params(a);
  p.M = p.scale_rows = r.S;
  p.once = (long long)a.N * (a.glu ? 2 : 1) * a.K * (r.E < r.S ? r.E : r.S) >= kOnceBytes;  // of the groups that can have rows
  p.groups = group_tiles(r, plan, gather, kind);
  const bool finish = by_finish(kind, 1, a.out_dtype);
  if (finish) {
    p.out = a.scratch;
    p.out_dtype = 2;
  }
  set_tiles(p, kind, a.glu, p.groups.bound);
  const auto launch = a.glu ? launch_grouped_glu : launch_grouped_plain;
  const hipError_t e = launch(p, kind, exact, workgroups(kind, (long long)p.tiles_m * p.tiles_n), 1, a.stream);
  if (e != hipSuccess || !finish) return e;
  return launch_finish(a.scratch, 1, r.S, a.N, false, a.out, a.out_dtype, a.out_scales, a.stream);
}

hipError_t launch_fp8_by_group(const Fp8Args& a, const RouteLayout& r, const int32_t* plan) {
  TileParams p = tile_params(a);
  p.groups = group_tiles(r, plan, false, kTileLists - 1);
  // tall tiles where they still fill the chip
  const long long tall = (long long)ceil_div(a.M, kRows[HALF]) * ceil_div(a.N, kCols[HALF]) * r.E;
  const int kind = tall >= device_cu_count() ? HALF : MID;
  set_tiles(p, kind, false, ceil_div(a.M, kRows[kind]));
  const long long tiles = (long long)p.tiles_m * p.tiles_n;  // (a group's; of all groups fewer than 2^31, as dw would not fit otherwise)
  const bool looping = kind == HALF;
  return launch_by_group(p, kind, true, looping ? workgroups(kind, tiles * r.E) : (unsigned)tiles, looping ? 1 : r.E, a.stream);
}

}  // namespace w4a16
