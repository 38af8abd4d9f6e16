// w4a16_dispatch.hip - rows moved into sorted order and back, with their gradients, by the plan
// of w4a16_route.
//
//   dispatch            xs[p] = x[order[p] / topk]                       (0 past the last group)
//   combine             y[t]  = sum_j w[t][j] ys[slot[t][j]]             (fp32, j ascending)
//   combine, w == 1     dx[t] = sum_j dxs[slot[t][j]]                    (dispatch's gradient)
//   combine_backward    dys[slot[t][j]] = w[t][j] dy[t],  dw[t][j] = <dy[t], ys[slot[t][j]]>
//
// A slot of no group adds nothing, whatever its weight and row hold. All are bound by HBM: every
// kernel goes over the tokens, so that a token's own row is read or written once and its topk
// sorted rows once each; no row is read twice and nothing is added with atomics. A wave takes 2 KiB
// of a token's row (two 16-byte accesses per lane and sorted row), so the slots and weights of
// its token are wave-uniform. Rows of a width that is no multiple of 16 bytes start at any
// element: the vectors are declared with the element's alignment, which global accesses of
// this GPU take as they are.
//
// Measured from cold, against a copy of a large tensor at 5.2 TB/s (bf16): 8192 tokens x 4096 to two rows
// each and back 71 us with the sort (389 MB); 16384 x 2048, eight rows each, with all gradients 557 us
// (2953 MB, 5.3 TB/s); 4099 x 2885, three rows each, whose vectors cross cache lines, dispatch and combine 20
// us each, gradients 40 (4.7 and 4.1 TB/s; with a fifth of the slots dropped 21, 18 and 38, and 16, 16 and 32 for
// rows of 2880). fp32 rows of 8192 x 4096, two each, combined to fp32 64 us, to bf16 55 (6.1 TB/s, although a lane then
// stores its four elements one by one).
#include <limits.h>

#include "w4a16_device.hpp"
#include "w4a16_routed.hpp"

namespace w4a16 {

namespace {

enum { T_F16 = 0, T_BF16 = 1, T_F32 = 2 };
enum { NARROW = 0, CACHED = 1, STREAM = 2, STREAM_LINES = 3 };

typedef u4_t u4_any_t __attribute__((aligned(2)));  // sixteen bytes at any element's address

template <int T>
struct Elem {
  typedef uint16_t raw;
  static constexpr int kVec = 8;  // elements in 16 bytes
};
template <>
struct Elem<T_F32> {
  typedef uint32_t raw;
  static constexpr int kVec = 4;
};

template <int T>
__device__ __forceinline__ float elem_value(typename Elem<T>::raw b) {
  if constexpr (T == T_F16) return (float)__builtin_bit_cast(_Float16, b);
  if constexpr (T == T_BF16) return __builtin_bit_cast(float, (uint32_t)b << 16);
  if constexpr (T == T_F32) return __builtin_bit_cast(float, b);
}
template <int T>
__device__ __forceinline__ typename Elem<T>::raw elem_bits(float v) {  // one rounding, to nearest even
  if constexpr (T == T_F16) return __builtin_bit_cast(uint16_t, (_Float16)v);
  if constexpr (T == T_BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
  if constexpr (T == T_F32) return __builtin_bit_cast(uint32_t, v);
}

// element i of a loaded vector
template <int T>
__device__ __forceinline__ float vec_value(u4_t v, int i) {
  if constexpr (T == T_F32)
    return elem_value<T>(v[i]);
  else
    return elem_value<T>((uint16_t)(v[i >> 1] >> (16 * (i & 1))));
}
template <int T>
__device__ __forceinline__ u4_t vec_pack(const float* f) {
  u4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (T == T_F32)
      v[i] = elem_bits<T>(f[i]);
    else
      v[i] = (uint32_t)elem_bits<T>(f[2 * i]) | (uint32_t)elem_bits<T>(f[2 * i + 1]) << 16;
  }
  return v;
}

// Vector c of a row of `width` elements starts at its element c V. The last one, where the width is
// no multiple of V, is moved back to end with the row: its first elements are then its
// neighbour's too, who reads and writes the same values. (Taken one by one, the last elements
// made the sort, the two moves and their gradients of 4099 bf16 tokens of 2885 elements, topk 3,
// take 133 us; moved back, 112.) Vectors past the row read its last one and store nothing, so that
// loads need no branch: the compiler puts a wait for all that is in flight before a load under
// one.
//
// Rows come in four modes. NARROW: shorter than a vector, taken element by element. CACHED.
// STREAM: the sorted rows take 64 MiB or more (kStreamBytes), a quarter of the last-level cache, and
// stores are non-temporal; STREAM_LINES: also the loads of the sorted rows, where these are whole
// cache lines (shared lines would be fetched twice).
template <int T>
__device__ __forceinline__ int vec_at(int c, int width) {
  return min(c * Elem<T>::kVec, width - Elem<T>::kVec);
}
// ONCE: the row is read for the last time
template <int T, int MODE, bool ONCE>
__device__ __forceinline__ u4_t load_vec(const typename Elem<T>::raw* row, int c, int width) {
  if constexpr (MODE != NARROW) {
    const u4_any_t* const at = reinterpret_cast<const u4_any_t*>(row + vec_at<T>(c, width));
    return ONCE && MODE == STREAM_LINES ? __builtin_nontemporal_load(at) : *at;
  }
  u4_t v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < Elem<T>::kVec - 1; ++i) {
    if (c > 0 || i >= width) continue;
    if constexpr (T == T_F32)
      v[i] = row[i];
    else
      v[i >> 1] |= (uint32_t)row[i] << (16 * (i & 1));
  }
  return v;
}
template <int T, int MODE>
__device__ __forceinline__ void store_vec(typename Elem<T>::raw* row, int c, int width, u4_t v) {
  if (c * Elem<T>::kVec >= width) return;
  if constexpr (MODE != NARROW) {
    u4_any_t* const at = reinterpret_cast<u4_any_t*>(row + vec_at<T>(c, width));
    if constexpr (MODE >= STREAM)
      __builtin_nontemporal_store(v, at);
    else
      *at = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < Elem<T>::kVec - 1; ++i) {
    if (i >= width) continue;
    if constexpr (T == T_F32)
      row[i] = v[i];
    else
      row[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
  }
}

constexpr int kRowWaves = 4;     // waves per workgroup, each with an item of its own
constexpr int kRowVecs = 2;      // vectors per lane and row, 2 KiB of a row per item; one for shorter rows than 1 KiB
constexpr int kTailWaves = 512;  // waves that clear the rows past the last group

struct RowParams {
  const void *x, *ys;
  void* out;
  const float* weights;
  float* dweights;
  const int32_t* plan;
  int S, E, topk, slot;
  int tokens, width;
  int vecs;        // vectors per lane and row: kRowVecs or 1
  int segs;        // items per token
  int tail_waves;  // waves after the items
};

// rows [offsets[E], S) of `rows` cleared by waves w, w + waves, ...
template <int T, int MODE>
__device__ __forceinline__ void clear_tail(const RowParams& p, void* rows, int w, int waves, int lane) {
  const int vecs = (p.width + Elem<T>::kVec - 1) / Elem<T>::kVec;
  for (int row = p.plan[p.E] + w; row < p.S; row += waves)
    for (int c = lane; c < vecs; c += 64)
      store_vec<T, MODE>(static_cast<typename Elem<T>::raw*>(rows) + (size_t)row * p.width, c, p.width, u4_t{0, 0, 0, 0});
}

template <int T, int MODE, int U>
__global__ __launch_bounds__(64 * kRowWaves) void dispatch_kernel(RowParams p) {
  typedef typename Elem<T>::raw raw;
  const int lane = threadIdx.x & 63;
  const int item = __builtin_amdgcn_readfirstlane(blockIdx.x * kRowWaves + (threadIdx.x >> 6));
  const int items = p.tokens * p.segs;
  if (item >= items) {
    if (item < items + p.tail_waves) clear_tail<T, MODE>(p, p.out, item - items, p.tail_waves, lane);
    return;
  }
  const int t = item / p.segs, c0 = (item - t * p.segs) * 64 * U + lane;
  const raw* src = static_cast<const raw*>(p.x) + (size_t)t * p.width;
  u4_t v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) v[u] = load_vec<T, MODE, false>(src, c0 + 64 * u, p.width);
  const int32_t* slot = p.plan + p.slot + (size_t)t * p.topk;
  for (int j = 0; j < p.topk; ++j) {
    const int row = slot[j];
    if (row < 0) continue;
    raw* dst = static_cast<raw*>(p.out) + (size_t)row * p.width;
#pragma unroll
    for (int u = 0; u < U; ++u) store_vec<T, MODE>(dst, c0 + 64 * u, p.width, v[u]);
  }
}

// The sorted rows and weights of choices j0 .. j0 + J - 1 of a token, all read at once: row -1 for
// slots of no group and past the last choice
template <int J>
__device__ __forceinline__ void load_choices(const RowParams& p, int t, int j0, int (&row)[J], float (&w)[J]) {
  const int32_t* slot = p.plan + p.slot + (size_t)t * p.topk;
  // no weights: any words there are, and 1
  const float* weight = p.weights ? p.weights + (size_t)t * p.topk : reinterpret_cast<const float*>(slot);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int at = min(j0 + j, p.topk - 1);
    row[j] = slot[at];
    w[j] = weight[at];
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    row[j] = j0 + j < p.topk ? row[j] : -1;
    w[j] = p.weights ? w[j] : 1.0f;
  }
}

// J: sorted rows in flight. A choice of no row reads row 0 and adds nothing.
template <int T, int TO, int J, int MODE, int U>
__global__ __launch_bounds__(64 * kRowWaves) void combine_kernel(RowParams p) {
  typedef typename Elem<T>::raw raw;
  constexpr int V = Elem<T>::kVec;
  const int lane = threadIdx.x & 63;
  const int item = __builtin_amdgcn_readfirstlane(blockIdx.x * kRowWaves + (threadIdx.x >> 6));
  if (item >= p.tokens * p.segs) return;
  const int t = item / p.segs, c0 = (item - t * p.segs) * 64 * U + lane;
  float acc[U][V];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[u][i] = 0.f;
  for (int j0 = 0; j0 < p.topk; j0 += J) {
    u4_t v[J][U];
    int row[J];
    float w[J];
    load_choices(p, t, j0, row, w);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const raw* src = static_cast<const raw*>(p.ys) + (size_t)max(row[j], 0) * p.width;
#pragma unroll
      for (int u = 0; u < U; ++u) v[j][u] = load_vec<T, MODE, true>(src, c0 + 64 * u, p.width);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (row[j] < 0) continue;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[u][i] = __builtin_fmaf(w[j], vec_value<T>(v[j][u], i), acc[u][i]);
    }
  }
  typedef typename Elem<TO>::raw out_raw;
  out_raw* dst = static_cast<out_raw*>(p.out) + (size_t)t * p.width;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if constexpr (Elem<TO>::kVec == V) {
      store_vec<TO, MODE>(dst, c0 + 64 * u, p.width, vec_pack<TO>(acc[u]));
    } else {  // fp32 rows to 16-bit tokens: a lane's four elements are half a vector
#pragma unroll
      for (int i = 0; i < V; ++i)
        if ((c0 + 64 * u) * V < p.width && (MODE != NARROW || i < p.width))
          dst[(MODE == NARROW ? 0 : vec_at<T>(c0 + 64 * u, p.width)) + i] = elem_bits<TO>(acc[u][i]);
    }
  }
}

// PER waves share a token: the products of dy with the token's sorted rows are summed per lane, then
// over the lanes and waves in a fixed order. Four waves, or one for rows up to 2 KiB, which leave most of
// four idle (30000 tokens x 160 bf16, topk 8: 138 -> 61 us).
template <int T, int J, int MODE, int PER>
__global__ __launch_bounds__(64 * kRowWaves) void combine_backward_kernel(RowParams p) {
  typedef typename Elem<T>::raw raw;
  constexpr int V = Elem<T>::kVec, TOKENS = kRowWaves / PER;  // tokens of a workgroup
  __shared__ float part[kRowWaves][J];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = (p.tokens + TOKENS - 1) / TOKENS;
  if ((int)blockIdx.x >= blocks) {  // the workgroups after the tokens'
    clear_tail<T, MODE>(p, p.out, (blockIdx.x - blocks) * kRowWaves + wave, p.tail_waves, lane);
    return;
  }
  const int t = blockIdx.x * TOKENS + (PER == 1 ? wave : 0);
  if (PER == 1 && t >= p.tokens) return;
  const int first = PER == 1 ? lane : threadIdx.x;
  const int vecs = (p.width + V - 1) / V;
  const raw* dy = static_cast<const raw*>(p.x) + (size_t)t * p.width;
  for (int j0 = 0; j0 < p.topk; j0 += J) {
    int row[J];
    float w[J], acc[J];
    load_choices(p, t, j0, row, w);
#pragma unroll
    for (int j = 0; j < J; ++j) acc[j] = 0.f;
    for (int c = first; c < vecs; c += 64 * PER) {
      const u4_t d = load_vec<T, MODE, false>(dy, c, p.width);
      u4_t v[J];
#pragma unroll
      for (int j = 0; j < J; ++j)
        v[j] = load_vec<T, MODE, true>(static_cast<const raw*>(p.ys) + (size_t)max(row[j], 0) * p.width, c, p.width);
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = vec_value<T>(d, i);
      // a last vector that was moved back: its neighbour's elements are not summed again
      const int again = MODE == NARROW ? 0 : c * V - vec_at<T>(c, p.width);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (row[j] < 0) continue;
        float g[V];
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = w[j] * f[i];
        if (again == 0) {
#pragma unroll
          for (int i = 0; i < V; ++i) acc[j] = __builtin_fmaf(f[i], vec_value<T>(v[j], i), acc[j]);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (i >= again) acc[j] = __builtin_fmaf(f[i], vec_value<T>(v[j], i), acc[j]);
        }
        store_vec<T, MODE>(static_cast<raw*>(p.out) + (size_t)row[j] * p.width, c, p.width, vec_pack<T>(g));
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) acc[j] += __shfl_xor(acc[j], o);
    if constexpr (PER > 1) {
      if (j0) __syncthreads();  // the sums of the choices before have been read
      if (lane == 0)
#pragma unroll
        for (int j = 0; j < J; ++j) part[wave][j] = acc[j];
      __syncthreads();
      if (threadIdx.x < J && j0 + threadIdx.x < p.topk) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) s += part[i][threadIdx.x];
        p.dweights[(size_t)t * p.topk + j0 + threadIdx.x] = s;
      }
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (lane == j && j0 + j < p.topk) p.dweights[(size_t)t * p.topk + j0 + j] = acc[j];
    }
  }
}

RowParams row_params(const RouteLayout& r, const int32_t* plan, int width, int vec) {
  RowParams p = {};
  p.plan = plan;
  p.S = r.S;
  p.E = r.E;
  p.topk = r.topk;
  p.slot = r.slot;
  p.tokens = r.S / r.topk;
  p.width = width;
  p.vecs = width <= 64 * vec ? 1 : kRowVecs;
  p.segs = ceil_div(width, 64 * p.vecs * vec);
  p.tail_waves = r.S < kTailWaves ? r.S : kTailWaves;
  return p;
}

}  // namespace

bool rows_fit(int tokens, int width) {
  // an item's last lanes index up to 1023 elements past the row before they are held back to it
  if (width > INT_MAX - 1023) return false;
  // a wave per token and 512 elements at most (fp32), a workgroup per token in the backward pass
  const long long waves = (long long)tokens * ceil_div(width, 64 * kRowVecs * 4) + kTailWaves;
  return waves < (1LL << 26) && ((long long)tokens + kTailWaves) * 64 * kRowWaves < (1LL << 32);
}

template <int T>
static int row_mode(const RowParams& p) {
  constexpr size_t bytes = sizeof(typename Elem<T>::raw);
  if (p.width < Elem<T>::kVec) return NARROW;
  if (p.S * (size_t)p.width * bytes < kStreamBytes) return CACHED;
  return p.width * bytes % 128 ? STREAM : STREAM_LINES;
}

template <int T, int MODE>
static void launch_dispatch_m(const RowParams& p, dim3 grid, hipStream_t s) {
  if (p.vecs == 1)
    hipLaunchKernelGGL((dispatch_kernel<T, MODE, 1>), grid, dim3(64 * kRowWaves), 0, s, p);
  else
    hipLaunchKernelGGL((dispatch_kernel<T, MODE, kRowVecs>), grid, dim3(64 * kRowWaves), 0, s, p);
}
template <int T>
static void launch_dispatch_t(const RowParams& p, dim3 grid, hipStream_t s) {
  switch (row_mode<T>(p)) {
    case NARROW: hipLaunchKernelGGL((dispatch_kernel<T, NARROW, 1>), grid, dim3(64 * kRowWaves), 0, s, p); break;
    case CACHED: launch_dispatch_m<T, CACHED>(p, grid, s); break;
    default: launch_dispatch_m<T, STREAM>(p, grid, s);
  }
}

hipError_t launch_dispatch(const void* x, const RouteLayout& r, const int32_t* plan, int width, int dtype,
                           void* xs, hipStream_t s) {
  RowParams p = row_params(r, plan, width, dtype == T_F32 ? 4 : 8);
  p.x = x;
  p.out = xs;
  const dim3 grid(ceil_div(p.tokens * p.segs + p.tail_waves, kRowWaves));
  if (dtype == T_F32)
    launch_dispatch_t<T_F32>(p, grid, s);
  else  // a copy: the 16-bit types are alike
    launch_dispatch_t<T_F16>(p, grid, s);
  return hipGetLastError();
}

template <int T, int TO, int J, int MODE>
static void launch_combine_j(const RowParams& p, dim3 grid, hipStream_t s) {
  if (p.vecs == 1)
    hipLaunchKernelGGL((combine_kernel<T, TO, J, MODE, 1>), grid, dim3(64 * kRowWaves), 0, s, p);
  else
    hipLaunchKernelGGL((combine_kernel<T, TO, J, MODE, kRowVecs>), grid, dim3(64 * kRowWaves), 0, s, p);
}
// Choices past the last read a row again, so five and six are taken by threes
static int rows_in_flight(int topk) { return topk <= 4 ? topk : topk <= 6 ? 3 : 8; }
template <int T, int TO, int MODE>
static void launch_combine_m(const RowParams& p, dim3 grid, hipStream_t s) {
  switch (rows_in_flight(p.topk)) {
    case 1: launch_combine_j<T, TO, 1, MODE>(p, grid, s); break;
    case 2: launch_combine_j<T, TO, 2, MODE>(p, grid, s); break;
    case 3: launch_combine_j<T, TO, 3, MODE>(p, grid, s); break;
    case 4: launch_combine_j<T, TO, 4, MODE>(p, grid, s); break;
    default: launch_combine_j<T, TO, 8, MODE>(p, grid, s);
  }
}
template <int T, int TO>
static void launch_combine_t(const RowParams& p, dim3 grid, hipStream_t s) {
  switch (row_mode<T>(p)) {
    case NARROW: hipLaunchKernelGGL((combine_kernel<T, TO, 1, NARROW, 1>), grid, dim3(64 * kRowWaves), 0, s, p); break;
    case CACHED: launch_combine_m<T, TO, CACHED>(p, grid, s); break;
    case STREAM: launch_combine_m<T, TO, STREAM>(p, grid, s); break;
    default: launch_combine_m<T, TO, STREAM_LINES>(p, grid, s);
  }
}

hipError_t launch_combine(const void* ys, const RouteLayout& r, const int32_t* plan, const float* weights,
                          int width, int dtype, void* y, int out_dtype, hipStream_t s) {
  RowParams p = row_params(r, plan, width, dtype == T_F32 ? 4 : 8);
  p.ys = ys;
  p.weights = weights;
  p.out = y;
  const dim3 grid(ceil_div(p.tokens * p.segs, kRowWaves));
  if (dtype == T_F16)
    launch_combine_t<T_F16, T_F16>(p, grid, s);
  else if (dtype == T_BF16)
    launch_combine_t<T_BF16, T_BF16>(p, grid, s);
  else if (out_dtype == T_F32)
    launch_combine_t<T_F32, T_F32>(p, grid, s);
  else if (out_dtype == T_F16)
    launch_combine_t<T_F32, T_F16>(p, grid, s);
  else
    launch_combine_t<T_F32, T_BF16>(p, grid, s);
  return hipGetLastError();
}

template <int T, int J, int MODE>
static void launch_backward_j(const RowParams& p, hipStream_t s) {
  const dim3 block(64 * kRowWaves);
  const int tail = ceil_div(p.tail_waves, kRowWaves);
  if (p.width <= 128 * Elem<T>::kVec)
    hipLaunchKernelGGL((combine_backward_kernel<T, J, MODE, 1>), dim3(ceil_div(p.tokens, kRowWaves) + tail), block, 0, s, p);
  else if constexpr (MODE != NARROW)
    hipLaunchKernelGGL((combine_backward_kernel<T, J, MODE, kRowWaves>), dim3(p.tokens + tail), block, 0, s, p);
}
template <int T, int MODE>
static void launch_backward_m(const RowParams& p, hipStream_t s) {
  switch (rows_in_flight(p.topk)) {
    case 1: launch_backward_j<T, 1, MODE>(p, s); break;
    case 2: launch_backward_j<T, 2, MODE>(p, s); break;
    case 3: launch_backward_j<T, 3, MODE>(p, s); break;
    case 4: launch_backward_j<T, 4, MODE>(p, s); break;
    default: launch_backward_j<T, 8, MODE>(p, s);
  }
}
template <int T>
static void launch_backward(const RowParams& p, hipStream_t s) {
  switch (row_mode<T>(p)) {
    case NARROW: launch_backward_j<T, 1, NARROW>(p, s); break;
    // odd rows, 4099 x 2885 at topk 3: over and over by itself 36 us cached, 41 streamed, but between the other
    // moves of a training step streamed (all of them 99 us, 104 cached); that one case is all that decides it
    case CACHED: launch_backward_m<T, CACHED>(p, s); break;
    case STREAM: launch_backward_m<T, STREAM>(p, s); break;
    default: launch_backward_m<T, STREAM_LINES>(p, s);
  }
}

hipError_t launch_combine_backward(const void* dy, const void* ys, const RouteLayout& r, const int32_t* plan,
                                   const float* weights, int width, int dtype, void* dys, float* dweights,
                                   hipStream_t s) {
  RowParams p = row_params(r, plan, width, dtype == T_F32 ? 4 : 8);
  p.x = dy;
  p.ys = ys;
  p.weights = weights;
  p.out = dys;
  p.dweights = dweights;
  p.tail_waves = round64(p.tail_waves);  // whole workgroups
  if (dtype == T_F16)
    launch_backward<T_F16>(p, s);
  else if (dtype == T_BF16)
    launch_backward<T_BF16>(p, s);
  else
    launch_backward<T_F32>(p, s);
  return hipGetLastError();
}

}  // namespace w4a16
