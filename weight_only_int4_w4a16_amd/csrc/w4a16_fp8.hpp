// w4a16_fp8.hpp - 8-bit floating point operators (e4m3 codes with a scale for each 128 values or block of
// 128 x 128): internal launchers, and what their kernels share.
//
// A scale is s = max|v| / 448 (448 the largest e4m3 value), at least 2^-126, and a code RN_e4m3(RN_f32(v / s)): two
// correctly rounded 32-bit steps and one to 8 bits, so that codes are reproducible decisions. A group that holds
// an infinity or a NaN becomes NaN throughout.
//
// Scales of rows lie by blocks of k: scales[kb][row], so that the rows of a tile read one block's scales as
// consecutive words.
#pragma once

#include "w4a16_device.hpp"
#include "w4a16_routed.hpp"

namespace w4a16 {

constexpr float kE4M3Most = 448.0f;
constexpr float kLeastScale = 0x1p-126f;
constexpr int kE4M3 = 3;  // as w4a16_dtype: codes with scales

// One product out[m][n] = sum over k blocks of (scale of x's row m) (scale of w's block or row n) (codes of row m) .
// (codes of row n). Pointers of grouped products are to the first group's.
struct Fp8Args {
  const uint8_t* x;   // codes [M][ldk]
  const float* xs;    // scales [KB][xs_ld]
  const uint8_t* w;   // codes [N][ldk] (swiglu: 2 N rows, gate first)
  const float* ws;    // block scales [ceil(N / 128)][KB] (swiglu: each half's blocks), or with w_rows [KB][N]
  bool w_rows;
  int M, N, K;        // N: columns of out
  int ldk;            // bytes from one row of codes to the next
  int xs_ld;          // x scales of one block of k
  bool glu;
  void* out;
  int out_dtype;      // 0 fp16, 1 bf16, 2 fp32, 3 e4m3 (glu: codes with scales)
  float* out_scales;  // [ceil(N / 128)][M], for e4m3
  const void* values; // x itself, of 16 bits, where the kernel quantizes it (fp8_takes_values; x and xs are not read)
  int values_dtype;
  float* scratch;     // fp32 sums of each slice of k, or h [M][N] where a kernel cannot quantize it by itself
  hipStream_t stream;
};

inline size_t fp8_blocks(int n) { return ((size_t)n + 127) / 128; }
inline int ceil16(int n) { return (n + 15) & ~15; }

// rows: codes [M][K], scales [ceil(K / 128)][M]; K % 16 == 0
hipError_t launch_fp8_rows(const void* x, int M, int K, int dtype, uint8_t* codes, float* scales, hipStream_t s);
// columns: codes [K][pitch] transposed, scales [row tiles][K]; a tile is 128 rows, or with a plan (r) one of
// its 128-row tiles (those past its list are left alone; pitch: 128 times the list's bound); with row_codes and
// row_scales the rows' codes too, of the tiles' rows (16-bit x, K % 16 == 0)
hipError_t launch_fp8_columns(const void* x, int M, int K, int dtype, uint8_t* codes, size_t pitch, float* scales,
                              uint8_t* row_codes, float* row_scales, const RouteLayout* r, const int32_t* plan,
                              hipStream_t s);
// Launches hold fewer than 2^32 threads: whether these do, for rows, and for columns and blocks of 128 x 128
bool fp8_rows_fit(int M, int K);
bool fp8_tiles_fit(int M, int K);
// blocks of 128 x 128: codes [N][K], scales [ceil(N / 128)][ceil(K / 128)]; codes_t, scales_t the same transposed, or NULL
hipError_t launch_fp8_weight(const void* w, int N, int K, int dtype, uint8_t* codes, float* scales, uint8_t* codes_t,
                             float* scales_t, hipStream_t s);

hipError_t launch_fp8(const Fp8Args& a);
// the rows and weights of a plan's groups; gather: x holds the tokens' rows
hipError_t launch_fp8_grouped(const Fp8Args& a, const RouteLayout& r, const int32_t* plan, bool gather);
// out[e][m][n] over the 128-row tiles of group e, which are the blocks of k (both operands scaled by rows)
hipError_t launch_fp8_by_group(const Fp8Args& a, const RouteLayout& r, const int32_t* plan);

// bytes of Fp8Args::scratch that a launch needs (0: none)
size_t fp8_scratch_bytes(int M, int N, int K, bool glu, int out_dtype, bool w_rows = false);
size_t fp8_grouped_scratch_bytes(const RouteLayout& r, int N, int out_dtype);
// whether a dense product of 16-bit x quantizes it as it reads it
bool fp8_takes_values(int M, int N, int K, bool glu, int out_dtype);
// whether the product's launches can index it
bool fp8_fits(int M, int N, int K, bool glu, int out_dtype, bool w_rows = false);
bool fp8_grouped_fits(const RouteLayout& r, int N, int K, bool glu, int out_dtype);
const char* fp8_name(int M, int N, int K, bool glu);

// ---- device side ----

// The scale of a group whose largest magnitude has these bits
__device__ __forceinline__ float fp8_scale(uint32_t amax) {
  if (amax >= 0x7F800000u) return __builtin_nanf("");
  const float s = __builtin_bit_cast(float, amax) / kE4M3Most;
  return s < kLeastScale ? kLeastScale : s;
}

// Division by a scale, correctly rounded: with r = RN(1 / s), two steps of q += r (v - q s) after q = v r
// give RN(v / s) (the remainders are exact). Scales under 2^-60 are taken 2^64 times as large, and so are
// their values, so that no remainder reaches the subnormal numbers where the quotient's code is not 0.
//
// For v of 16 bits (DT 0, 1) one step gives the same codes. After it q = RN(v / s (1 + e)), |e| <= 2^-46, so that a code could
// differ only where v / s lies within 2^-46 of b +- half an ulp, b one of the 5-bit numbers midway between two codes. Let
// v = A 2^i and s = RN(B 2^j / 448), A and B integers under 2^11. Then 7 A 2^m and b B are integers (b's taken) under 2^17
// within 2^-23 of each other, so they are equal, and s is off by exactly that half ulp: with s's 24 bits S,
// 7 S - B 2^k = r, 0 < |r| <= 3, and |r| b 2^20 (or 21) = B 2^k, both being multiples of 2^12 under 2^27 that near. If 7 divides b it
// divides B, and r is 0; if not, 7 A 2^m = b B = |r| b^2 2^n has no solution. A zero group's scale divides zeros, and no
// other fp16 group has a scale under 2^-60.
struct Fp8Divisor {
  float s, r, up;
};
__device__ __forceinline__ Fp8Divisor fp8_divisor(float scale) {
  Fp8Divisor d;
  d.up = scale < 0x1p-60f ? 0x1p64f : 1.0f;
  d.s = scale * d.up;
  d.r = 1.0f / d.s;
  return d;
}
template <int DT>
__device__ __forceinline__ float fp8_quotient(float v, const Fp8Divisor& d) {
  if constexpr (DT != 0) v *= d.up;
  float q = v * d.r;
  q = __builtin_fmaf(__builtin_fmaf(-q, d.s, v), d.r, q);
  if constexpr (DT == 2) q = __builtin_fmaf(__builtin_fmaf(-q, d.s, v), d.r, q);
  return __builtin_copysignf(q, v);  // the steps make +0 of -0
}

// four values as codes, one a byte
__device__ __forceinline__ uint32_t fp8_pack(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

// v of the lane that a DPP control names
template <int CTRL>
__device__ __forceinline__ uint32_t fp8_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}
// the largest of each sixteen lanes, in all of them (rotations by 8, 4, 2, 1)
__device__ __forceinline__ uint32_t max_of_16_lanes(uint32_t v) {
  v = max(v, fp8_dpp<0x128>(v));
  v = max(v, fp8_dpp<0x124>(v));
  v = max(v, fp8_dpp<0x122>(v));
  return max(v, fp8_dpp<0x121>(v));
}

typedef unsigned short us2_t __attribute__((ext_vector_type(2)));
// vectors at any address that their elements may have (rows may start anywhere)
typedef u4_t u4_any_t __attribute__((aligned(2)));
typedef h8_t h8_any_t __attribute__((aligned(2)));
typedef b8_t b8_any_t __attribute__((aligned(2)));
typedef f4_t f4_any_t __attribute__((aligned(4)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));

// Eight results of a row to out (as w4a16_dtype, not e4m3), of which the row still has `some`
__device__ __forceinline__ void fp8_store8(void* out, size_t at, const float (&v)[8], int some, int dtype) {
  if (some < 8) {
    for (int j = 0; j < 8; ++j)
      if (j < some) store_out(out, at + j, v[j], dtype);
  } else if (dtype == 2) {
    float* const dst = static_cast<float*>(out) + at;
    *reinterpret_cast<f4_any_t*>(dst) = f4_t{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f4_any_t*>(dst + 4) = f4_t{v[4], v[5], v[6], v[7]};
  } else if (dtype == 0) {
    h8_t o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = (_Float16)v[j];
    *reinterpret_cast<h8_any_t*>(static_cast<_Float16*>(out) + at) = o;
  } else {
    b8_t o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = (__bf16)v[j];
    *reinterpret_cast<b8_any_t*>(static_cast<__bf16*>(out) + at) = o;
  }
}

// Eight consecutive values of a row, by their type (as w4a16_dtype)
template <int DT>
struct Eight;

template <int DT>
struct Eight16 {
  u4_t v;
  __device__ __forceinline__ void clear() { v = u4_t{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void load(const void* row, size_t i) {
    v = *reinterpret_cast<const u4_any_t*>(static_cast<const uint16_t*>(row) + i);
  }
  __device__ __forceinline__ void load_some(const void* row, size_t i, int n) {
    clear();
    for (int j = 0; j < 8; ++j)
      if (j < n) v[j >> 1] |= (uint32_t)static_cast<const uint16_t*>(row)[i + j] << (16 * (j & 1));
  }
  // without the first n (of 1 to 7), zeros behind
  __device__ __forceinline__ void drop(int n) {
    if (n & 4) v = u4_t{v[2], v[3], 0u, 0u};
    if (n & 2) v = u4_t{v[1], v[2], v[3], 0u};
    if (n & 1) v = u4_t{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
  }
  __device__ __forceinline__ float value(int j) const {
    const uint16_t b = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
    if constexpr (DT == 0) return (float)__builtin_bit_cast(_Float16, b);
    else return __builtin_bit_cast(float, (uint32_t)b << 16);
  }
  // magnitudes, two a word
  static constexpr int kWords = 4;
  __device__ __forceinline__ uint32_t magnitude(int w) const { return v[w] & 0x7FFF7FFFu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2_t, a), __builtin_bit_cast(us2_t, b)));
  }
  // the bits of a magnitude as a 32-bit float's: of value h of a word, or of the word's largest
  static __device__ __forceinline__ uint32_t float_bits(uint32_t w, int h) {
    const uint16_t b = (uint16_t)(w >> (16 * h));
    if constexpr (DT == 0) return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, b));
    else return (uint32_t)b << 16;
  }
  static __device__ __forceinline__ uint32_t largest_bits(uint32_t w) { return float_bits(max(w & 0xFFFFu, w >> 16), 0); }
  static constexpr int kPerWord = 2;
};
template <>
struct Eight<0> : Eight16<0> {};
template <>
struct Eight<1> : Eight16<1> {};
template <>
struct Eight<2> {
  float v[8];
  __device__ __forceinline__ void clear() {
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
  }
  __device__ __forceinline__ void load(const void* row, size_t i) {
    const float* p = static_cast<const float*>(row) + i;
    const f4_t a = *reinterpret_cast<const f4_any_t*>(p), b = *reinterpret_cast<const f4_any_t*>(p + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
  }
  __device__ __forceinline__ void load_some(const void* row, size_t i, int n) {
    for (int j = 0; j < 8; ++j) v[j] = j < n ? static_cast<const float*>(row)[i + j] : 0.f;
  }
  __device__ __forceinline__ float value(int j) const { return v[j]; }
  static constexpr int kWords = 8;
  __device__ __forceinline__ uint32_t magnitude(int w) const { return __builtin_bit_cast(uint32_t, v[w]) & 0x7FFFFFFFu; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t float_bits(uint32_t w, int) { return w; }
  static __device__ __forceinline__ uint32_t largest_bits(uint32_t w) { return w; }
  static constexpr int kPerWord = 1;
};

}  // namespace w4a16
