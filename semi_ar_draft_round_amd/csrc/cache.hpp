// The paged cache's shapes, page layouts and 4-bit codes (include/dspark_cache.h).
#pragma once

#include "common.hpp"
#include "dspark_cache.h"

namespace dspark {

// abi.hip: DSPARK_OK if the current device is a gfx950.
dspark_status check_device();
int compute_units();

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kCacheMaxR = 4096;
constexpr int kCacheMaxGamma = 1023;
constexpr int kCacheMaxHeads = 1024;
constexpr int kCacheMaxPages = 1 << 20;
constexpr int kCacheMaxT = 1 << 26;  // rows of a read: its grid stays below 2^32 threads

// Byte offsets inside one head's part of a page (dspark_cache.h, Pages).
template <int FMT, int D>
struct PageLayout;

template <int D>
struct PageLayout<DSPARK_CACHE_BF16, D> {
  static __host__ __device__ int64_t head_bytes(int P) { return 4LL * P * D; }
  // 8 dims 8*g .. of token t of the page
  static __device__ int64_t k(int P, int t, int g) {
    return (static_cast<int64_t>(t >> 4) * (16 * D) + (g * 16 + (t & 15)) * 8) * 2;
  }
  // tokens 8*(t/8) .. of dim d
  static __device__ int64_t v(int P, int t, int d) {
    return 2LL * P * D + (static_cast<int64_t>(t >> 4) * (16 * D) + (((t >> 3) & 1) * D + d) * 8) * 2;
  }
};

template <int D>
struct PageLayout<DSPARK_CACHE_FP4, D> {
  static constexpr int E = D / 32;
  static __host__ __device__ int64_t head_bytes(int P) { return static_cast<int64_t>(P) * (D + E + 4); }
  // the 16 bytes of dims 32*g .. of token t
  static __device__ int64_t k(int P, int t, int g) {
    return static_cast<int64_t>(t >> 4) * (8 * D) + (g * 16 + (t & 15)) * 16;
  }
  static __device__ int64_t k_scale(int P, int t) { return static_cast<int64_t>(P) * (D / 2) + t * E; }
  // tokens 8*(t/8) .. of dim d: 4 bytes
  static __device__ int64_t v(int P, int t, int d) {
    return static_cast<int64_t>(P) * (D / 2 + E) + static_cast<int64_t>(t >> 4) * (8 * D) +
           ((((t >> 3) & 1) * 32 + (d & 31)) * E + (d >> 5)) * 4;
  }
  static __device__ int64_t v_scale(int P, int t) { return static_cast<int64_t>(P) * (D + E) + t * 4LL; }
};

// Rows of request r this time, 0 .. gamma + 1, from a device value.
__device__ __forceinline__ int rows_of(int ell, int gamma) { return ell < 0 ? 0 : (ell > gamma ? gamma : ell) + 1; }

// The page of a table entry, or -1.
__device__ __forceinline__ int page_or_none(int id, int n_pages) {
  return static_cast<uint32_t>(id) < static_cast<uint32_t>(n_pages) ? id : -1;
}

// Two fp32 values as a pair of bf16, each to nearest, ties to even.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  union {
    bf16x2 b;
    uint32_t u;
  } r;
  r.b = bf16x2{static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return r.u;
}

// Two e2m1 codes (byte SEL of w) times 2^(exponent of scale) as bf16, exact.
template <int SEL>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t w, float scale) {
  union {
    bf16x2 b;
    uint32_t u;
  } r;
  r.b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL);
  return r.u;
}

// Eight codes times the scale of a K scale byte b: 2^(b - 127), or NaN for
// 255.  The conversion reads the scale's exponent field as such a byte: 255
// gives NaN for every code, 0 gives 2^-127.
__device__ __forceinline__ float k_scale_value(uint32_t b) { return __uint_as_float(b << 23); }
__device__ __forceinline__ u32x4 fp4_octet(uint32_t w, float scale) {
  return u32x4{fp4_pair<0>(w, scale), fp4_pair<1>(w, scale), fp4_pair<2>(w, scale), fp4_pair<3>(w, scale)};
}

// The value of another lane by a fixed pattern, without the way through LDS
// that a shuffle takes; 0 in rows of 16 lanes outside ROWS and where the
// pattern has no source.  All lanes involved are active.
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140, kTurn8 = 0x128;
constexpr int kUp1 = 0x111, kUp2 = 0x112, kUp4 = 0x114, kUp8 = 0x118, kLast16 = 0x142, kLast32 = 0x143;
template <int PATTERN, int ROWS = 0xF>
__device__ __forceinline__ int lane_pattern(int x) {
  return __builtin_amdgcn_update_dpp(0, x, PATTERN, ROWS, 0xF, false);
}
template <int PATTERN, int ROWS = 0xF>
__device__ __forceinline__ float lane_pattern(float x) {
  return __int_as_float(lane_pattern<PATTERN, ROWS>(__float_as_int(x)));
}
template <int PATTERN, int ROWS = 0xF>
__device__ __forceinline__ double lane_pattern(double x) {
  return __hiloint2double(lane_pattern<PATTERN, ROWS>(__double2hiint(x)),
                          lane_pattern<PATTERN, ROWS>(__double2loint(x)));
}
template <int PATTERN, int ROWS = 0xF>
__device__ __forceinline__ int64_t lane_pattern(int64_t x) {
  const uint32_t lo = lane_pattern<PATTERN, ROWS>(static_cast<int>(x));
  return static_cast<int64_t>(lane_pattern<PATTERN, ROWS>(static_cast<int>(x >> 32))) << 32 | lo;
}

// f over the values of this lane and those before it, for f with f(x, 0) = x.
// All 64 lanes are active.
template <typename T, typename F>
__device__ __forceinline__ T wave_scan(T x, F f) {
  x = f(x, lane_pattern<kUp1>(x));
  x = f(x, lane_pattern<kUp2>(x));
  x = f(x, lane_pattern<kUp4>(x));
  x = f(x, lane_pattern<kUp8>(x));
  x = f(x, lane_pattern<kLast16, 0xA>(x));  // the sums of 16 into the next 16,
  x = f(x, lane_pattern<kLast32, 0xC>(x));  // that of the first 32 into the others
  return x;
}

}  // namespace dspark
