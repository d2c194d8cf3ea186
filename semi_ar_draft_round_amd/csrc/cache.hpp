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
// gives NaN for every code, 0 gives 2^-127 (both checked on the device).
__device__ __forceinline__ float k_scale_value(uint32_t b) { return __uint_as_float(b << 23); }
__device__ __forceinline__ u32x4 fp4_octet(uint32_t w, float scale) {
  return u32x4{fp4_pair<0>(w, scale), fp4_pair<1>(w, scale), fp4_pair<2>(w, scale), fp4_pair<3>(w, scale)};
}

}  // namespace dspark
