// Rows on their way into the cache: what the appends of all page formats share
// (a head's norm and rotation, sums over the lanes of a head).
#pragma once

#include "cache.hpp"

namespace dspark {

constexpr int kGroup = 8;  // tokens of a V word
constexpr int kThreads = 256;

struct AppendArgs {
  int R, gamma, Hq, Hkv, P, n_pages, max_pages, groups;
  const uint16_t *q, *k, *v;
  int64_t ldq, ldk, ldv;
  const uint16_t *wq, *wk;
  float eps;
  const double* freq;
  int rot, adjacent;
  const int32_t *row0, *ell, *len, *table;
  uint16_t* q_out;
  char* pool;
  int64_t page_bytes;
  int page_shift;
  float per_q, per_k, per_half;  // 1 / Hq, 1 / Hkv, 1 / (rot / 2)
};

// x / y for 0 <= x < 2^14, 1 <= y <= 2^10 and inv = 1 / y in fp32: x + 1/2 is
// at least 1 / (2 y) from a multiple of y, far more than the product's error.
__device__ __forceinline__ int small_quotient(int x, float inv) {
  return static_cast<int>((static_cast<float>(x) + 0.5f) * inv);
}

// f over the values of L = 4, 8, 16 or 32 neighbouring lanes, the same in each
// (f commutes, so also the same bits).
template <int L, typename T, typename F>
__device__ __forceinline__ T over_lanes(T x, F f) {
  x = f(x, lane_pattern<kSwap1>(x));
  x = f(x, lane_pattern<kSwap2>(x));
  if constexpr (L > 4) x = f(x, lane_pattern<kMirror8>(x));
  if constexpr (L > 8) x = f(x, lane_pattern<kMirror16>(x));
  if constexpr (L > 16) x = f(x, __shfl_xor(x, 16));
  return x;
}

__device__ __forceinline__ float inv_sqrt(float x) { return rsqrtf(x); }
__device__ __forceinline__ double inv_sqrt(double x) { return 1.0 / sqrt(x); }

// The norm and the rotation of one head, 8 dims per lane, in the type T.
// li: the lane's place in the head; w: the norm's weights of its dims; cs:
// cosine and sine of pair i at 2 i.
template <typename T, int D>
__device__ __forceinline__ void norm_rotate(T (&x)[8], int li, bool norm, const u32x4& w, float eps, int rot,
                                            bool adjacent, const T* cs) {
  constexpr int L = D / 8;
  if (norm) {
    T ss = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
    ss = over_lanes<L>(ss, [](T p, T q) { return p + q; });
    T s = inv_sqrt(ss * static_cast<T>(1.0 / D) + static_cast<T>(eps));
    if constexpr (sizeof(T) == 4) {
      // a sum of squares that fp32 does not hold, or not whole (an |x| past
      // 2^60, or a sum below 2^-96): the head again in fp64, a rare branch of
      // the wave; its test costs 0.2 us of 12.2 for 128 x up to 17 packed rows
      const bool in_range = __float_as_uint(ss) - 0x0F800000u < 0x7B800000u - 0x0F800000u;  // 2^-96 .. 2^120
      if (__builtin_expect(__any(!in_range), 0)) {
        double s2 = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) s2 += static_cast<double>(x[e]) * x[e];
        s2 = over_lanes<L>(s2, [](double p, double q) { return p + q; });
        s2 = inv_sqrt(s2 * (1.0 / D) + static_cast<double>(eps));
        if (!in_range) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = static_cast<float>(x[e] * s2);
          s = 1.f;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = x[e] * s * static_cast<T>(bf16_to_f32(static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)))));
  }
  if (rot == 0) return;
  if (adjacent) {
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      if (li * 8 + e < rot) {
        const int i = li * 4 + e / 2;
        const T c = cs[2 * i], s = cs[2 * i + 1], a = x[e], b = x[e + 1];
        x[e] = a * c - b * s;
        x[e + 1] = b * c + a * s;
      }
    return;
  }
  // partner dims are rot / 2 = 8 * hl away; lanes past rot read some lane and keep their own
  const int hl = rot / 16;
  const int lane = threadIdx.x & 63, base = lane - li;
  const bool first = li < hl, second = !first && li < 2 * hl;
  const int partner = base + (first ? li + hl : second ? li - hl : li);
  if constexpr (L == 16)
    if (2 * hl == L) {  // all of a head of 128 dims: the partner is 8 lanes away in the same 16
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const T y = lane_pattern<kTurn8>(x[e]);
        const int i = (li & 7) * 8 + e;
        const T c = cs[2 * i], s = cs[2 * i + 1];
        x[e] = first ? x[e] * c - y * s : x[e] * c + y * s;
      }
      return;
    }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const T y = __shfl(x[e], partner);
    if (first || second) {
      const int i = (first ? li : li - hl) * 8 + e;
      const T c = cs[2 * i], s = cs[2 * i + 1];
      x[e] = first ? x[e] * c - y * s : x[e] * c + y * s;
    }
  }
}

__device__ __forceinline__ u32x4 pack_bf16(const float (&x)[8]) {
  u32x4 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = bf16_pair(x[2 * j], x[2 * j + 1]);
  return r;
}

__device__ __forceinline__ void unpack(const u32x4& v, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = bf16_to_f32(static_cast<uint16_t>(v[e / 2] >> (16 * (e & 1))));
}

}  // namespace dspark
