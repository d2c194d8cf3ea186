// Tiles of 32 cached tokens as operands of the matrix cores: what attention
// over the pages and the weighing of the pages share (include/dspark_cache.h).
#pragma once

#include "cache.hpp"

namespace dspark {

constexpr int kTile = 32;  // tokens of a tile, and query rows of one
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kFar = 1 << 29;  // past every table (2^20 pages of 128 tokens)

__device__ __forceinline__ bf16x8 as_bf16(u32x4 x) {
  union {
    u32x4 u;
    bf16x8 b;
  } c;
  c.u = x;
  return c.b;
}

// A (quotient of) counts below 2^52, by a double division and its correction:
// shorter code than the 64-bit integer division.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  int64_t q = static_cast<int64_t>(static_cast<double>(x) / static_cast<double>(y));
  const int64_t r = x - q * y;
  if (r < 0) --q;
  if (r >= y) ++q;
  return q;
}

// The same in every lane, so in scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// The token that K row slot p (0 .. 15) of a 16-token block holds: with this
// order the accumulators of half h are tokens 8 h .. 8 h + 7 in turn.
__device__ __forceinline__ int token_of_slot(int p) { return ((p >> 2) & 1) * 8 + (p >> 3) * 4 + (p & 3); }

// Keeps a rare branch a branch: without it the compiler turns the few
// instructions inside into selects that every tile pays for.
__device__ __forceinline__ void rare() { asm volatile(""); }

// Loads before this stay before those after it: they return in the order of
// their use (the scheduler likes to reverse them, and the first product then
// waits for the last load).  Everything but vector memory may cross.
__device__ __forceinline__ void keep_load_order() { __builtin_amdgcn_sched_barrier(0x78F); }

// The keys of one tile, loaded ahead of their use: this lane's row (token slot
// lane % 32 of the tile), the 8 dims of its half at every step.  Addresses are
// a wave's base (the page's part for the head and the token in it, in scalar
// registers) and a lane's constant offset.
template <int FMT, int D>
struct KTile;

template <int D>
struct KTile<DSPARK_CACHE_BF16, D> {
  u32x4 x[D / 16];
  static __device__ __forceinline__ uint32_t lane_offset(int slot, int h) {
    return (slot >> 4) * (32 * D) + (h * 16 + token_of_slot(slot & 15)) * 16;
  }
  __device__ __forceinline__ void load(const char* head, int, int t, uint32_t lane, int) {
    const char* p = head + static_cast<int64_t>(t >> 4) * (32 * D);
#pragma unroll
    for (int u = 0; u < D / 16; ++u) x[u] = *reinterpret_cast<const u32x4*>(p + u * 512 + lane);
  }
  static __device__ __forceinline__ int q_dim(int u, int h) { return 16 * u + 8 * h; }
  __device__ __forceinline__ u32x4 operand(int u, int) const { return x[u]; }
  __device__ __forceinline__ f32x16 scores(const u32x4 (&q)[D / 16], int) const {
    f32x16 s = {0.f};
#pragma unroll
    for (int u = 0; u < D / 16; ++u)
      s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(x[u]), as_bf16(q[u]), s, 0, 0, 0);
    return s;
  }
};

// 4 bits: a 16-byte load is 32 dims of a token, one scale group; half h takes
// groups h, h + 2, ..: four products' operands each, in the order q_dim gives.
template <int D>
struct KTile<DSPARK_CACHE_FP4, D> {
  static constexpr int E = D / 32;
  u32x4 x[D / 64];
  uint32_t sc[(E + 3) / 4];
  static __device__ __forceinline__ uint32_t lane_offset(int slot, int h) {
    return (slot >> 4) * (8 * D) + (h * 16 + token_of_slot(slot & 15)) * 16;
  }
  // token: the lane's token counted from t
  __device__ __forceinline__ void load(const char* head, int P, int t, uint32_t lane, int token) {
    const char* p = head + static_cast<int64_t>(t >> 4) * (8 * D);
#pragma unroll
    for (int g = 0; g < D / 64; ++g) x[g] = *reinterpret_cast<const u32x4*>(p + g * 512 + lane);
    const char* b = head + P * (D / 2) + t * E + static_cast<uint32_t>(token * E);
    if constexpr (E == 2) {
      sc[0] = *reinterpret_cast<const uint16_t*>(b);
    } else {
#pragma unroll
      for (int i = 0; i < E / 4; ++i) sc[i] = *reinterpret_cast<const uint32_t*>(b + 4 * i);
    }
  }
  static __device__ __forceinline__ int q_dim(int u, int h) { return 32 * (2 * (u / 4) + h) + 8 * (u % 4); }
  __device__ __forceinline__ u32x4 operand(int u, int h) const {
    return fp4_octet(x[u / 4][u % 4], k_scale_value((sc[u / 8] >> (16 * (u / 4 & 1) + 8 * h)) & 0xFFu));
  }
  __device__ __forceinline__ f32x16 scores(const u32x4 (&q)[D / 16], int h) const {
    f32x16 s = {0.f};
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
      const float scale = k_scale_value((sc[g / 2] >> (16 * (g & 1) + 8 * h)) & 0xFFu);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(fp4_octet(x[g][v], scale)), as_bf16(q[4 * g + v]), s, 0, 0,
                                                    0);
    }
    return s;
  }
};

// 8 bits: a 16-byte load is 16 dims of a token; half h takes groups h, h + 2,
// ..: two products' operands each.  One scale for the token's block.
template <int D>
struct KTile<DSPARK_CACHE_FP8, D> {
  u32x4 x[D / 32];
  uint32_t sc;
  static __device__ __forceinline__ uint32_t lane_offset(int slot, int h) {
    return (slot >> 4) * (16 * D) + (h * 16 + token_of_slot(slot & 15)) * 16;
  }
  __device__ __forceinline__ void load(const char* head, int P, int t, uint32_t lane, int token) {
    const char* p = head + static_cast<int64_t>(t >> 4) * (16 * D);
#pragma unroll
    for (int g = 0; g < D / 32; ++g) x[g] = *reinterpret_cast<const u32x4*>(p + g * 512 + lane);
    sc = *reinterpret_cast<const uint8_t*>(head + 2 * P * D + (t >> 4) + static_cast<uint32_t>(token >> 4));
  }
  static __device__ __forceinline__ int q_dim(int u, int h) { return 16 * (2 * (u / 2) + h) + 8 * (u % 2); }
  __device__ __forceinline__ u32x4 operand(int u, int) const {
    return fp8_octet(x[u / 2][2 * (u % 2)], x[u / 2][2 * (u % 2) + 1], k_scale_value(sc));
  }
  __device__ __forceinline__ f32x16 scores(const u32x4 (&q)[D / 16], int) const {
    f32x16 s = {0.f};
    const float scale = k_scale_value(sc);
#pragma unroll
    for (int u = 0; u < D / 16; ++u)
      s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          as_bf16(fp8_octet(x[u / 2][2 * (u % 2)], x[u / 2][2 * (u % 2) + 1], scale)), as_bf16(q[u]), s, 0, 0, 0);
    return s;
  }
};

}  // namespace dspark
