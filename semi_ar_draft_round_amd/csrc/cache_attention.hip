// Grouped-head attention of a round's rows over the paged cache, with an
// optional sliding window and visible first tokens (include/dspark_cache.h).
//
// The plain form of the kernel: one wave per (row, query head).  A lane
// scores one of 64 tokens at a time; the softmax is online (running maximum
// and sum), and the output's dims are dealt to the lanes.
#include "cache.hpp"

namespace dspark {

namespace {

struct AttnArgs {
  int R, gamma, Hq, Hkv, P, n_pages, max_pages;
  const uint16_t* q;
  float scale;
  int window, sinks;
  const int32_t *row0, *ell, *len, *table;
  const char* pool;
  int64_t page_bytes;
  uint16_t* out;
  float* lse;
};

__device__ __forceinline__ float e2m1(uint32_t c) {
  const uint32_t m = c & 7u;
  const float y = m < 2u ? 0.5f * m : __uint_as_float((126u + (m >> 1)) << 23) * (1.f + 0.5f * (m & 1u));
  return (c & 8u) ? -y : y;
}

template <int FMT, int D>
__device__ float k_value(const char* head, int P, int t, int d) {
  typedef PageLayout<FMT, D> L;
  if constexpr (FMT == DSPARK_CACHE_BF16) {
    return bf16_to_f32(reinterpret_cast<const uint16_t*>(head + L::k(P, t, d / 8))[d % 8]);
  } else {
    const uint32_t b = static_cast<uint8_t>(head[L::k(P, t, d / 32) + (d % 32) / 2]);
    return e2m1(b >> (4 * (d & 1)) & 15u) * k_scale_value(static_cast<uint8_t>(head[L::k_scale(P, t) + d / 32]));
  }
}

template <int FMT, int D>
__device__ float v_value(const char* head, int P, int t, int d) {
  typedef PageLayout<FMT, D> L;
  if constexpr (FMT == DSPARK_CACHE_BF16) {
    return bf16_to_f32(reinterpret_cast<const uint16_t*>(head + L::v(P, t, d))[t % 8]);
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(head + L::v(P, t, d));
    return e2m1(w >> (4 * (t & 7)) & 15u) * *reinterpret_cast<const float*>(head + L::v_scale(P, t));
  }
}

template <int FMT, int D>
__global__ __launch_bounds__(64) void cache_attention_rows(AttnArgs a) {
  typedef PageLayout<FMT, D> L;
  __shared__ float qs[D];
  const int r = blockIdx.x / (a.gamma + 1), i = blockIdx.x % (a.gamma + 1), hq = blockIdx.y;
  const int lane = threadIdx.x;
  if (i >= rows_of(a.ell[r], a.gamma) || a.len[r] < 0) return;
  const int64_t row = (a.row0 ? static_cast<int64_t>(a.row0[r]) : static_cast<int64_t>(r) * (a.gamma + 1)) + i;
  const int64_t pos = static_cast<int64_t>(a.len[r]) + i;
  const uint16_t* q = a.q + (row * a.Hq + hq) * D;
  for (int d = lane; d < D; d += 64) qs[d] = bf16_to_f32(q[d]);
  __syncthreads();
  const int64_t head_off = (hq / (a.Hq / a.Hkv)) * L::head_bytes(a.P);
  const int32_t* table = a.table + static_cast<int64_t>(r) * a.max_pages;
  const int64_t cap = static_cast<int64_t>(a.max_pages) * a.P;
  const int64_t end = pos + 1 < cap ? pos + 1 : cap;
  const int64_t low = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;

  float m = neg_inf(), l = 0.f, o[D / 64];
#pragma unroll
  for (int j = 0; j < D / 64; ++j) o[j] = 0.f;
  for (int64_t t0 = 0; t0 < end; t0 += 64) {
    if (t0 >= a.sinks && t0 + 64 <= low) {
      t0 = (low / 64) * 64 - 64;
      continue;
    }
    const int64_t t = t0 + lane;
    const bool in = t < end && (t >= low || t < a.sinks);
    const int id = in ? page_or_none(table[t / a.P], a.n_pages) : -1;
    float s = neg_inf();
    if (id >= 0) {
      const char* head = a.pool + id * a.page_bytes + head_off;
      s = 0.f;
      for (int d = 0; d < D; ++d) s += qs[d] * k_value<FMT, D>(head, a.P, static_cast<int>(t % a.P), d);
      s *= a.scale;
    }
    const float top = fmaxf(m, wave_reduce_max(s));
    const float base = top == neg_inf() ? 0.f : top;
    const float p = id >= 0 ? expf(s - base) : 0.f, keep = expf(m - base);
    l = l * keep + wave_reduce_sum(p);
    m = top;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) o[j] *= keep;
    for (int k = 0; k < 64; ++k) {
      const int page = __shfl(id, k);
      if (page < 0) continue;
      const float w = __shfl(p, k);
      const char* head = a.pool + page * a.page_bytes + head_off;
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
        o[j] += w * v_value<FMT, D>(head, a.P, static_cast<int>((t0 + k) % a.P), j * 64 + lane);
    }
  }
#pragma unroll
  for (int j = 0; j < D / 64; ++j)
    a.out[(row * a.Hq + hq) * D + j * 64 + lane] = static_cast<uint16_t>(bf16_bits_rne(l != 0.f ? o[j] / l : 0.f));
  if (a.lse && lane == 0) a.lse[row * a.Hq + hq] = l != 0.f ? m + logf(l) : neg_inf();
}

template <int FMT, int D>
hipError_t run(AttnArgs& a, hipStream_t s) {
  a.page_bytes = a.Hkv * PageLayout<FMT, D>::head_bytes(a.P);
  cache_attention_rows<FMT, D><<<dim3(a.R * (a.gamma + 1), a.Hq), 64, 0, s>>>(a);
  return hipGetLastError();
}

template <int FMT>
hipError_t run_d(int D, AttnArgs& a, hipStream_t s) {
  return D == 64 ? run<FMT, 64>(a, s) : D == 128 ? run<FMT, 128>(a, s) : run<FMT, 256>(a, s);
}

}  // namespace

size_t cache_attention_workspace_bytes(int R, int gamma, int Hq, int Hkv, int D) {
  (void)R, (void)gamma, (void)Hq, (void)Hkv, (void)D;
  return 256;
}

hipError_t cache_attention_launch(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages,
                                  int max_pages, const void* q, float scale, int window, int sinks,
                                  const int32_t* row0, const int32_t* ell, const int32_t* len, const int32_t* table,
                                  const void* pool, void* out, float* lse, void* ws, hipStream_t s) {
  (void)ws;
  AttnArgs a{R, gamma, Hq, Hkv, P, n_pages, max_pages, static_cast<const uint16_t*>(q), scale, window,
             window > 0 ? sinks : 0, row0, ell, len, table, static_cast<const char*>(pool), 0,
             static_cast<uint16_t*>(out), lse};
  return fmt == DSPARK_CACHE_BF16 ? run_d<DSPARK_CACHE_BF16>(D, a, s) : run_d<DSPARK_CACHE_FP4>(D, a, s);
}

}  // namespace dspark
