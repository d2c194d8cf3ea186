// The append into 8-bit pages: norms and rotation as for the other formats,
// and blocks of 16 tokens that share a scale (include/dspark_cache.h).
//
// A block's scale is known when all of its new rows are, so one wave takes a
// block's keys of one head, another its values: it holds the block's new rows
// in registers, finds their largest magnitude, compares the scale that the
// block's committed tokens have, and writes codes.  Only where the scale grew
// are the committed tokens' codes read, rounded again and written back.
//   keys    D / 8 lanes a row, 8 dims each, as the norm and the rotation want
//           it; fp64, so that a code does not depend on the order of a sum;
//   values  a lane has its dims of all 16 tokens, which is how the pages hold
//           them: no exchange, whole 8-byte words.
// Queries go to work groups of their own, as a head slot a row and head.
//
// A code is rounded once: fp64 is cut to fp32 with what was cut off kept in
// the last bit (a value between two codes, or between a code and the border
// beside it, stays there), and the conversion rounds that.
#include "cache_rows.hpp"

namespace dspark {

namespace {

constexpr int kBlock = 16;  // tokens that share a scale
constexpr int kLow = -117, kHigh = 119;  // exponents of a scale
constexpr float kMost = 448.f;           // the largest code

// y cut to fp32, its last bit set if anything was lost; |y| <= 448.
__device__ __forceinline__ float cut_odd(double y) {
  const uint64_t b = __double_as_longlong(y);
  const int ex = static_cast<int>((b >> 52) & 0x7FF) - 1023 + 127;
  const uint32_t sign = static_cast<uint32_t>(b >> 63) << 31;
  if (ex <= 0) return __uint_as_float(sign);  // below 2^-126: far below half of the least code
  const uint32_t m = static_cast<uint32_t>(b >> 29) & 0x7FFFFFu, lost = (b & 0x1FFFFFFFull) != 0;
  return __uint_as_float(sign | static_cast<uint32_t>(ex) << 23 | m | lost);
}

// Four e4m3 codes, each to nearest, ties to even; |x| <= 448 or NaN.
__device__ __forceinline__ uint32_t codes_of(float x0, float x1, float x2, float x3) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(x0, x1, 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(x2, x3, w, true);
}

// Codes under a scale `f` = 2^-n of what they were.
__device__ __forceinline__ uint32_t rescale(uint32_t w, float f) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  return codes_of(a[0] * f, a[1] * f, b[0] * f, b[1] * f);
}

// The smallest exponent e with x <= 448 2^e, within the limits.
__device__ __forceinline__ int exponent_for(double x) {
  if (!(x > 0)) return kLow;
  const int q = ilogb(x);  // 448 = 1.75 2^8
  return min(kHigh, max(kLow, ldexp(x, -q) <= 1.75 ? q - 8 : q - 7));
}
__device__ __forceinline__ int exponent_of(uint8_t byte) { return min(kHigh, max(kLow, static_cast<int>(byte) - 127)); }

// 16 tokens of one request's row of blocks: tokens first .. first + n - 1 of
// the block are new, those before `first` committed.
struct Block {
  int first, n;
  int64_t row;   // of the first new token
  int64_t t0;    // its position
  int t;         // the block's first token within its page
  char* page;
};

template <int D>
__device__ __forceinline__ void append_keys(const AppendArgs& a, const Block& b, int head, int lane, const u32x4& w_k,
                                            const u32x4 (&raw)[kBlock * D / 512], const double* cs) {
  typedef PageLayout<DSPARK_CACHE_FP8, D> PL;
  constexpr int L = D / 8, RW = 64 / L, IT = kBlock / RW;
  const int li = lane % L, sub = lane / L;
  double x[IT][8], top = 0;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int j = it * RW + sub;
    const bool mine = j >= b.first && j < b.first + b.n;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[it][e] = 0;
    if (it * RW + RW <= b.first || it * RW >= b.first + b.n) continue;  // the same in every lane
    float f[8];
    unpack(raw[it], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[it][e] = f[e];
    norm_rotate<double, D>(x[it], li, a.wk != nullptr, w_k, a.eps, a.rot, a.adjacent != 0,
                           cs + (mine ? j - b.first : 0) * D);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (!mine) x[it][e] = 0;
      if (fabs(x[it][e]) <= 1.7976931348623157e308) top = fmax(top, fabs(x[it][e]));
    }
  }
  if (!b.page) return;
  top = over_lanes<32>(top, [](double p, double q) { return fmax(p, q); });
  top = fmax(top, __shfl_xor(top, 32));
  char* hp = b.page + head * PL::head_bytes(a.P);
  uint8_t* byte = reinterpret_cast<uint8_t*>(hp + PL::k_scale(a.P, b.t));
  const int before = b.first > 0 ? exponent_of(*byte) : kLow;
  const int e2 = max(before, exponent_for(top));
  const double f = ldexp(1.0, -e2);
  const float again = ldexpf(1.f, before - e2);
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int j = it * RW + sub;
    u32x2* p = reinterpret_cast<u32x2*>(hp + PL::k(a.P, b.t + j, li / 2) + (li & 1) * 8);
    if (j >= b.first && j < b.first + b.n) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double v = x[it][e];
        y[e] = fabs(v) <= 1.7976931348623157e308 ? cut_odd(fmin(fmax(v * f, -448.0), 448.0)) : __builtin_nanf("");
      }
      *p = u32x2{codes_of(y[0], y[1], y[2], y[3]), codes_of(y[4], y[5], y[6], y[7])};
    } else if (j < b.first && e2 > before) {
      const u32x2 w = *p;
      *p = u32x2{rescale(w[0], again), rescale(w[1], again)};
    }
  }
  if (lane == 0) *byte = static_cast<uint8_t>(e2 + 127);
}

template <int D>
__device__ __forceinline__ void append_values(const AppendArgs& a, const Block& b, int head, int lane) {
  typedef PageLayout<DSPARK_CACHE_FP8, D> PL;
  constexpr int DP = D / 64;  // dims of a lane
  if (!b.page) return;
  char* hp = b.page + head * PL::head_bytes(a.P);
  uint8_t* byte = reinterpret_cast<uint8_t*>(hp + PL::v_scale(a.P, b.t));
  const int before = b.first > 0 ? exponent_of(*byte) : kLow;
  const uint16_t* src = a.v + static_cast<int64_t>(head) * D + lane * DP;
  float x[DP][kBlock], top = 0.f;
#pragma unroll
  for (int j = 0; j < kBlock; ++j) {
    uint16_t v[DP];
#pragma unroll
    for (int d = 0; d < DP; ++d) v[d] = 0;
    if (j >= b.first && j < b.first + b.n)
      __builtin_memcpy(v, __builtin_assume_aligned(src + (b.row + j - b.first) * a.ldv, 2 * DP), 2 * DP);
#pragma unroll
    for (int d = 0; d < DP; ++d) x[d][j] = bf16_to_f32(v[d]);
  }
#pragma unroll
  for (int d = 0; d < DP; ++d)
#pragma unroll
    for (int j = 0; j < kBlock; ++j)
      if (fabsf(x[d][j]) <= 3.4028234e38f) top = fmaxf(top, fabsf(x[d][j]));
  top = over_lanes<32>(top, [](float p, float q) { return fmaxf(p, q); });
  top = fmaxf(top, xor32(top));
  const int e2 = max(before, exponent_for(top));
  const float f = ldexpf(1.f, -e2), again = ldexpf(1.f, before - e2);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // bits of the new tokens, and of the committed ones, among these eight
    const int lo = min(max(b.first - 8 * h, 0), 8), hi = min(max(b.first + b.n - 8 * h, 0), 8);
    const uint64_t upto = hi == 8 ? ~0ull : (1ull << (8 * hi)) - 1ull, old = lo == 8 ? ~0ull : (1ull << (8 * lo)) - 1ull;
    const uint64_t fresh = upto & ~old;
    const bool grown = old && e2 > before;
    if (!fresh && !grown) continue;
#pragma unroll
    for (int d = 0; d < DP; ++d) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = x[d][8 * h + j];
        y[j] = fabsf(v) <= 3.4028234e38f ? fminf(fmaxf(v * f, -kMost), kMost) : __builtin_nanf("");
      }
      u32x2 w{codes_of(y[0], y[1], y[2], y[3]), codes_of(y[4], y[5], y[6], y[7])};
      u32x2* p = reinterpret_cast<u32x2*>(hp + PL::v(a.P, b.t + 8 * h, lane * DP + d));
      if (fresh != ~0ull) {
        const u32x2 was = *p;
        const u32x2 kept = grown ? u32x2{rescale(was[0], again), rescale(was[1], again)} : was;
        const uint32_t n0 = static_cast<uint32_t>(fresh), n1 = static_cast<uint32_t>(fresh >> 32);
        const uint32_t o0 = static_cast<uint32_t>(old), o1 = static_cast<uint32_t>(old >> 32);
        w[0] = (w[0] & n0) | (kept[0] & o0) | (was[0] & ~(n0 | o0));
        w[1] = (w[1] & n1) | (kept[1] & o1) | (was[1] & ~(n1 | o1));
      }
      *p = w;
    }
  }
  if (lane == 0) *byte = static_cast<uint8_t>(e2 + 127);
}

// Work groups of a block: `parts` of keys and as many of values, four heads
// each, then those of queries.
template <int D>
__global__ __launch_bounds__(kThreads) void cache_append8_kernel(AppendArgs a, int parts) {
  constexpr int L = D / 8, kHeads = kThreads / L;
  __shared__ double lds[kBlock * D];
  const int r = blockIdx.z, y = blockIdx.y;
  const int half = a.rot / 2;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, li = threadIdx.x % L;
  // what does not depend on anything, at once
  const int n_rows = rows_of(a.ell[r], a.gamma);
  const int64_t len = a.len[r];
  const int64_t row0 = a.row0 ? static_cast<int64_t>(a.row0[r]) : static_cast<int64_t>(r) * (a.gamma + 1);
  const int pair0 = threadIdx.x - small_quotient(threadIdx.x, a.per_half) * half;
  const double freq0 = half ? a.freq[pair0] : 0.0;
  u32x4 w{0u, 0u, 0u, 0u};
  const uint16_t* norm = y < parts ? a.wk : a.wq;
  if (norm) w = *reinterpret_cast<const u32x4*>(norm + li * 8);
  if (len < 0) return;
  const int64_t base = (len / kBlock + blockIdx.x) * kBlock;
  const int64_t t0 = base > len ? base : len;
  const int64_t t1 = base + kBlock < len + n_rows ? base + kBlock : len + n_rows;
  if (t0 >= t1) return;
  const int64_t slot = base >> a.page_shift;
  const int id = slot < a.max_pages ? page_or_none(a.table[static_cast<int64_t>(r) * a.max_pages + slot], a.n_pages)
                                    : -1;
  const Block b{static_cast<int>(t0 - base), static_cast<int>(t1 - t0), row0 + (t0 - len), t0,
                static_cast<int>(base & (a.P - 1)), id >= 0 ? a.pool + id * a.page_bytes : nullptr};
  auto turns_of = [&](int row, int p, int i) {
    const double f = i == static_cast<int>(threadIdx.x) || kThreads % half == 0 ? freq0 : a.freq[p];
    const double turns = static_cast<double>(t0 + row) * f * 0.15915494309189535;
    return turns - rint(turns);
  };

  if (y < parts) {
    constexpr int RW = 64 / L, IT = kBlock / RW;
    const int head = min(4 * y + wave, a.Hkv - 1);
    u32x4 raw[IT];
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int j = it * RW + lane / L;
      raw[it] = u32x4{0u, 0u, 0u, 0u};
      if (j >= b.first && j < b.first + b.n)
        raw[it] = *reinterpret_cast<const u32x4*>(a.k + (b.row + j - b.first) * a.ldk + static_cast<int64_t>(head) * D + li * 8);
    }
    for (int i = threadIdx.x; i < b.n * half; i += kThreads) {
      const int row = small_quotient(i, a.per_half), p = i - row * half;
      double s, c;
      sincospi(2.0 * turns_of(row, p, i), &s, &c);
      lds[row * D + 2 * p] = c;
      lds[row * D + 2 * p + 1] = s;
    }
    __syncthreads();
    if (4 * y + wave < a.Hkv) append_keys<D>(a, b, head, lane, w, raw, lds);
    return;
  }
  if (y < 2 * parts) {
    const int head = 4 * (y - parts) + wave;
    if (head < a.Hkv) append_values<D>(a, b, head, lane);
    return;
  }
  // queries: a contiguous run of heads of rows, whole rounds of head slots
  const int nq = b.n * a.Hq;
  const int rounds = ceil_div(nq, kHeads * static_cast<int>(gridDim.y - 2 * parts));
  const int u_lo = (y - 2 * parts) * rounds * kHeads, u_hi = min(nq, u_lo + rounds * kHeads);
  if (u_lo >= u_hi) return;
  float* cs = reinterpret_cast<float*>(lds);
  auto source = [&](int u) {
    const int j = small_quotient(u, a.per_q);
    return a.q + (b.row + j) * a.ldq + (u - j * a.Hq) * D + li * 8;
  };
  int u = u_lo + threadIdx.x / L;
  u32x4 raw{0u, 0u, 0u, 0u};
  if (u < u_hi) raw = *reinterpret_cast<const u32x4*>(source(u));
  const int j_a = small_quotient(u_lo, a.per_q), j_b = small_quotient(u_hi - 1, a.per_q);
  for (int i = threadIdx.x; i < (j_b - j_a + 1) * half; i += kThreads) {
    const int j = small_quotient(i, a.per_half), p = i - j * half, row = j_a + j;
    float s, c;
    sincospif(2.f * static_cast<float>(turns_of(row, p, i)), &s, &c);
    cs[row * D + 2 * p] = c;
    cs[row * D + 2 * p + 1] = s;
  }
  __syncthreads();
#pragma unroll 1
  for (; u < u_hi; u += kHeads) {
    const u32x4 now = raw;
    if (u + kHeads < u_hi) raw = *reinterpret_cast<const u32x4*>(source(u + kHeads));
    const int j = small_quotient(u, a.per_q);
    float x[8];
    unpack(now, x);
    norm_rotate<float, D>(x, li, a.wq != nullptr, w, a.eps, a.rot, a.adjacent != 0, cs + j * D);
    *reinterpret_cast<u32x4*>(a.q_out + ((b.row + j) * a.Hq + (u - j * a.Hq)) * D + li * 8) = pack_bf16(x);
  }
}

template <int D>
hipError_t run(AppendArgs& a, hipStream_t s) {
  constexpr int kHeads = kThreads / (D / 8);
  a.page_bytes = a.Hkv * PageLayout<DSPARK_CACHE_FP8, D>::head_bytes(a.P);
  a.groups = ceil_div(a.gamma + kBlock, kBlock);  // aligned blocks that gamma + 1 tokens can touch
  const int64_t gx = static_cast<int64_t>(a.R) * a.groups;
  const int most = ceil_div(kBlock * a.Hq, kHeads);
  const int64_t want = 12LL * compute_units() / gx;
  const int gq = want < 1 ? 1 : want > most ? most : static_cast<int>(want);
  const int parts = ceil_div(a.Hkv, 4);
  a.page_shift = __builtin_ctz(a.P);
  a.per_q = 1.f / a.Hq;
  a.per_k = 1.f / a.Hkv;
  a.per_half = a.rot > 0 ? 2.f / a.rot : 0.f;
  cache_append8_kernel<D><<<dim3(a.groups, 2 * parts + gq, a.R), kThreads, 0, s>>>(a, parts);
  return hipGetLastError();
}

}  // namespace

hipError_t cache_append8_launch(int D, AppendArgs& a, hipStream_t s) {
  return D == 64 ? run<64>(a, s) : D == 128 ? run<128>(a, s) : run<256>(a, s);
}

}  // namespace dspark
