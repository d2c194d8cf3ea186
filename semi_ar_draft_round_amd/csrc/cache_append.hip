// Norms of queries and keys per head, the position rotation in the same pass
// and the new tokens' K and V into the cache's pages; cached tokens back out
// as dense rows (include/dspark_cache.h).
//
// A group is the (at most 8) new tokens of one request that share an aligned
// group of 8 tokens: V is stored with a dim's 8 tokens together, so whoever
// works on the group owns the 16-byte (4-bit: 4-byte) words it writes.  D / 8
// lanes hold a head, 8 dims each: 16-byte loads, the sum of squares over those
// lanes, the rotation's partner a shuffle away (or in the same lane for
// adjacent pairs).  Several work groups share a group's heads, each a
// contiguous run of them, so that each makes the sines and cosines of the few
// rows it works on, in LDS, for all its heads.
//
// Latency bounds it: a chain of loads (the length, the page's id, the row),
// the sines, one pass over the rows.  GPU time with heads of 128 dims and 8
// heads of keys: one token, 32 query heads, 3.5 us; 128 requests of up to 17
// packed rows, 56 query heads, 12.3 us (15.1 with the sums over a head and the
// rotation's partners through LDS instead of lane patterns), of which V of
// groups that are not whole, in 2-byte stores, is 1.8; 4 x 512 rows 14.5 us.
#include "cache_rows.hpp"

namespace dspark {

namespace {

// e2m1 code of x / one for 16-bit x and one, or of fp64 x with one = 1: the
// borders are multiples of `one`, exact in T.  Nearest, ties to the even code.
template <typename T>
__device__ __forceinline__ uint32_t code_of(T x, T one) {
  const T y = x < 0 ? -x : x;
  const uint32_t c = (y > static_cast<T>(0.25) * one) + (y >= static_cast<T>(0.75) * one) +
                     (y > static_cast<T>(1.25) * one) + (y >= static_cast<T>(1.75) * one) +
                     (y > static_cast<T>(2.5) * one) + (y >= static_cast<T>(3.5) * one) +
                     (y > static_cast<T>(5.0) * one);
  return c | (x < 0 ? 8u : 0u);
}

// One key head into a 4-bit page, fp64 throughout: lane li holds 8 of the 32
// dims of a scale group, four lanes make the group.
template <int D>
__device__ __forceinline__ void store_k_fp4(const double (&x)[8], int li, char* head, int P, int t) {
  typedef PageLayout<DSPARK_CACHE_FP4, D> L;
  double top = 0;
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    top = fmax(top, fabs(x[e]));
    bad |= !(fabs(x[e]) < 3.4028236692093846e38);  // 2^128
  }
  top = over_lanes<4>(top, [](double p, double q) { return fmax(p, q); });
  bad = over_lanes<4>(static_cast<int>(bad), [](int p, int q) { return p | q; }) != 0;
  int e2 = -126;
  if (top > 0 && !bad) {
    e2 = ilogb(top) - 2;                    // top / 2^e2 in [4, 8)
    if (ldexp(top, -e2) > 7.0) ++e2;
    e2 = min(125, max(-126, e2));           // 6 * 2^125 is the largest finite bf16 value of a code
  }
  uint32_t w = 0;
  const double f = bad ? 0.0 : ldexp(1.0, -e2);
#pragma unroll
  for (int e = 0; e < 8; ++e) w |= (bad ? 0u : code_of(x[e] * f, 1.0)) << (4 * e);
  *reinterpret_cast<uint32_t*>(head + L::k(P, t, li / 4) + (li & 3) * 4) = w;
  if ((li & 3) == 0) head[L::k_scale(P, t) + li / 4] = static_cast<char>(bad ? 255 : e2 + 127);
}

// V of one head of a 16-bit page: all 8 tokens of the group, transposed in
// registers so that every store is a dim's 16 bytes ..
template <int D>
__device__ __forceinline__ void store_v8_bf16(const uint16_t* src, int64_t ldv, char* dst) {
  u32x4 x[kGroup];
#pragma unroll
  for (int j = 0; j < kGroup; ++j) x[j] = *reinterpret_cast<const u32x4*>(src + j * ldv);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = __builtin_amdgcn_perm(x[2 * j + 1][e / 2], x[2 * j][e / 2], (e & 1) ? 0x07060302u : 0x05040100u);
    *reinterpret_cast<u32x4*>(dst + 16 * e) = w;
  }
}

// .. or one token, whose neighbours in those 16 bytes stay as they are: a
// lane takes dims li, li + L, .., so that a store's lanes lie side by side
// (eight dims a line) and not a line apart.
template <int D>
__device__ __forceinline__ void store_v1_bf16(const uint16_t* src, int li, char* dst) {
  constexpr int L = D / 8;
  uint16_t x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = src[e * L + li];
#pragma unroll
  for (int e = 0; e < 8; ++e) *reinterpret_cast<uint16_t*>(dst + 16 * (e * L + li)) = x[e];
}

// V of one head of a 4-bit page, a token a head slot: the slots of a wave
// hold 64 / (D / 8) tokens of the group in turn, make their codes, and put
// them together into the part of a dim's word that these tokens fill: 4, 2 or
// 1 bytes for heads of 64, 128 and 256 dims.  src: the lane's 8 dims of token
// j if that is new (j in first .. first + n - 1), else unused.
template <int D>
__device__ __forceinline__ void store_v_fp4(const uint16_t* src, int li, int j, int first, int n, char* head, int P,
                                            int t8) {
  typedef PageLayout<DSPARK_CACHE_FP4, D> L;
  constexpr int kLanes = D / 8, kTokens = 64 / kLanes;
  const bool mine = j >= first && j < first + n;
  u32x4 x{0u, 0u, 0u, 0u};
  if (mine) x = *reinterpret_cast<const u32x4*>(src);
  float f[8], top = 0.f;
  bool bad = false;
  unpack(x, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    top = fmaxf(top, fabsf(f[e]));
    bad |= !(fabsf(f[e]) <= 3.4028234e38f);
  }
  top = over_lanes<kLanes>(top, [](float p, float q) { return fmaxf(p, q); });
  bad = over_lanes<kLanes>(static_cast<int>(bad), [](int p, int q) { return p | q; }) != 0;
  // 6 |v| against the borders times max |v|: products of 16-bit values with
  // numbers of at most 3 bits, exact in fp32; above 2^100 both sides are
  // scaled down first so that they stay finite
  const float sc = top > 1.2676506e30f ? 7.8886091e-31f : 1.f;
  const int j0 = j & ~(kTokens - 1), at = 4 * (j - j0);
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = (bad || top == 0.f ? 0u : code_of(6.f * (f[e] * sc), top * sc)) << at;
#pragma unroll
  for (int o = kLanes; o < 64; o <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] |= static_cast<uint32_t>(__shfl_xor(static_cast<int>(w[e]), o));
  if (mine && li == 0) *reinterpret_cast<float*>(head + L::v_scale(P, t8 + j)) = bad ? __builtin_nanf("") : top / 6.f;
  // bits of the new tokens among these; each slot stores its share of the 8 dims
  const int lo = max(first, j0) - j0, hi = min(first + n, j0 + kTokens) - j0;
  if (lo >= hi) return;
  const uint32_t bits = static_cast<uint32_t>(((1ull << (4 * (hi - lo))) - 1ull) << (4 * lo));
  const int part = j - j0;
  char* p = head + L::v(P, t8, li * 8) + j0 / 2;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e % kTokens == part) {
      // dims 8 li .. of a group of 32 are consecutive in the first of the two dim axes
      char* q = p + e * (4 * L::E);
      if constexpr (kTokens == 8) {
        uint32_t* z = reinterpret_cast<uint32_t*>(q);
        *z = hi - lo == 8 ? w[e] : (*z & ~bits) | w[e];
      } else if constexpr (kTokens == 4) {
        uint16_t* z = reinterpret_cast<uint16_t*>(q);
        *z = static_cast<uint16_t>(hi - lo == 4 ? w[e] : (*z & ~bits) | w[e]);
      } else {
        uint8_t* z = reinterpret_cast<uint8_t*>(q);
        *z = static_cast<uint8_t>(hi - lo == 2 ? w[e] : (*z & ~bits) | w[e]);
      }
    }
}

// A unit is a head slot's work: one head of one row for q and k; V of a 16-bit
// page by head (whole groups) or head and row, of a 4-bit page by head and
// token of the group.  In that order, so that the fp64 angles of 4-bit keys
// are made by the few work groups that hold such units.
template <int FMT, int D>
__global__ __launch_bounds__(kThreads, 4) void cache_append_kernel(AppendArgs a) {
  constexpr int L = D / 8, kHeads = kThreads / L;  // head slots of the work group
  __shared__ float cs[kGroup * D];
  __shared__ double cs64[FMT == DSPARK_CACHE_FP4 ? kGroup * D : 1];
  const int r = blockIdx.z, g = blockIdx.x;
  const int half = a.rot / 2;
  // what does not depend on anything, at once
  const int n_rows = rows_of(a.ell[r], a.gamma);
  const int64_t len = a.len[r];
  const int64_t row0 = a.row0 ? static_cast<int64_t>(a.row0[r]) : static_cast<int64_t>(r) * (a.gamma + 1);
  const int pair0 = threadIdx.x - small_quotient(threadIdx.x, a.per_half) * half;
  const double freq0 = half ? a.freq[pair0] : 0.0;
  const int li = threadIdx.x % L;
  u32x4 w_q{0u, 0u, 0u, 0u}, w_k{0u, 0u, 0u, 0u};
  if (a.wq) w_q = *reinterpret_cast<const u32x4*>(a.wq + li * 8);
  if (a.wk) w_k = *reinterpret_cast<const u32x4*>(a.wk + li * 8);
  if (len < 0) return;
  // tokens [t0, t1) of this group
  const int64_t base = (len / kGroup + g) * kGroup;
  const int64_t t0 = base > len ? base : len;
  const int64_t t1 = base + kGroup < len + n_rows ? base + kGroup : len + n_rows;
  if (t0 >= t1) return;
  const int n = static_cast<int>(t1 - t0), first = static_cast<int>(t0 - base);
  const int nq = n * a.Hq, nqk = nq + n * a.Hkv;
  const bool whole = n == kGroup;
  const int v0 = FMT == DSPARK_CACHE_FP4 ? (nqk + kGroup - 1) / kGroup * kGroup : nqk;
  const int units = v0 + (FMT == DSPARK_CACHE_FP4 ? a.Hkv * kGroup : whole ? a.Hkv : n * a.Hkv);
  // this work group's run of them, whole rounds of kHeads
  const int rounds = ceil_div(units, kHeads * static_cast<int>(gridDim.y));
  const int u_lo = blockIdx.y * rounds * kHeads, u_hi = min(units, u_lo + rounds * kHeads);
  if (u_lo >= u_hi) return;
  const int64_t row_first = row0 + (t0 - len);
  const int64_t slot = base >> a.page_shift;
  const int id = slot < a.max_pages ? page_or_none(a.table[static_cast<int64_t>(r) * a.max_pages + slot], a.n_pages)
                                    : -1;
  const int t8 = static_cast<int>(base & (a.P - 1));
  char* page = id >= 0 ? a.pool + id * a.page_bytes : nullptr;

  // row and source of a q or k unit
  auto row_of = [&](int u) { return u < nq ? small_quotient(u, a.per_q) : small_quotient(u - nq, a.per_k); };
  auto source = [&](int u, int j) {
    return u < nq ? a.q + (row_first + j) * a.ldq + (u - j * a.Hq) * D
                  : a.k + (row_first + j) * a.ldk + (u - nq - j * a.Hkv) * D;
  };
  int u = u_lo + threadIdx.x / L;
  u32x4 raw{0u, 0u, 0u, 0u};  // the next q or k unit's values, loaded a round ahead
  if (u < min(u_hi, nqk)) raw = *reinterpret_cast<const u32x4*>(source(u, row_of(u)) + li * 8);

  // sines and cosines of the rows of this run's q and k units
  const bool has_q = u_lo < nq, has_k = u_hi > nq && u_lo < nqk;
  const int k_a = has_k ? row_of(max(u_lo, nq)) : 0, k_b = has_k ? row_of(min(u_hi, nqk) - 1) : -1;
  const int q_a = has_q ? row_of(u_lo) : k_a, q_b = has_q ? row_of(min(u_hi, nq) - 1) : k_b;
  const int j_a = has_k ? min(q_a, k_a) : q_a, j_b = max(q_b, k_b);
  for (int i = threadIdx.x; i < (j_b - j_a + 1) * half; i += kThreads) {
    const int j = small_quotient(i, a.per_half), p = i - j * half, row = j_a + j;
    const double f = i == static_cast<int>(threadIdx.x) || kThreads % half == 0 ? freq0 : a.freq[p];
    const double turns = static_cast<double>(t0 + row) * f * 0.15915494309189535;
    const double t = turns - rint(turns);
    // queries always get the fp32 ones, whatever else this run holds: a row's
    // bits do not depend on how the work is cut
    float s, c;
    sincospif(2.f * static_cast<float>(t), &s, &c);
    if (FMT == DSPARK_CACHE_FP4 && row >= k_a && row <= k_b) {
      double s64, c64;
      sincospi(2.0 * t, &s64, &c64);
      cs64[FMT == DSPARK_CACHE_FP4 ? row * D + 2 * p : 0] = c64;
      cs64[FMT == DSPARK_CACHE_FP4 ? row * D + 2 * p + 1 : 0] = s64;
    }
    cs[row * D + 2 * p] = c;
    cs[row * D + 2 * p + 1] = s;
  }
  __syncthreads();

#pragma unroll 1
  for (; u < u_hi; u += kHeads) {
    if (u >= v0) {
      if (!page) continue;
      const int v = u - v0;
      if constexpr (FMT == DSPARK_CACHE_BF16) {
        const int j = whole ? 0 : small_quotient(v, a.per_k), h = v - j * a.Hkv;
        const uint16_t* src = a.v + (row_first + j) * a.ldv + static_cast<int64_t>(h) * D;
        char* dst = page + h * PageLayout<FMT, D>::head_bytes(a.P) + PageLayout<FMT, D>::v(a.P, t8, 0);
        if (whole) store_v8_bf16<D>(src + li * 8, a.ldv, dst + 128 * li);
        else store_v1_bf16<D>(src, li, dst + 2 * (first + j));
      } else {
        const int h = v / kGroup, j = v % kGroup;
        store_v_fp4<D>(a.v + (row_first + j - first) * a.ldv + static_cast<int64_t>(h) * D + li * 8, li, j, first, n,
                       page + h * PageLayout<FMT, D>::head_bytes(a.P), a.P, t8);
      }
      continue;
    }
    if (u >= nqk) continue;  // between the keys and V's whole rounds
    const u32x4 now = raw;
    if (u + kHeads < min(u_hi, nqk)) raw = *reinterpret_cast<const u32x4*>(source(u + kHeads, row_of(u + kHeads)) + li * 8);
    const int j = row_of(u);
    const bool is_q = u < nq;
    const int head = is_q ? u - j * a.Hq : u - nq - j * a.Hkv;
    if constexpr (FMT == DSPARK_CACHE_FP4) {
      if (!is_q) {
        float f[8];
        unpack(now, f);
        double x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = f[e];
        norm_rotate<double, D>(x, li, a.wk != nullptr, w_k, a.eps, a.rot, a.adjacent != 0, cs64 + j * D);
        if (page) store_k_fp4<D>(x, li, page + head * PageLayout<FMT, D>::head_bytes(a.P), a.P, t8 + first + j);
        continue;
      }
    }
    float x[8];
    unpack(now, x);
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = is_q ? w_q[e] : w_k[e];
    norm_rotate<float, D>(x, li, is_q ? a.wq != nullptr : a.wk != nullptr, w, a.eps, a.rot, a.adjacent != 0, cs + j * D);
    const u32x4 y = pack_bf16(x);
    if (is_q) {
      *reinterpret_cast<u32x4*>(a.q_out + ((row_first + j) * a.Hq + head) * D + li * 8) = y;
    } else if (page) {
      char* hp = page + head * PageLayout<FMT, D>::head_bytes(a.P);
      if constexpr (FMT == DSPARK_CACHE_BF16)
        *reinterpret_cast<u32x4*>(hp + PageLayout<FMT, D>::k(a.P, t8 + first + j, li)) = y;
    }
  }
}

struct ReadArgs {
  int R, T, Hkv, P, n_pages, max_pages;
  const int32_t *start, *count, *table;
  const char* pool;
  int64_t page_bytes;
  uint16_t *k, *v;
};

// The append's units the other way round: a lane reads the 8 tokens of its 8
// dims (V) or one token's 8 dims (K) and writes 16-byte pieces of the rows.
template <int FMT, int D>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(ReadArgs a) {
  typedef PageLayout<FMT, D> PL;
  constexpr int L = D / 8, kHeads = kThreads / L;
  const int r = blockIdx.z, g = blockIdx.x;
  const int64_t start = a.start ? a.start[r] : 0;
  const int n_rows = min(max(a.count[r], 0), a.T);
  if (start < 0) return;
  const int64_t base = (start / kGroup + g) * kGroup;
  const int64_t t0 = base > start ? base : start;
  const int64_t t1 = base + kGroup < start + n_rows ? base + kGroup : start + n_rows;
  if (t0 >= t1) return;
  const int64_t slot = base / a.P;
  const int id = slot < a.max_pages ? page_or_none(a.table[static_cast<int64_t>(r) * a.max_pages + slot], a.n_pages)
                                    : -1;
  const int t8 = static_cast<int>(base % a.P);
  const int first = static_cast<int>(t0 - base), n = static_cast<int>(t1 - t0);
  const int64_t row_first = static_cast<int64_t>(r) * a.T + (t0 - start);
  const int li = threadIdx.x % L;
  for (int u = blockIdx.y * kHeads + threadIdx.x / L; u < 2 * a.Hkv; u += gridDim.y * kHeads) {
    const int h = u >> 1;
    const char* head = id >= 0 ? a.pool + id * a.page_bytes + h * PL::head_bytes(a.P) : nullptr;
    u32x4 x[kGroup];
#pragma unroll
    for (int j = 0; j < kGroup; ++j) x[j] = u32x4{0u, 0u, 0u, 0u};
    if (head && (u & 1) == 0) {
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
        if (j >= first && j < first + n) {
          if constexpr (FMT == DSPARK_CACHE_BF16) {
            x[j] = *reinterpret_cast<const u32x4*>(head + PL::k(a.P, t8 + j, li));
          } else if constexpr (FMT == DSPARK_CACHE_FP8) {
            const u32x2 w = *reinterpret_cast<const u32x2*>(head + PL::k(a.P, t8 + j, li / 2) + (li & 1) * 8);
            x[j] = fp8_octet(w[0], w[1], k_scale_value(static_cast<uint8_t>(head[PL::k_scale(a.P, t8)])));
          } else {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(head + PL::k(a.P, t8 + j, li / 4) + (li & 3) * 4);
            x[j] = fp4_octet(w, k_scale_value(static_cast<uint8_t>(head[PL::k_scale(a.P, t8 + j) + li / 4])));
          }
        }
    } else if (head) {
      u32x4 y[8];  // y[e]: 8 tokens of dim li * 8 + e, as bf16
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (FMT == DSPARK_CACHE_BF16) {
          y[e] = *reinterpret_cast<const u32x4*>(head + PL::v(a.P, t8, li * 8 + e));
        } else if constexpr (FMT == DSPARK_CACHE_FP8) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(head + PL::v(a.P, t8, li * 8 + e));
          y[e] = fp8_octet(w[0], w[1], k_scale_value(static_cast<uint8_t>(head[PL::v_scale(a.P, t8)])));
        } else {
          const u32x4 c = fp4_octet(*reinterpret_cast<const uint32_t*>(head + PL::v(a.P, t8, li * 8 + e)), 1.f);
          const float* sc = reinterpret_cast<const float*>(head + PL::v_scale(a.P, t8));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            y[e][j] = bf16_pair(bf16_to_f32(static_cast<uint16_t>(c[j])) * sc[2 * j],
                                bf16_to_f32(static_cast<uint16_t>(c[j] >> 16)) * sc[2 * j + 1]);
        }
      }
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[j][e] = ((y[2 * e][j / 2] >> (16 * (j & 1))) & 0xFFFFu) |
                    ((y[2 * e + 1][j / 2] >> (16 * (j & 1))) & 0xFFFFu) << 16;
    }
    uint16_t* out = (u & 1) ? a.v : a.k;
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
      if (j >= first && j < first + n)
        *reinterpret_cast<u32x4*>(out + ((row_first + j - first) * a.Hkv + h) * D + li * 8) = x[j];
  }
}

template <int FMT, int D>
hipError_t append_run(AppendArgs& a, hipStream_t s) {
  constexpr int kHeads = kThreads / (D / 8);
  a.page_bytes = a.Hkv * PageLayout<FMT, D>::head_bytes(a.P);
  a.groups = ceil_div(a.gamma + kGroup, kGroup);  // aligned groups that gamma + 1 tokens can touch
  const int64_t gx = static_cast<int64_t>(a.R) * a.groups;
  // a round of head slots a work group where there are few token groups, else
  // about 12 work groups a compute unit (4 at a time): 128 x 17 packed rows and
  // 4 x 512 rows take 12.3 and 14.5 us, with 8 a unit 11.9 and 15.0, with 24
  // 14.0 and 17.8; 32 x 17 rows of 4-bit pages with their read 15.8, 16.9, 15.9
  const int v_units = FMT == DSPARK_CACHE_FP4 ? kGroup * a.Hkv + kGroup - 1 : kGroup * a.Hkv;
  const int most = ceil_div(kGroup * (a.Hq + a.Hkv) + v_units, kHeads);
  const int64_t want = 12LL * compute_units() / gx;
  const int gy = want < 1 ? 1 : want > most ? most : static_cast<int>(want);
  a.page_shift = __builtin_ctz(a.P);
  a.per_q = 1.f / a.Hq;
  a.per_k = 1.f / a.Hkv;
  a.per_half = a.rot > 0 ? 2.f / a.rot : 0.f;
  cache_append_kernel<FMT, D><<<dim3(a.groups, gy, a.R), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <int FMT, int D>
hipError_t read_run(ReadArgs& a, hipStream_t s) {
  constexpr int kHeads = kThreads / (D / 8);
  a.page_bytes = a.Hkv * PageLayout<FMT, D>::head_bytes(a.P);
  const int groups = ceil_div(a.T - 1 + kGroup, kGroup);
  cache_read_kernel<FMT, D><<<dim3(groups, ceil_div(2 * a.Hkv, kHeads), a.R), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <int FMT>
hipError_t append_d(int D, AppendArgs& a, hipStream_t s) {
  return D == 64 ? append_run<FMT, 64>(a, s) : D == 128 ? append_run<FMT, 128>(a, s) : append_run<FMT, 256>(a, s);
}
template <int FMT>
hipError_t read_d(int D, ReadArgs& a, hipStream_t s) {
  return D == 64 ? read_run<FMT, 64>(a, s) : D == 128 ? read_run<FMT, 128>(a, s) : read_run<FMT, 256>(a, s);
}

}  // namespace

// cache_append8.hip
hipError_t cache_append8_launch(int D, AppendArgs& a, hipStream_t s);

hipError_t cache_append_launch(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages, int max_pages,
                               const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                               const void* wq, const void* wk, float eps, const double* freq, int rot, int adjacent,
                               const int32_t* row0, const int32_t* ell, const int32_t* len, const int32_t* table,
                               void* q_out, void* pool, hipStream_t s) {
  AppendArgs a{R, gamma, Hq, Hkv, P, n_pages, max_pages, 0,
               static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
               ldq, ldk, ldv, static_cast<const uint16_t*>(wq), static_cast<const uint16_t*>(wk), eps, freq, rot,
               adjacent, row0, ell, len, table, static_cast<uint16_t*>(q_out), static_cast<char*>(pool), 0, 0, 0.f,
               0.f, 0.f};
  return fmt == DSPARK_CACHE_BF16   ? append_d<DSPARK_CACHE_BF16>(D, a, s)
         : fmt == DSPARK_CACHE_FP8 ? cache_append8_launch(D, a, s)
                                   : append_d<DSPARK_CACHE_FP4>(D, a, s);
}

hipError_t cache_read_launch(int fmt, int R, int T, int Hkv, int D, int P, int n_pages, int max_pages,
                             const int32_t* start, const int32_t* count, const int32_t* table, const void* pool,
                             void* k, void* v, hipStream_t s) {
  ReadArgs a{R, T, Hkv, P, n_pages, max_pages, start, count, table, static_cast<const char*>(pool), 0,
             static_cast<uint16_t*>(k), static_cast<uint16_t*>(v)};
  return fmt == DSPARK_CACHE_BF16   ? read_d<DSPARK_CACHE_BF16>(D, a, s)
         : fmt == DSPARK_CACHE_FP8 ? read_d<DSPARK_CACHE_FP8>(D, a, s)
                                   : read_d<DSPARK_CACHE_FP4>(D, a, s);
}

}  // namespace dspark
