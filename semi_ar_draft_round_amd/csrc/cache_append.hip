// Norms of queries and keys per head, the position rotation in the same pass
// and the new tokens' K and V into the cache's pages; cached tokens back out
// as dense rows (include/dspark_cache.h).
//
// A work group takes the (at most 8) new tokens of one request that share an
// aligned group of 8 tokens: V is stored with a dim's 8 tokens together, so
// the group owns the 16-byte (4-bit: 4-byte) words it writes.  D / 8 lanes
// hold a head, 8 dims each: 16-byte loads, the sum of squares over those
// lanes, the rotation's partner a shuffle away (or in the same lane for
// adjacent pairs).  Sines and cosines of the group's positions are made once
// per work group in LDS and serve all heads.
#include "cache.hpp"

namespace dspark {

namespace {

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
};

__device__ __forceinline__ double shfl_xor_t(double x, int o) { return __shfl_xor(x, o); }
__device__ __forceinline__ float shfl_xor_t(float x, int o) { return __shfl_xor(x, o); }

__device__ __forceinline__ float inv_sqrt(float x) { return 1.f / sqrtf(x); }
__device__ __forceinline__ double inv_sqrt(double x) { return 1.0 / sqrt(x); }

// The norm and the rotation of one head, 8 dims per lane, in the type T.
// li: the lane's place in the head; cs: cosine and sine of pair i at 2 i.
template <typename T, int D>
__device__ __forceinline__ void norm_rotate(T (&x)[8], int li, const uint16_t* w, float eps, int rot, bool adjacent,
                                            const T* cs) {
  constexpr int L = D / 8;
  if (w) {
    T ss = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
    for (int o = 1; o < L; o <<= 1) ss += shfl_xor_t(ss, o);
    const T s = inv_sqrt(ss * static_cast<T>(1.0 / D) + static_cast<T>(eps));
    const u32x4 wv = *reinterpret_cast<const u32x4*>(w + li * 8);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = x[e] * s * static_cast<T>(bf16_to_f32(static_cast<uint16_t>(wv[e / 2] >> (16 * (e & 1)))));
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

__device__ __forceinline__ void unpack(const u32x4& v, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = bf16_to_f32(static_cast<uint16_t>(v[e / 2] >> (16 * (e & 1))));
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
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    top = fmax(top, shfl_xor_t(top, o));
    bad |= __shfl_xor(static_cast<int>(bad), o) != 0;
  }
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

// .. or one token, whose neighbours in those 16 bytes stay as they are.
__device__ __forceinline__ void store_v1_bf16(const uint16_t* src, char* dst) {
  const u32x4 x = *reinterpret_cast<const u32x4*>(src);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    *reinterpret_cast<uint16_t*>(dst + 16 * e) = static_cast<uint16_t>(x[e / 2] >> (16 * (e & 1)));
}

// V of one head of a 4-bit page: tokens first .. first + n - 1 of the group
// of 8 at src, a dim's 8 codes in one word; words with other tokens in them
// are read and merged.
template <int D>
__device__ __forceinline__ void store_v_fp4(const uint16_t* src, int64_t ldv, int li, int first, int n, char* head,
                                            int P, int t8) {
  typedef PageLayout<DSPARK_CACHE_FP4, D> L;
  u32x4 x[kGroup];
#pragma unroll
  for (int j = 0; j < kGroup; ++j) {
    x[j] = u32x4{0u, 0u, 0u, 0u};
    if (j >= first && j < first + n) x[j] = *reinterpret_cast<const u32x4*>(src + (j - first) * ldv);
  }
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = 0;
#pragma unroll
  for (int j = 0; j < kGroup; ++j) {
    if (j < first || j >= first + n) continue;  // the same for all lanes of the head
    float f[8], top = 0.f;
    bool bad = false;
    unpack(x[j], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      top = fmaxf(top, fabsf(f[e]));
      bad |= !(fabsf(f[e]) <= 3.4028234e38f);
    }
#pragma unroll
    for (int o = 1; o < D / 8; o <<= 1) {
      top = fmaxf(top, __shfl_xor(top, o));
      bad |= __shfl_xor(static_cast<int>(bad), o) != 0;
    }
    // 6 |v| against the borders times max |v|: products of 16-bit values with
    // numbers of at most 3 bits, exact in fp32; above 2^100 both sides are
    // scaled down first so that they stay finite
    const float sc = top > 1.2676506e30f ? 7.8886091e-31f : 1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      w[e] |= (bad || top == 0.f ? 0u : code_of(6.f * (f[e] * sc), top * sc)) << (4 * j);
    if (li == 0) *reinterpret_cast<float*>(head + L::v_scale(P, t8 + j)) = bad ? __builtin_nanf("") : top / 6.f;
  }
  const uint32_t mine = static_cast<uint32_t>(((1ull << (4 * n)) - 1ull) << (4 * first));
  // dims 8 li .. of a group of 32: consecutive in the first of the two dim axes
  uint32_t* p = reinterpret_cast<uint32_t*>(head + L::v(P, t8, li * 8));
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e * L::E] = n == kGroup ? w[e] : (p[e * L::E] & ~mine) | w[e];
}

template <int FMT, int D>
__global__ __launch_bounds__(kThreads, 4) void cache_append_kernel(AppendArgs a) {
  constexpr int L = D / 8, kHeads = kThreads / L;  // head slots of the work group
  // keys of 4-bit pages need fp64 sines as well
  __shared__ float cs[kGroup * D];
  __shared__ double cs64[FMT == DSPARK_CACHE_FP4 ? kGroup * D : 1];
  const int r = blockIdx.x / a.groups, g = blockIdx.x % a.groups;
  const int n_rows = rows_of(a.ell[r], a.gamma);
  const int64_t len = a.len[r];
  if (len < 0) return;
  // tokens [t0, t1) of this group
  const int64_t base = (len / kGroup + g) * kGroup;
  const int64_t t0 = base > len ? base : len;
  const int64_t t1 = base + kGroup < len + n_rows ? base + kGroup : len + n_rows;
  if (t0 >= t1) return;
  const int n = static_cast<int>(t1 - t0), first = static_cast<int>(t0 - base);
  const int64_t row_first =
      (a.row0 ? static_cast<int64_t>(a.row0[r]) : static_cast<int64_t>(r) * (a.gamma + 1)) + (t0 - len);
  const int64_t slot = base / a.P;
  const int id = slot < a.max_pages ? page_or_none(a.table[static_cast<int64_t>(r) * a.max_pages + slot], a.n_pages)
                                    : -1;
  const int t8 = static_cast<int>(base % a.P);
  char* page = id >= 0 ? a.pool + id * a.page_bytes : nullptr;

  // a unit is one head of one row (q, k, and V one row at a time), or V of a
  // head for a whole group; every lane of a head slot takes the same unit, so
  // the shuffles inside a head are whole
  const int li = threadIdx.x % L;
  const int per_row = a.Hq + a.Hkv;
  const bool whole = FMT == DSPARK_CACHE_FP4 || n == kGroup;
  const int units = n * per_row + (whole ? a.Hkv : n * a.Hkv);
  int u = blockIdx.y * kHeads + threadIdx.x / L;
  // V and the first row need no angles: they are on their way while those are made
  auto row_of = [&](int unit, const uint16_t** src) {
    const int j = unit / per_row, head = unit - j * per_row;
    *src = head < a.Hq ? a.q + (row_first + j) * a.ldq + head * D
                       : a.k + (row_first + j) * a.ldk + (head - a.Hq) * D;
    return j;
  };
  u32x4 raw{0u, 0u, 0u, 0u};
  if (u < n * per_row) {
    const uint16_t* src;
    row_of(u, &src);
    raw = *reinterpret_cast<const u32x4*>(src + li * 8);
  }
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int row = i / half, p = i - row * half;
    const double turns = static_cast<double>(t0 + row) * a.freq[p] * 0.15915494309189535;
    const double t = turns - rint(turns);
    if constexpr (FMT == DSPARK_CACHE_FP4) {
      double s, c;
      sincospi(2.0 * t, &s, &c);
      cs64[row * D + 2 * p] = c;
      cs64[row * D + 2 * p + 1] = s;
      cs[row * D + 2 * p] = static_cast<float>(c);
      cs[row * D + 2 * p + 1] = static_cast<float>(s);
    } else {
      float s, c;
      sincospif(2.f * static_cast<float>(t), &s, &c);
      cs[row * D + 2 * p] = c;
      cs[row * D + 2 * p + 1] = s;
    }
  }
  __syncthreads();

#pragma unroll 1
  for (; u < units; u += gridDim.y * kHeads) {
    if (u >= n * per_row) {
      const int v = u - n * per_row;
      const int h = whole ? v : v % a.Hkv, j = whole ? 0 : v / a.Hkv;
      const uint16_t* src = a.v + (row_first + j) * a.ldv + static_cast<int64_t>(h) * D + li * 8;
      if (!page) continue;
      char* head = page + h * PageLayout<FMT, D>::head_bytes(a.P);
      if constexpr (FMT == DSPARK_CACHE_BF16) {
        char* dst = head + PageLayout<FMT, D>::v(a.P, t8, li * 8);
        if (whole) store_v8_bf16<D>(src, a.ldv, dst);
        else store_v1_bf16(src, dst + 2 * (first + j));
      } else {
        store_v_fp4<D>(src, a.ldv, li, first, n, head, a.P, t8);
      }
      continue;
    }
    const uint16_t* src;
    const int j = row_of(u, &src), head = u - j * per_row;
    const bool is_q = head < a.Hq;
    const u32x4 now = raw;
    const int next = u + gridDim.y * kHeads;
    if (next < n * per_row) {
      row_of(next, &src);
      raw = *reinterpret_cast<const u32x4*>(src + li * 8);
    }
    if constexpr (FMT == DSPARK_CACHE_FP4) {
      if (!is_q) {
        float f[8];
        unpack(now, f);
        double x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = f[e];
        norm_rotate<double, D>(x, li, a.wk, a.eps, a.rot, a.adjacent != 0, cs64 + j * D);
        if (page)
          store_k_fp4<D>(x, li, page + (head - a.Hq) * PageLayout<FMT, D>::head_bytes(a.P), a.P, t8 + first + j);
        continue;
      }
    }
    float x[8];
    unpack(now, x);
    norm_rotate<float, D>(x, li, is_q ? a.wq : a.wk, a.eps, a.rot, a.adjacent != 0, cs + j * D);
    const u32x4 y = pack_bf16(x);
    if (is_q) {
      *reinterpret_cast<u32x4*>(a.q_out + ((row_first + j) * a.Hq + head) * D + li * 8) = y;
    } else if (page) {
      char* hp = page + (head - a.Hq) * PageLayout<FMT, D>::head_bytes(a.P);
      if constexpr (FMT == DSPARK_CACHE_BF16)
        *reinterpret_cast<u32x4*>(hp + PageLayout<FMT, D>::k(a.P, t8 + first + j, li)) = y;
    }
  }
}

struct ReadArgs {
  int R, T, Hkv, P, n_pages, max_pages, groups;
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
  const int r = blockIdx.x / a.groups, g = blockIdx.x % a.groups;
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
  // enough work groups along the heads to fill the device when there are few token groups
  const int most = ceil_div(kGroup * (a.Hq + a.Hkv) + a.Hkv, kHeads);
  const int64_t want = 16LL * compute_units() / gx;
  const int gy = want < 1 ? 1 : want > most ? most : static_cast<int>(want);
  cache_append_kernel<FMT, D><<<dim3(static_cast<unsigned>(gx), gy), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <int FMT, int D>
hipError_t read_run(ReadArgs& a, hipStream_t s) {
  constexpr int kHeads = kThreads / (D / 8);
  a.page_bytes = a.Hkv * PageLayout<FMT, D>::head_bytes(a.P);
  a.groups = ceil_div(a.T - 1 + kGroup, kGroup);
  const int64_t gx = static_cast<int64_t>(a.R) * a.groups;
  cache_read_kernel<FMT, D><<<dim3(static_cast<unsigned>(gx), ceil_div(2 * a.Hkv, kHeads)), kThreads, 0, s>>>(a);
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

hipError_t cache_append_launch(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages, int max_pages,
                               const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                               const void* wq, const void* wk, float eps, const double* freq, int rot, int adjacent,
                               const int32_t* row0, const int32_t* ell, const int32_t* len, const int32_t* table,
                               void* q_out, void* pool, hipStream_t s) {
  AppendArgs a{R, gamma, Hq, Hkv, P, n_pages, max_pages, 0,
               static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
               ldq, ldk, ldv, static_cast<const uint16_t*>(wq), static_cast<const uint16_t*>(wk), eps, freq, rot,
               adjacent, row0, ell, len, table, static_cast<uint16_t*>(q_out), static_cast<char*>(pool), 0};
  return fmt == DSPARK_CACHE_BF16 ? append_d<DSPARK_CACHE_BF16>(D, a, s) : append_d<DSPARK_CACHE_FP4>(D, a, s);
}

hipError_t cache_read_launch(int fmt, int R, int T, int Hkv, int D, int P, int n_pages, int max_pages,
                             const int32_t* start, const int32_t* count, const int32_t* table, const void* pool,
                             void* k, void* v, hipStream_t s) {
  ReadArgs a{R, T, Hkv, P, n_pages, max_pages, 0, start, count, table, static_cast<const char*>(pool), 0,
             static_cast<uint16_t*>(k), static_cast<uint16_t*>(v)};
  return fmt == DSPARK_CACHE_BF16 ? read_d<DSPARK_CACHE_BF16>(D, a, s) : read_d<DSPARK_CACHE_FP4>(D, a, s);
}

}  // namespace dspark
