// The append into 8-bit pages: norms and rotation as for the other formats,
// and blocks of 16 tokens that share a scale (include/dspark_cache.h).
//
// A block's scale is known when all of its new rows are, so a task is a
// block's keys of some heads, or its values: the rows are held in registers,
// their largest magnitudes meet in LDS, the scale that the block's committed
// tokens have is compared, and codes are written.  Only where the scale grew
// are the committed tokens' codes read, rounded again and written back.  With
// two threads a dim, whatever D is, a task has 16 slots of D / 8 threads:
//   keys     a slot for a (head, row): as many heads as have room, so that the
//            few rows that most requests bring fill the work group; fp64, so
//            that a code does not depend on the order of a sum (but in the last
//            bit of its sines, which are made by turning on from a run's first);
//   values   a thread for a dim's 8 tokens, a word of the pages: one head, or
//            two where the rows touch one half of the block;
//   queries  a slot for a (row, head).
//
// A code is rounded once: fp64 is cut to fp32 with what was cut off kept in
// the last bit (a value between two codes, or between a code and the border
// beside it, stays there), and the conversion rounds that.
//
// What bounds it is latency: the length, the page's id, the rows and the block's
// codes are loads one after another, and a block's bounds need all of its rows.
// With 8 heads of keys of 128 dims: one token, 32 query heads, 4.5 .. 5.1 us;
// 128 requests of up to 17 packed rows, 56 query heads, 22 .. 24 us, 31 MB, and
// 31 with the read of their page tables after them, where the 16-bit append of
// the same rows takes 12.3.  Those took 40 with a wave for a head and all its
// rows, in fp64 also where there are none, and 43 with contiguous runs of tasks
// instead of every y-th.
#include "cache_rows.hpp"

namespace dspark {

namespace {

constexpr int kBlock = 16;  // tokens that share a scale
constexpr int kLow = -117, kHigh = 119;  // exponents of a scale

constexpr float kEnd = 448.f * 0x1p119f;  // what larger numbers are held as

// x cut to fp32, its last bit set if anything was lost; past kEnd that, and
// NaN for what is not finite.
__device__ __forceinline__ float cut_odd(double x) {
  const double y = fmin(fmax(x, -static_cast<double>(kEnd)), static_cast<double>(kEnd));
  const float f = static_cast<float>(y);  // to nearest: at most one step beyond y
  const double z = static_cast<double>(f);
  uint32_t b = __float_as_uint(f) - (fabs(z) > fabs(y) ? 1u : 0u);
  b |= z != y ? 1u : 0u;
  return fabs(x) <= 1.7976931348623157e308 ? __uint_as_float(b) : __builtin_nanf("");
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

// The smallest exponent e with x <= 448 2^e = 1.75 2^(e + 8), within the limits; x >= 0.
__device__ __forceinline__ int exponent_for(float x) {
  const uint32_t b = __float_as_uint(x);
  return min(kHigh, max(kLow, static_cast<int>(b >> 23) - 127 - ((b & 0x7FFFFFu) <= 0x600000u ? 8 : 7)));
}
__device__ __forceinline__ int exponent_of(uint8_t byte) { return min(kHigh, max(kLow, static_cast<int>(byte) - 127)); }

// The largest of a wave's values, in every lane.
__device__ __forceinline__ float largest(float x) {
  x = over_lanes<32>(x, [](float p, float q) { return fmaxf(p, q); });
  return fmaxf(x, xor32(x));
}

// The grid's x are a request's blocks, its y take a block's tasks in turn:
// keys, values, queries.
template <int D>
__global__ __launch_bounds__(2 * D) void cache_append8_kernel(AppendArgs a) {
  typedef PageLayout<DSPARK_CACHE_FP8, D> PL;
  constexpr int T = 2 * D, L = D / 8;
  static_assert(T / L == kBlock, "a token or a head for every L threads");
  __shared__ double cs64[kBlock * D];  // cosines and sines of the new rows: for keys,
  __shared__ float cs[kBlock * D];     // and for queries
  __shared__ uint32_t tops[3][kBlock];
  const int r = blockIdx.z;
  const int half = a.rot / 2;
  const int slot = threadIdx.x / L, li = threadIdx.x % L;
  // what does not depend on anything, at once
  const int n_rows = rows_of(a.ell[r], a.gamma);
  const int64_t len = a.len[r];
  const int64_t row0 = a.row0 ? static_cast<int64_t>(a.row0[r]) : static_cast<int64_t>(r) * (a.gamma + 1);
  const int part = small_quotient(threadIdx.x, a.per_half), pair = threadIdx.x - part * half;
  const double freq = half ? a.freq[pair] : 0.0;
  u32x4 w_q{0u, 0u, 0u, 0u}, w_k{0u, 0u, 0u, 0u};
  if (a.wq) w_q = *reinterpret_cast<const u32x4*>(a.wq + li * 8);
  if (a.wk) w_k = *reinterpret_cast<const u32x4*>(a.wk + li * 8);
  if (len < 0) return;
  // tokens first .. first + n - 1 of the block are new, those before committed
  const int64_t base = (len / kBlock + blockIdx.x) * kBlock;
  const int64_t t0 = base > len ? base : len;
  const int64_t t1 = base + kBlock < len + n_rows ? base + kBlock : len + n_rows;
  if (t0 >= t1) return;
  const int first = static_cast<int>(t0 - base), n = static_cast<int>(t1 - t0);
  const int64_t row = row0 + (t0 - len);
  const float per_n = 1.f / n;
  const int h0 = first >> 3, both = (first + n - 1) >> 3 != h0;  // the block's halves that the rows touch
  const int heads_k = small_quotient(kBlock, per_n), heads_v = both ? 1 : 2;
  const int end_k = ceil_div(a.Hkv, heads_k), end_v = end_k + ceil_div(a.Hkv, heads_v);
  const int nq = n * a.Hq, tasks = end_v + ceil_div(nq, kBlock);
  const int step = gridDim.y;
  int task = blockIdx.y;
  if (task >= tasks) return;
  const int64_t place = base >> a.page_shift;
  const int id = place < a.max_pages ? page_or_none(a.table[static_cast<int64_t>(r) * a.max_pages + place], a.n_pages)
                                     : -1;
  char* const page = id >= 0 ? a.pool + id * a.page_bytes : nullptr;
  const int t = static_cast<int>(base & (a.P - 1));

  // this slot's (head, row) of a task of keys
  const int hk = small_quotient(slot, per_n), jk = slot - hk * n;
  auto load_k = [&](int task) {
    const int head = task * heads_k + hk;
    return hk < heads_k && head < a.Hkv
               ? *reinterpret_cast<const u32x4*>(a.k + (row + jk) * a.ldk + static_cast<int64_t>(head) * D + li * 8)
               : u32x4{0u, 0u, 0u, 0u};
  };
  auto load_q = [&](int task) {
    const int u = (task - end_v) * kBlock + slot, i = small_quotient(u, a.per_q);
    return u >= 0 && u < nq ? *reinterpret_cast<const u32x4*>(a.q + (row + i) * a.ldq + (u - i * a.Hq) * D + li * 8)
                            : u32x4{0u, 0u, 0u, 0u};
  };
  const bool keys = task < end_k;
  u32x4 raw = keys ? load_k(task) : load_q(task);

  // sines and cosines of the block's new rows, a run of rows of a pair a
  // thread: in fp32 for queries; for keys in fp64, the run's first and the
  // step from row to row, which takes a product where another sine would be
  if (threadIdx.x < 3 * kBlock) tops[0][threadIdx.x] = 0;
  if (half) {
    const int across = T / half;
    auto turns_of = [&](int i) {
      const double turns = static_cast<double>(t0 + i) * freq * 0.15915494309189535;
      return turns - rint(turns);
    };
    if (keys) {
      const int each = ceil_div(n, across), from = part * each, to = part < across ? min(from + each, n) : 0;
      if (from < to) {
        const double turn1 = freq * 0.15915494309189535;
        double c0 = 1, s0 = 0, c1 = 1, s1 = 0;
#pragma unroll 1
        for (int k = 0; k < (each > 1 ? 2 : 1); ++k) {
          c1 = c0, s1 = s0;
          sincospi(2.0 * (k == 0 && each > 1 ? turn1 - rint(turn1) : turns_of(from)), &s0, &c0);
        }
#pragma unroll 1
        for (int i = from; i < to; ++i) {
          cs64[i * D + 2 * pair] = c0;
          cs64[i * D + 2 * pair + 1] = s0;
          const double c = c0 * c1 - s0 * s1;
          s0 = s0 * c1 + c0 * s1;
          c0 = c;
        }
      }
    }
    {
#pragma unroll 1
      for (int i = part; i < n && part < across; i += across) {
        float s, c;
        sincospif(2.f * static_cast<float>(turns_of(i)), &s, &c);
        cs[i * D + 2 * pair] = c;
        cs[i * D + 2 * pair + 1] = s;
      }
    }
  }
  __syncthreads();

  // The exponent of a block's scale, from one thread's contribution of each
  // slot or wave; the barrier also stands between the loads of the old byte and
  // its new value.  Of three sets of maxima one is in use, one may still be
  // read from the task before, and one is cleared for the next.
  int turn = 0;
  auto exponent_of_block = [&](float top, bool mine, int which, int before) {
    if (mine) atomicMax(&tops[turn][which], __float_as_uint(top));
    const int next = turn == 2 ? 0 : turn + 1;
    if (threadIdx.x < kBlock) tops[next][threadIdx.x] = 0;
    __syncthreads();
    top = __uint_as_float(tops[turn][which]);
    turn = next;
    return max(before, exponent_for(top));
  };

#pragma unroll 1
  for (; task < end_k; task += step) {
    const u32x4 now = raw;
    raw = task + step < end_k ? load_k(task + step) : load_q(task + step);
    if (!page) continue;
    const int head = task * heads_k + hk;
    const bool live = hk < heads_k && head < a.Hkv;
    char* hp = page + min(head, a.Hkv - 1) * PL::head_bytes(a.P);
    uint8_t* byte = reinterpret_cast<uint8_t*>(hp + PL::k_scale(a.P, t));
    const int before = first > 0 ? exponent_of(*byte) : kLow;
    float f[8], x[8], top = 0.f;
    unpack(now, f);
    double y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = f[e];
    norm_rotate<double, D>(y, li, a.wk != nullptr, w_k, a.eps, a.rot, a.adjacent != 0, cs64 + jk * D);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = cut_odd(y[e]);
      top = fmaxf(top, fabsf(x[e]));  // (not a NaN)
    }
    top = over_lanes<L>(top, [](float p, float q) { return fmaxf(p, q); });
    const int e2 = exponent_of_block(top, live && li == 0, min(hk, kBlock - 1), before);
    if (live) {
      const float g = ldexpf(1.f, -e2);
      const int64_t at = (li & 1) * 8;
      *reinterpret_cast<u32x2*>(hp + PL::k(a.P, t + first + jk, li / 2) + at) =
          u32x2{codes_of(x[0] * g, x[1] * g, x[2] * g, x[3] * g), codes_of(x[4] * g, x[5] * g, x[6] * g, x[7] * g)};
      if (e2 > before) {  // the head's slots share its committed tokens
        const float again = ldexpf(1.f, before - e2);
        for (int j = jk; j < first; j += n) {
          u32x2* p = reinterpret_cast<u32x2*>(hp + PL::k(a.P, t + j, li / 2) + at);
          const u32x2 was = *p;
          *p = u32x2{rescale(was[0], again), rescale(was[1], again)};
        }
      }
      if (jk == 0 && li == 0) *byte = static_cast<uint8_t>(e2 + 127);
    }
  }

#pragma unroll 1
  for (; task < end_v; task += step) {
    if (task + step >= end_v) raw = load_q(task + step);
    if (!page) continue;
    const int g = threadIdx.x / D, d = threadIdx.x % D;
    const int head = (task - end_k) * heads_v + (both ? 0 : g), h = both ? g : h0;
    const bool live = head < a.Hkv;
    // this thread's tokens are 8 h .. of the block: lo of them committed, up to hi new
    const int lo = max(first - 8 * h, 0), hi = min(first + n - 8 * h, 8);
    char* hp = page + min(head, a.Hkv - 1) * PL::head_bytes(a.P);
    uint8_t* byte = reinterpret_cast<uint8_t*>(hp + PL::v_scale(a.P, t));
    u32x2* p = reinterpret_cast<u32x2*>(hp + PL::v(a.P, t + 8 * h, d));
    const int before = first > 0 ? exponent_of(*byte) : kLow;
    const u32x2 was = *p;
    const uint16_t* src = a.v + (row + 8 * h - first) * a.ldv + static_cast<int64_t>(min(head, a.Hkv - 1)) * D + d;
    uint16_t raw_v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) raw_v[j] = src[min(max(j, lo), hi - 1) * a.ldv];  // (all at once: no branches)
    float x[8], top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = j >= lo && j < hi ? bf16_to_f32(raw_v[j]) : 0.f;
      x[j] = fabsf(v) <= 3.4028234e38f ? fminf(fmaxf(v, -kEnd), kEnd) : __builtin_nanf("");
      top = fmaxf(top, fabsf(x[j]));  // (not a NaN)
    }
    const int e2 = exponent_of_block(largest(top), live && (threadIdx.x & 63) == 0, both ? 0 : g, before);
    if (live) {
      const float f = ldexpf(1.f, -e2);
      u32x2 w{codes_of(x[0] * f, x[1] * f, x[2] * f, x[3] * f), codes_of(x[4] * f, x[5] * f, x[6] * f, x[7] * f)};
      if (hi - lo < 8) {  // the others' bytes of the word
        const float again = ldexpf(1.f, before - e2);
        u32x2 kept = was;
        if (lo > 0 && e2 > before) kept = u32x2{rescale(was[0], again), rescale(was[1], again)};
        const uint64_t old = (1ull << (8 * lo)) - 1ull, fresh = (hi == 8 ? ~0ull : (1ull << (8 * hi)) - 1ull) & ~old;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t nw = static_cast<uint32_t>(fresh >> (32 * i)), ow = static_cast<uint32_t>(old >> (32 * i));
          w[i] = (w[i] & nw) | (kept[i] & ow) | (was[i] & ~(nw | ow));
        }
      }
      if (h0 == 1 && e2 > before) {  // the first half, all of it committed
        const float again = ldexpf(1.f, before - e2);
        u32x2* q = reinterpret_cast<u32x2*>(hp + PL::v(a.P, t, d));
        const u32x2 then = *q;
        *q = u32x2{rescale(then[0], again), rescale(then[1], again)};
      }
      *p = w;
      if (d == 0 && h == h0) *byte = static_cast<uint8_t>(e2 + 127);
    }
  }

#pragma unroll 1
  for (; task < tasks; task += step) {
    const u32x4 now = raw;
    raw = load_q(task + step);
    const int u = (task - end_v) * kBlock + slot, i = min(small_quotient(u, a.per_q), n - 1);
    float x[8];
    unpack(now, x);
    norm_rotate<float, D>(x, li, a.wq != nullptr, w_q, a.eps, a.rot, a.adjacent != 0, cs + i * D);
    if (u < nq) *reinterpret_cast<u32x4*>(a.q_out + ((row + i) * a.Hq + (u - i * a.Hq)) * D + li * 8) = pack_bf16(x);
  }
}

// Work groups of a compute unit that are asked for.  With their read, 128 x up
// to 17 packed rows take 31.3, 30.6, 30.9 and 30.9 us with 4, 6, 8 and 12, 4 x
// 512 rows 27.8, 28.8, 28.4, 29.8, 32 x 17 rows 17.1, 17.6, 19.7, 20.9.
constexpr int64_t kPerUnit = 6;

template <int D>
hipError_t run(AppendArgs& a, hipStream_t s) {
  a.page_bytes = a.Hkv * PageLayout<DSPARK_CACHE_FP8, D>::head_bytes(a.P);
  a.groups = ceil_div(a.gamma + kBlock, kBlock);  // aligned blocks that gamma + 1 tokens can touch
  const int64_t want = kPerUnit * compute_units() / (static_cast<int64_t>(a.R) * a.groups);
  const int rows = a.gamma + 1 < kBlock ? a.gamma + 1 : kBlock;
  const int most = 2 * a.Hkv + ceil_div(rows * a.Hq, kBlock);
  const int gy = want < 1 ? 1 : want > most ? most : static_cast<int>(want);
  a.page_shift = __builtin_ctz(a.P);
  a.per_q = 1.f / a.Hq;
  a.per_half = a.rot > 0 ? 2.f / a.rot : 0.f;
  cache_append8_kernel<D><<<dim3(a.groups, gy, a.R), 2 * D, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t cache_append8_launch(int D, AppendArgs& a, hipStream_t s) {
  return D == 64 ? run<64>(a, s) : D == 128 ? run<128>(a, s) : run<256>(a, s);
}

}  // namespace dspark
