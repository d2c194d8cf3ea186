// How much attention the tokens of every page get from a round's rows
// (include/dspark_cache.h): sum of exp(score - lse) over the rows and heads,
// per request and page.
//
// One pass over the keys.  The scores are attention's: S^T = K Q^T on the
// matrix cores, a lane's 16 accumulators being 16 tokens' scores of one query
// row.  The log-sum is given, so nothing runs and nothing is joined: a lane
// adds its exponentials, over a page's tiles and the row tiles, and 64 lanes'
// sums meet once per page and head.
//
// A page's sum belongs to one work group, so that no order of atomics is in
// it: chunks (a page, or two of 16 tokens) are numbered over the requests and
// every work group takes a contiguous run of them, with all their heads.  Its
// waves take heads in turn (and rows in blocks of kRows), or chunks where
// heads are few; each leaves its sums in LDS, added up in the waves' order.
//
// Memory bounds it: 128 requests of up to 17 rows x 7 query heads a head over
// ragged contexts up to 8192 take 247 us with 16-bit pages of 8 heads of 128
// dims, 5.3 TB/s of the 1.30 GB of keys (277 in a graph, one after another; 1.44
// GB fetched; vector units busy 28 % of the time, matrix units 15); 32 single
// tokens over 4096 .. 16384 tokens of 8 bits 79 us.  Chunks of missing pages are
// loaded too, not multiplied (32 single tokens over 131072 tokens with 48 of 2048
// pages left 276 us, over those 48 pages alone 38).  A short context is a chain of loads
// (lengths, page ids, query rows, keys) and barriers: one token over 4095 tokens
// 9.1 us.  With work groups of four waves the ragged requests took 292 in a
// graph, the one token 2.1 us more, chunks of 512 rows 366 us instead of 191;
// only a request of 17 rows alone over 131055 tokens was faster, 71 us for 76.
#include "cache_tiles.hpp"

namespace dspark {

namespace {

constexpr int kRowTiles = 2;    // row tiles of a wave: query rows and two tiles of keys fit its registers
constexpr int kRows = kRowTiles * kTile;
constexpr int kRun = 64;        // chunks that a work group takes at a time, a lane each

struct WeighArgs {
  int R, gamma, Hq, Hkv, G, P, n_pages, max_pages;
  const uint16_t* q;
  float scale_log2;         // |scale| log2(e) (1 for a zero scale, with q masked to zero)
  uint32_t q_keep, q_flip;  // q & keep ^ flip: the scale's sign, or zero
  int window, sinks;
  const float* lse;
  const int32_t *row0, *ell, *len, *table;
  const char* pool;
  int64_t page_bytes;
  float keep;
  float* mass;
};

// Waves of a work group, one on a compute unit: as many as its registers hold
// (256 dims: one a SIMD).
constexpr int waves_of(int D) { return D == 256 ? 4 : 8; }

// A request's chunks that any of its rows can see: 0 .. head - 1, then first
// .., count in all; positions fit 32 bits.
struct Span {
  int n;        // rows
  int len;      // the first one's position, at most kFar
  int pages;    // table entries up to the last row's
  int head, first, count;
  int weight;   // units of a chunk
};

__device__ __forceinline__ Span span_of(const WeighArgs& a, int r, int chunk) {
  const int n = rows_of(a.ell[r], a.gamma), len = a.len[r];
  Span s{n, min(len, kFar), 0, 0, 0, 0, 1};
  if (n == 0 || len < 0) {
    s.n = 0;
    return s;
  }
  const int end = min(s.len + n, a.max_pages * a.P);
  s.pages = (end + a.P - 1) / a.P;
  const int chunks = (end + chunk - 1) / chunk;
  s.count = chunks;
  if (a.window > 0) {
    const int low = s.len + 1 - a.window;
    s.first = low > 0 ? min(low / chunk, chunks) : 0;
    s.head = min((min(a.sinks, end) + chunk - 1) / chunk, s.first);
    s.count = s.head + chunks - s.first;
  }
  // what a chunk costs: its keys, and the products of its row tiles
  s.weight = 1 + (n * a.G + kTile - 1) / kTile;
  return s;
}

// TWO: pages of 16 tokens, two a tile.
template <int FMT, int D, bool TWO>
__global__ __launch_bounds__(waves_of(D) * 64) void cache_weigh_kernel(WeighArgs a) {
  typedef PageLayout<FMT, D> L;
  constexpr int W = waves_of(D), T = W * 64, KS = D / 16;
  __shared__ int64_t lds_cum[kCacheMaxR];  // units of requests 0 .. r
  __shared__ int64_t lds_scan[W];
  __shared__ float lds_sum[W][2 * kRun];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int h = lane >> 5, col = lane & 31;
  const int chunk = TWO ? 2 * a.P : a.P;
  const int lp = 31 - __clz(a.P), tiles_per = chunk / kTile;

  // units before every request
  const int per = ceil_div(a.R, T);
  const int r0 = min(a.R, static_cast<int>(threadIdx.x) * per), r1 = min(a.R, r0 + per);
  int64_t sum = 0;
  for (int r = r0; r < r1; ++r) {
    const Span s = span_of(a, r, chunk);
    sum += static_cast<int64_t>(s.count) * s.weight;
    lds_cum[r] = sum;
  }
  const int64_t incl = wave_scan(sum, [](int64_t p, int64_t q) { return p + q; });
  if (lane == 63) lds_scan[wave] = incl;
  __syncthreads();
  int64_t before = incl - sum, N = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < wave) before += lds_scan[w];
    N += lds_scan[w];
  }
  for (int r = r0; r < r1; ++r) lds_cum[r] += before;
  __syncthreads();

  const int64_t share = quotient(N, gridDim.x), rest = N - share * gridDim.x;
  const int wg = blockIdx.x;
  const int64_t u0 = share * wg + (wg < rest ? wg : rest), u1 = u0 + share + (wg < rest ? 1 : 0);
  int lo = 0;
#pragma unroll 1
  for (int64_t u = u0; u < u1;) {
    // the request of unit u: the first whose sum is past it
    int hi = a.R - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (lds_cum[mid] > u) hi = mid;
      else lo = mid + 1;
    }
    const int r = uniform(lo);
    Span b = span_of(a, r, chunk);
    b = Span{uniform(b.n),    uniform(b.len),   uniform(b.pages), uniform(b.head),
             uniform(b.first), uniform(b.count), uniform(b.weight)};
    const int64_t base = r > 0 ? lds_cum[r - 1] : 0, end = lds_cum[r];
    // the chunks whose first unit is in this run
    const int c0 = uniform(static_cast<int>(quotient(u - base + b.weight - 1, b.weight)));
    const int c1 = uniform(u1 < end ? static_cast<int>(quotient(u1 - base + b.weight - 1, b.weight)) : b.count);
    u = end;
    const int rows = b.n * a.G, blocks = ceil_div(rows, kRows), items = a.Hkv * blocks;
    const int64_t first_row = a.row0 ? static_cast<int64_t>(a.row0[r]) : static_cast<int64_t>(r) * (a.gamma + 1);
    const int32_t* table = a.table + static_cast<int64_t>(r) * a.max_pages;
    // waves along the items (heads and row blocks), the others along the chunks
    const int along = items >= W ? W : items >= 4 ? 4 : items >= 2 ? 2 : 1, across = W / along;
    const int wi = wave % along, wc = wave / along;
#pragma unroll 1
    for (int run = c0; run < c1; run += kRun) {
      const int n = min(kRun, c1 - run);
      // this lane's chunk: its first token and its pages
      const int mine = min(run + lane, c1 - 1);
      const int my_tok = (mine < b.head ? mine : mine - b.head + b.first) * chunk;
      const int s0 = my_tok >> lp;
      const int id0 = s0 < a.max_pages ? page_or_none(table[s0], a.n_pages) : -1;
      const int id1 = !TWO ? id0 : s0 + 1 < a.max_pages ? page_or_none(table[s0 + 1], a.n_pages) : -1;
      lds_sum[wave][lane] = 0.f;
      lds_sum[wave][kRun + lane] = 0.f;
#pragma unroll 1
      for (int item = wi; item < items; item += along) {
        const int hk = item / blocks, m0 = (item - hk * blocks) * kRows;
        const int row_tiles = min(kRowTiles, ceil_div(rows - m0, kTile));
        const int pos_a = b.len + m0 / a.G, pos_b = b.len + (min(m0 + kRows, rows) - 1) / a.G;
        const int low_a = a.window > 0 ? pos_a - a.window + 1 : 0, low_b = a.window > 0 ? pos_b - a.window + 1 : 0;
        // chunks that all rows see whole, and those that some row sees
        const unsigned long long clear_v = __ballot(id0 >= 0 && id1 >= 0 && my_tok + chunk - 1 <= pos_a &&
                                                    (my_tok >= low_b || my_tok + chunk <= a.sinks));
        const unsigned long long some_v = __ballot((id0 >= 0 || id1 >= 0) && my_tok <= pos_b &&
                                                   (my_tok + chunk > low_a || my_tok < a.sinks));
        u32x4 q[kRowTiles][KS];
        float minus_lse[kRowTiles];  // in base 2; -inf for a row that is none or sees nothing
        int pos[kRowTiles];
#pragma unroll
        for (int x = 0; x < kRowTiles; ++x) {
          const int row = min(m0 + x * kTile + col, rows - 1);
          const int i = row / a.G, g = row - i * a.G;
          const int64_t at = (first_row + i) * a.Hq + hk * a.G + g;
          const float z = a.lse[at];
          minus_lse[x] = m0 + x * kTile + col < rows && z != neg_inf() ? -z * kLog2e : neg_inf();
          pos[x] = b.len + i;
          if (x < row_tiles)
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              q[x][k] = *reinterpret_cast<const u32x4*>(a.q + at * D + KTile<FMT, D>::q_dim(k, h));
#pragma unroll
              for (int y = 0; y < 4; ++y) q[x][k][y] = (q[x][k][y] & a.q_keep) ^ a.q_flip;
            }
        }
        const char* pool = a.pool + hk * L::head_bytes(a.P);
        auto head_of = [&](int id) { return pool + max(id, 0) * a.page_bytes; };
        const uint32_t k_lane = KTile<FMT, D>::lane_offset(TWO ? col & 15 : col, h);
        const int k_token = (TWO ? 0 : col & 16) + token_of_slot(col & 15);
        // tile k of this wave: chunk wc + k / tiles_per * across of the run
        const int total = (n > wc ? (n - wc + across - 1) / across : 0) * tiles_per;
        auto chunk_at = [&](int k) { return wc + k / tiles_per * across; };
        auto load = [&](KTile<FMT, D>& kt, int k) {
          const int c = chunk_at(k), t = (k % tiles_per) * kTile;
          const int i0 = __builtin_amdgcn_readlane(id0, c);
          const int i1 = TWO ? __builtin_amdgcn_readlane(id1, c) : i0;
          kt.load(head_of(TWO && col >= 16 ? i1 : i0), a.P, TWO ? 0 : t, k_lane, k_token);
        };
        float p0 = 0.f, p1 = 0.f;  // this lane's share of the chunk's pages
        auto weigh = [&](const KTile<FMT, D>& kt, int k) {
          const int c = chunk_at(k);
          if ((some_v >> c) & 1u) {
            f32x16 s[kRowTiles];
#pragma unroll
            for (int x = 0; x < kRowTiles; ++x) s[x] = f32x16{0.f};
#pragma unroll
            for (int d = 0; d < KS; ++d) {
              const u32x4 key = kt.operand(d, h);
#pragma unroll
              for (int x = 0; x < kRowTiles; ++x)
                if (x < row_tiles)
                  s[x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(key), as_bf16(q[x][d]), s[x], 0, 0, 0);
            }
            const bool clear = (clear_v >> c) & 1u;
            const int tok = __builtin_amdgcn_readlane(my_tok, c) + (k % tiles_per) * kTile;
            const bool have0 = __builtin_amdgcn_readlane(id0, c) >= 0, have1 = __builtin_amdgcn_readlane(id1, c) >= 0;
#pragma unroll
            for (int x = 0; x < kRowTiles; ++x)
              if (x < row_tiles) {
                float p[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x][j], a.scale_log2, minus_lse[x]));
                if (!clear) {
                  rare();
                  const int low = a.window > 0 ? pos[x] - a.window + 1 : 0;
#pragma unroll
                  for (int j = 0; j < 16; ++j) {
                    const int t = tok + 16 * (j / 8) + 8 * h + j % 8;
                    const bool see = (j < 8 ? have0 : have1) && t <= pos[x] && (t >= low || t < a.sinks);
                    p[j] = see ? p[j] : 0.f;
                  }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) p0 += p[j], p1 += p[8 + j];
              }
          }
          if ((k + 1) % tiles_per == 0) {  // the chunk's last tile
            if (!TWO) p0 += p1;
            const auto sum = [](float p, float q) { return p + q; };
            const float x0 = wave_scan(p0, sum), x1 = TWO ? wave_scan(p1, sum) : 0.f;
            if (lane == 63) {
              lds_sum[wave][c] += x0;
              if (TWO) lds_sum[wave][kRun + c] += x1;
            }
            p0 = p1 = 0.f;
          }
        };
        KTile<FMT, D> ka, kb;
        if (total > 0) load(ka, 0);
#pragma unroll 1
        for (int k = 0; k < total; k += 2) {
          load(kb, min(k + 1, total - 1));
          weigh(ka, k);
          if (k + 1 < total) {
            load(ka, min(k + 2, total - 1));
            weigh(kb, k + 1);
          }
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < (TWO ? 2 : 1) * n; i += T) {
        const int c = TWO ? i >> 1 : i, odd = TWO ? i & 1 : 0;
        const int x = run + c;
        const int s = (((x < b.head ? x : x - b.head + b.first) * chunk) >> lp) + odd;
        float m = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) m += lds_sum[w][odd * kRun + c];
        if (s < b.pages) {
          float* p = a.mass + static_cast<int64_t>(r) * a.max_pages + s;
          *p = a.keep == 0.f ? m : __builtin_fmaf(a.keep, *p, m);  // (0: whatever was there)
        }
      }
      __syncthreads();
    }
  }

  // entries that no row sees only fade: first those work groups that had no chunks
  if (a.keep != 1.f) {
    const int parts = ceil_div(a.max_pages, T);
    for (int64_t x = gridDim.x - 1 - blockIdx.x; x < static_cast<int64_t>(a.R) * parts; x += gridDim.x) {
      const int r = static_cast<int>(x / parts), s = static_cast<int>(x % parts) * T + threadIdx.x;
      const Span b = span_of(a, r, chunk);
      const int c = (TWO ? s >> 1 : s);
      if (b.n > 0 && s < a.max_pages && (s >= b.pages || (c >= b.head && c < b.first))) {
        float* p = a.mass + static_cast<int64_t>(r) * a.max_pages + s;
        *p = a.keep == 0.f ? 0.f : a.keep * *p;
      }
    }
  }
}

template <int FMT, int D>
hipError_t run_p(WeighArgs& a, hipStream_t s) {
  a.page_bytes = a.Hkv * PageLayout<FMT, D>::head_bytes(a.P);
  const int grid = compute_units();
  if (a.P == 16) cache_weigh_kernel<FMT, D, true><<<grid, waves_of(D) * 64, 0, s>>>(a);
  else cache_weigh_kernel<FMT, D, false><<<grid, waves_of(D) * 64, 0, s>>>(a);
  return hipGetLastError();
}

template <int FMT>
hipError_t run_d(int D, WeighArgs& a, hipStream_t s) {
  return D == 64 ? run_p<FMT, 64>(a, s) : D == 128 ? run_p<FMT, 128>(a, s) : run_p<FMT, 256>(a, s);
}

}  // namespace

hipError_t cache_weigh_launch(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages, int max_pages,
                              const void* q, float scale, int window, int sinks, const float* lse,
                              const int32_t* row0, const int32_t* ell, const int32_t* len, const int32_t* table,
                              const void* pool, float keep, float* mass, hipStream_t s) {
  WeighArgs a{};
  a.R = R, a.gamma = gamma, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv, a.P = P, a.n_pages = n_pages, a.max_pages = max_pages;
  a.q = static_cast<const uint16_t*>(q);
  a.scale_log2 = scale == 0.f ? 1.f : (scale < 0.f ? -scale : scale) * kLog2e;
  a.q_keep = scale == 0.f ? 0u : 0xFFFFFFFFu;
  a.q_flip = scale < 0.f ? 0x80008000u : 0u;
  a.window = window, a.sinks = window > 0 ? sinks : 0;
  a.lse = lse, a.row0 = row0, a.ell = ell, a.len = len, a.table = table;
  a.pool = static_cast<const char*>(pool);
  a.keep = keep, a.mass = mass;
  return fmt == DSPARK_CACHE_BF16  ? run_d<DSPARK_CACHE_BF16>(D, a, s)
         : fmt == DSPARK_CACHE_FP8 ? run_d<DSPARK_CACHE_FP8>(D, a, s)
                                   : run_d<DSPARK_CACHE_FP4>(D, a, s);
}

}  // namespace dspark
