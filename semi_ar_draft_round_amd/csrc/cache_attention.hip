// Grouped-head attention of a round's rows over the paged cache, with an
// optional sliding window and visible first tokens (include/dspark_cache.h).
//
// A request's (n tokens) x (Hq / Hkv heads of one key/value head) rows form
// the M query rows of that head; a wave takes 32 of them and 32 tokens at a
// time (a tile) through v_mfma_f32_32x32x16_bf16:
//   S^T = K Q^T    K rows are the A operand, so a lane's 16 accumulators are
//                  16 tokens' scores of ONE query row: the running maximum and
//                  sum stay in the lane (one exchange with lane ^ 32);
//   O^T += V^T P^T the scores' registers are the B operand as they stand: K
//                  rows are fed in an order that puts tokens 8h .. 8h + 7 of
//                  each 16 into half h of the wave, which is where the B
//                  operand wants them, and V lies in the pages with a dim's 8
//                  tokens together, which is the A operand.
// Nothing goes through LDS on the way: pages hold both operands in 16-byte
// pieces, contiguous over the lanes that read them.
//
// Work is split over tokens as well as rows.  The units (request, row block,
// head, tile) are numbered in that order, and every work group takes an equal
// contiguous run of them, whatever the requests' lengths.  A (request, row
// block, head) that lies in one run is finished there; of one that crosses
// runs, every part leaves (max, sum, unnormalised output) in the workspace,
// and a second launch joins them in order.
#include "cache.hpp"

namespace dspark {

namespace {

constexpr int kTile = 32;       // tokens of a tile, and query rows of a wave
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
  int R, gamma, Hq, Hkv, P, n_pages, max_pages;
  int blocks;              // row blocks a request can have
  int min_units;           // the least units worth a work group
  int slot_tiles;          // row tiles of a workspace slot
  const uint16_t* q;
  float scale_log2;        // |scale| log2(e) (1 for a zero scale, with q masked to zero)
  uint32_t q_keep, q_flip; // q & keep ^ flip: the scale's sign, or zero
  int window, sinks;
  const int32_t *row0, *ell, *len, *table;
  const char* pool;
  int64_t page_bytes;
  uint16_t* out;
  float* lse;
  // workspace: descriptors, (max, sum) pairs, outputs
  int32_t* desc;
  float2* ml;
  float* part;
};

template <int D>
struct Shape {
  static constexpr int kWaves = D == 256 ? 4 : 8;
  static constexpr int kSteps = D / 16;      // products of a tile's scores
  static constexpr int kBlocks = D / 32;     // 32-dim blocks of the output
};

// What a work group leaves for the join: the part it opened but did not close.
struct Desc {
  int parts;   // 0: nothing
  int r, block, head;
};

__device__ __forceinline__ bf16x8 as_bf16(u32x4 x) {
  union {
    u32x4 u;
    bf16x8 b;
  } c;
  c.u = x;
  return c.b;
}

// The tiles that a block of query tokens [i0, i1] of a request can see: tiles
// 0 .. head - 1, then `first` .. last; count in all.
struct Span {
  int head, first, count;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int64_t len, int i0, int i1) {
  const int64_t cap = static_cast<int64_t>(a.max_pages) * a.P;
  int64_t end = len + i1 + 1;
  if (end > cap) end = cap;
  const int tiles = static_cast<int>((end + kTile - 1) / kTile);
  Span s{0, 0, tiles};
  if (a.window > 0) {
    const int64_t low = len + i0 - a.window + 1;
    const int first = low > 0 ? static_cast<int>(low / kTile) : 0;
    const int64_t sk = a.sinks < end ? a.sinks : end;
    s.head = static_cast<int>((sk + kTile - 1) / kTile);
    if (s.head > first) s.head = first;
    s.first = first;
    s.count = s.head + (tiles > first ? tiles - first : 0);
  }
  if (s.count == 0) {  // nothing to see: one tile, all of it masked, writes the empty result
    s.first = tiles - 1;
    s.count = 1;
  }
  return s;
}

// A request's row block: its query rows m0 .. m0 + rows - 1.
struct Block {
  int n, m0, rows;
  int64_t len;
  Span span;
};
__device__ __forceinline__ Block block_of(const AttnArgs& a, int entry, int rows_max) {
  const int r = entry / a.blocks, c = entry % a.blocks;
  const int G = a.Hq / a.Hkv;
  Block b;
  b.n = rows_of(a.ell[r], a.gamma);
  b.len = a.len[r];
  b.m0 = c * rows_max;
  const int M = b.n * G;
  b.rows = min(rows_max, M - b.m0);
  if (b.rows <= 0 || b.len < 0) {
    b.rows = 0;
    b.span = Span{0, 0, 0};
    return b;
  }
  b.span = span_of(a, b.len, b.m0 / G, (b.m0 + b.rows - 1) / G);
  return b;
}

// The token that K row slot p (0 .. 15) of a 16-token block holds: with this
// order the accumulators of half h are tokens 8 h .. 8 h + 7 in turn.
__device__ __forceinline__ int token_of_slot(int p) { return ((p >> 2) & 1) * 8 + (p >> 3) * 4 + (p & 3); }

// The operands of one tile, loaded ahead of their use.  K: this lane's row
// (token slot lane % 32 of the tile), the 8 dims of its half at every step.
// V: this lane's dim (lane % 32 of every block of 32), the 8 tokens of its
// half of each 16.
template <int FMT, int D>
struct KTile;
template <int FMT, int D>
struct VTile;

template <int D>
struct KTile<DSPARK_CACHE_BF16, D> {
  u32x4 x[D / 16];
  __device__ __forceinline__ void load(const char* head, int P, int t, int h) {
    const char* p = head + PageLayout<DSPARK_CACHE_BF16, D>::k(P, t, h);
#pragma unroll
    for (int u = 0; u < D / 16; ++u) x[u] = *reinterpret_cast<const u32x4*>(p + u * 512);
  }
  static __device__ __forceinline__ int q_dim(int u, int h) { return 16 * u + 8 * h; }
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
  __device__ __forceinline__ void load(const char* head, int P, int t, int h) {
    typedef PageLayout<DSPARK_CACHE_FP4, D> L;
    const char* p = head + L::k(P, t, h);
#pragma unroll
    for (int g = 0; g < D / 64; ++g) x[g] = *reinterpret_cast<const u32x4*>(p + g * 512);
    const char* b = head + L::k_scale(P, t);
    if constexpr (E == 2) {
      sc[0] = *reinterpret_cast<const uint16_t*>(b);
    } else {
#pragma unroll
      for (int i = 0; i < E / 4; ++i) sc[i] = *reinterpret_cast<const uint32_t*>(b + 4 * i);
    }
  }
  static __device__ __forceinline__ int q_dim(int u, int h) { return 32 * (2 * (u / 4) + h) + 8 * (u % 4); }
  __device__ __forceinline__ f32x16 scores(const u32x4 (&q)[D / 16], int h) const {
    f32x16 s = {0.f};
    bool bad = false;
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
      const uint32_t b = (sc[g / 2] >> (16 * (g & 1) + 8 * h)) & 0xFFu;
      bad |= b == 255u;
      const float scale = __uint_as_float(b << 23);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint32_t w = x[g][v];
        const u32x4 k{fp4_pair<0>(w, scale), fp4_pair<1>(w, scale), fp4_pair<2>(w, scale), fp4_pair<3>(w, scale)};
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(k), as_bf16(q[4 * g + v]), s, 0, 0, 0);
      }
    }
    // a NaN scale makes its token's scores NaN: slot r is accumulator j of half h with 8 (j / 4) + 4 h + j % 4 = r
    const unsigned long long rows = __ballot(bad);
    if (rows) {
      const uint32_t r = static_cast<uint32_t>(rows) | static_cast<uint32_t>(rows >> 32);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if ((r >> (8 * (j / 4) + 4 * h + j % 4)) & 1u) s[j] = __builtin_nanf("");
    }
    return s;
  }
};

template <int D>
struct VTile<DSPARK_CACHE_BF16, D> {
  u32x4 x[2][D / 32];
  __device__ __forceinline__ void load(int s, const char* head, int P, int t16, int row, int h) {
    const char* p = head + PageLayout<DSPARK_CACHE_BF16, D>::v(P, t16 + 8 * h, row);
#pragma unroll
    for (int b = 0; b < D / 32; ++b) x[s][b] = *reinterpret_cast<const u32x4*>(p + b * 512);
  }
  __device__ __forceinline__ u32x4 operand(int s, int b) const { return x[s][b]; }
  __device__ __forceinline__ float weight(int, float p) const { return p; }
};

// 4 bits: a token's scale goes into its weights.
template <int D>
struct VTile<DSPARK_CACHE_FP4, D> {
  static constexpr int E = D / 32;
  uint32_t x[2][E];
  f32x4 sc[2][2];
  __device__ __forceinline__ void load(int s, const char* head, int P, int t16, int row, int h) {
    typedef PageLayout<DSPARK_CACHE_FP4, D> L;
    const char* p = head + L::v(P, t16 + 8 * h, row);
    if constexpr (E == 2) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(p);
      x[s][0] = w[0], x[s][1] = w[1];
    } else {
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(p + 16 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[s][4 * i + j] = w[j];
      }
    }
    const f32x4* b = reinterpret_cast<const f32x4*>(head + L::v_scale(P, t16 + 8 * h));
    sc[s][0] = b[0];
    sc[s][1] = b[1];
  }
  __device__ __forceinline__ u32x4 operand(int s, int b) const {
    const uint32_t w = x[s][b];
    return u32x4{fp4_pair<0>(w, 1.f), fp4_pair<1>(w, 1.f), fp4_pair<2>(w, 1.f), fp4_pair<3>(w, 1.f)};
  }
  __device__ __forceinline__ float weight(int j, float p) const { return p * sc[j / 8][(j % 8) / 4][j % 4]; }
};

// Running softmax of a lane's query row (m is the row's, l the lane's own
// tokens') and its part of the output.
template <int D>
struct Acc {
  float m, l;
  f32x16 o[D / 32];
};

template <int D>
__device__ __forceinline__ void join(Acc<D>& a, float m, float l, float* scale_a, float* scale_b) {
  const float top = fmaxf(a.m, m), base = top == neg_inf() ? 0.f : top;
  *scale_a = __builtin_amdgcn_exp2f(a.m - base);
  *scale_b = __builtin_amdgcn_exp2f(m - base);
  a.l = a.l * *scale_a + l * *scale_b;
  a.m = top;
}

// A visible value that is not finite in a tile that some rows see and others
// do not: the products above took it as zero, because zero weights times an
// infinity are NaN; here each row adds what it does see.  Rare and slow.
template <int D>
__device__ __forceinline__ void add_non_finite(f32x16 (&o)[D / 32], const float (&p)[16], uint32_t visible,
                                            const char* head0, const char* head1, int P, int t0, int t1, int lane) {
  typedef PageLayout<DSPARK_CACHE_BF16, D> L;
  const int h = lane >> 5;
  for (int t = 0; t < 32; ++t) {
    float w = 0.f;
    bool see = false;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (16 * (j / 8) + j % 8 == (t & ~8)) {
        w = p[j];
        see = (visible >> j) & 1u;
      }
    // the half that holds token t hands it over
    const int from = (lane & 31) + 32 * ((t >> 3) & 1);
    w = __shfl(w, from);
    see = __shfl(static_cast<int>(see), from) != 0;
    const char* head = t < 16 ? head0 : head1;
    const int tt = (t < 16 ? t0 : t1) + (t & 15);
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int d = b * 32 + 8 * (j / 4) + 4 * h + j % 4;
        const float v = bf16_to_f32(reinterpret_cast<const uint16_t*>(head + L::v(P, tt, d))[tt & 7]);
        if (see && !(fabsf(v) <= 3.4028234e38f)) o[b][j] += w * v;
      }
  }
}

template <int FMT, int D>
__global__ __launch_bounds__(Shape<D>::kWaves * 64) void cache_attention_tiles(AttnArgs a) {
  typedef PageLayout<FMT, D> L;
  constexpr int W = Shape<D>::kWaves, T = W * 64, NB = D / 32, KS = D / 16;
  __shared__ f32x4 lds_o[W / 2][NB * 4][64];
  __shared__ float2 lds_ml[W / 2][64];
  __shared__ int64_t lds_scan[W];
  __shared__ int64_t lds_base;
  __shared__ int lds_entry;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int h = lane >> 5, col = lane & 31;
  const int rows_max = W * kTile;
  const int G = a.Hq / a.Hkv;

  // Units before every entry (request, row block): runs of entries per thread, then a scan.
  const int entries = a.R * a.blocks;
  const int per = ceil_div(entries, T);
  const int e0 = min(entries, static_cast<int>(threadIdx.x) * per), e1 = min(entries, e0 + per);
  int64_t mine = 0;
  for (int e = e0; e < e1; ++e) {
    const Block b = block_of(a, e, rows_max);
    if (b.rows > 0) mine += static_cast<int64_t>(b.span.count) * a.Hkv;
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t t = __shfl_up(incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 63) lds_scan[wave] = incl;
  __syncthreads();
  int64_t before = 0, N = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const int64_t s = lds_scan[w];
    if (w < wave) before += s;
    N += s;
  }
  const int64_t units_wg = N / a.min_units;
  const int nb = units_wg < 1 ? 1 : units_wg < gridDim.x ? static_cast<int>(units_wg) : static_cast<int>(gridDim.x);
  const int wg = blockIdx.x;
  Desc left{0, 0, 0, 0};
  if (wg < nb && N > 0) {
    const int64_t u0 = N * wg / nb, u1 = N * (wg + 1) / nb;
    int64_t at = before + incl - mine;
    if (u0 >= at && u0 < at + mine) {
      int e = e0;
      for (; e < e1; ++e) {
        const Block b = block_of(a, e, rows_max);
        const int64_t n = b.rows > 0 ? static_cast<int64_t>(b.span.count) * a.Hkv : 0;
        if (u0 < at + n) break;
        at += n;
      }
      lds_entry = e;
      lds_base = at;
    }
    __syncthreads();
    int entry = lds_entry;
    int64_t base = lds_base;

    for (int64_t u = u0; u < u1;) {
      const Block b = block_of(a, entry, rows_max);
      const int64_t total = b.rows > 0 ? static_cast<int64_t>(b.span.count) * a.Hkv : 0;
      if (u >= base + total) {
        base += total;
        ++entry;
        continue;
      }
      const int r = entry / a.blocks;
      const int hk = static_cast<int>((u - base) / b.span.count);
      const int64_t seg = base + static_cast<int64_t>(hk) * b.span.count;
      const int t0 = static_cast<int>(u - seg);
      const int t1 = u1 - seg < b.span.count ? static_cast<int>(u1 - seg) : b.span.count;
      const int qt = ceil_div(b.rows, kTile);
      const int WT = qt == 1 ? W : qt == 2 ? W / 2 : qt <= 4 ? W / 4 : 1;  // waves along the tokens
      const int wq = wave % qt, wt = wave / qt;
      const bool active = wt < WT;

      // this lane's query row
      const int row = min(wq * kTile + col, b.rows - 1);
      const int i = (b.m0 + row) / G, g = (b.m0 + row) % G;
      const int64_t first_row =
          a.row0 ? static_cast<int64_t>(a.row0[r]) : static_cast<int64_t>(r) * (a.gamma + 1);
      const int64_t out_at = ((first_row + i) * a.Hq + hk * G + g);
      const int64_t pos = b.len + i;
      const int64_t low = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
      // the wave's first and last rows
      const int row_a = min(wq * kTile, b.rows - 1), row_b = min(wq * kTile + kTile, b.rows) - 1;
      const int64_t pos_a = b.len + (b.m0 + row_a) / G, pos_b = b.len + (b.m0 + row_b) / G;
      const int64_t low_a = a.window > 0 && pos_a - a.window + 1 > 0 ? pos_a - a.window + 1 : 0;
      const int64_t low_b = a.window > 0 && pos_b - a.window + 1 > 0 ? pos_b - a.window + 1 : 0;

      Acc<D> acc;
      acc.m = neg_inf();
      acc.l = 0.f;
#pragma unroll
      for (int x = 0; x < NB; ++x) acc.o[x] = f32x16{0.f};

      const int steps = active && t0 + wt < t1 ? (t1 - t0 - wt + WT - 1) / WT : 0;
      if (steps > 0) {
        u32x4 q[KS];
#pragma unroll
        for (int x = 0; x < KS; ++x) {
          q[x] = *reinterpret_cast<const u32x4*>(a.q + out_at * D + KTile<FMT, D>::q_dim(x, h));
#pragma unroll
          for (int y = 0; y < 4; ++y) q[x][y] = (q[x][y] & a.q_keep) ^ a.q_flip;
        }
        const int64_t head_off = hk * L::head_bytes(a.P);
        const int32_t* table = a.table + static_cast<int64_t>(r) * a.max_pages;
        const int lp = 31 - __clz(a.P);
        // page ids of the wave's next 64 tiles, one tile a lane (two pages a tile when P is 16)
        int id0_v = -1, id1_v = -1;
        auto tile_at = [&](int k) {
          const int t = t0 + wt + k * WT;
          return t < b.span.head ? t : t - b.span.head + b.span.first;
        };
        auto fetch_ids = [&](int k0) {
          const int64_t tok = static_cast<int64_t>(tile_at(k0 + lane)) * kTile;
          const int64_t s0 = tok >> lp, s1 = (tok + 16) >> lp;
          const bool in = k0 + lane < steps;
          id0_v = in && s0 < a.max_pages ? page_or_none(table[s0], a.n_pages) : -1;
          id1_v = in && s1 < a.max_pages ? page_or_none(table[s1], a.n_pages) : -1;
        };
        KTile<FMT, D> kt;
        VTile<FMT, D> vt;
        // pages of the tile in flight; a missing one is read as page 0 and masked
        int id0 = 0, id1 = 0;
        int64_t tok = 0;
        const char *head0 = nullptr, *head1 = nullptr;
        int in0 = 0, in1 = 0;
        auto aim = [&](int k) {
          if ((k & 63) == 0) fetch_ids(k);
          id0 = __builtin_amdgcn_readlane(id0_v, k & 63);
          id1 = __builtin_amdgcn_readlane(id1_v, k & 63);
          tok = static_cast<int64_t>(tile_at(k)) * kTile;
          head0 = a.pool + max(id0, 0) * a.page_bytes + head_off;
          head1 = a.pool + max(id1, 0) * a.page_bytes + head_off;
          in0 = static_cast<int>(tok & (a.P - 1));
          in1 = static_cast<int>((tok + 16) & (a.P - 1));
        };
        auto load_k = [&]() {
          kt.load(col < 16 ? head0 : head1, a.P, (col < 16 ? in0 : in1) + token_of_slot(col & 15), h);
        };
        aim(0);
        load_k();
        vt.load(0, head0, a.P, in0, col, h);
        vt.load(1, head1, a.P, in1, col, h);
        for (int k = 0; k < steps; ++k) {
          f32x16 s = kt.scores(q, h);
          const int c0 = id0, c1 = id1, ci0 = in0, ci1 = in1;
          const int64_t ct = tok;
          const char *ch0 = head0, *ch1 = head1;
          const bool more = k + 1 < steps;
          if (more) {
            aim(k + 1);
            load_k();
          }
          const bool clear = c0 >= 0 && c1 >= 0 && ct + kTile - 1 <= pos_a && (ct >= low_b || ct + kTile <= a.sinks);
          uint32_t visible = 0xFFFFu;
          if (!clear) {
            visible = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int64_t t = ct + 16 * (j / 8) + 8 * h + j % 8;
              const bool see = (j < 8 ? c0 : c1) >= 0 && t <= pos && (t >= low || t < a.sinks);
              s[j] = see ? s[j] : neg_inf();
              visible |= static_cast<uint32_t>(see) << j;
            }
          }
          float top = s[0];
#pragma unroll
          for (int j = 1; j < 16; ++j) top = fmaxf(top, s[j]);
          top = fmaxf(top, xor32(top));
          const float m = fmaxf(acc.m, top * a.scale_log2);
          const float ref = m == neg_inf() ? 0.f : m;
          float p[16], sum = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j], a.scale_log2, -ref));
            sum += p[j];
          }
          if (__any(m != acc.m)) {
            const float keep = __builtin_amdgcn_exp2f(acc.m - ref);
            acc.l *= keep;
            acc.m = m;
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
              for (int j = 0; j < 16; ++j) acc.o[x][j] *= keep;
          }
          acc.l += sum;
          u32x4 pk[2];
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float x = vt.weight(j, p[j]), y = vt.weight(j + 1, p[j + 1]);
            if (FMT == DSPARK_CACHE_FP4 && !clear) {  // a hidden token's scale may be anything
              x = (visible >> j) & 1u ? x : 0.f;
              y = (visible >> (j + 1)) & 1u ? y : 0.f;
            }
            pk[j / 8][(j % 8) / 2] = bf16_pair(x, y);
          }
          bool odd = false;
          if (FMT == DSPARK_CACHE_BF16 && !clear) {
            // tokens that no row of the wave sees become zeros; of the others, values that are not finite too
            if constexpr (FMT == DSPARK_CACHE_BF16) {
#pragma unroll
              for (int s2 = 0; s2 < 2; ++s2) {
                u32x4 keep{0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int64_t t = ct + 16 * s2 + 8 * h + e;
                  const bool see = (s2 ? c1 : c0) >= 0 && t <= pos_b && (t >= low_a || t < a.sinks);
                  keep[e / 2] |= see ? 0xFFFFu << (16 * (e & 1)) : 0u;
                }
#pragma unroll
                for (int x = 0; x < NB; ++x)
#pragma unroll
                  for (int w = 0; w < 4; ++w) {
                    uint32_t v = vt.x[s2][x][w] & keep[w];
                    if ((v & 0x7F80u) == 0x7F80u) odd = true, v &= 0xFFFF0000u;
                    if ((v & 0x7F800000u) == 0x7F800000u) odd = true, v &= 0x0000FFFFu;
                    vt.x[s2][x][w] = v;
                  }
              }
            }
          }
#pragma unroll
          for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
            for (int x = 0; x < NB; ++x)
              acc.o[x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(vt.operand(s2, x)), as_bf16(pk[s2]), acc.o[x],
                                                                 0, 0, 0);
          if constexpr (FMT == DSPARK_CACHE_BF16)
            if (__any(odd)) add_non_finite<D>(acc.o, p, visible, ch0, ch1, a.P, ci0, ci1, lane);
          if (more) {
            vt.load(0, head0, a.P, in0, col, h);
            vt.load(1, head1, a.P, in1, col, h);
          }
        }
      }

      // join the waves along the tokens, halving
      for (int step = WT / 2; step >= 1; step >>= 1) {
        __syncthreads();
        if (active && wt >= step && wt < 2 * step) {
          const int slot = (wt - step) * qt + wq;
          lds_ml[slot][lane] = make_float2(acc.m, acc.l);
#pragma unroll
          for (int x = 0; x < NB; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              lds_o[slot][x * 4 + j][lane] =
                  f32x4{acc.o[x][4 * j], acc.o[x][4 * j + 1], acc.o[x][4 * j + 2], acc.o[x][4 * j + 3]};
        }
        __syncthreads();
        if (active && wt < step) {
          const int slot = wt * qt + wq;
          const float2 ml = lds_ml[slot][lane];
          float sa, sb;
          join<D>(acc, ml.x, ml.y, &sa, &sb);
#pragma unroll
          for (int x = 0; x < NB; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f32x4 y = lds_o[slot][x * 4 + j][lane];
#pragma unroll
              for (int z = 0; z < 4; ++z) acc.o[x][4 * j + z] = acc.o[x][4 * j + z] * sa + y[z] * sb;
            }
        }
      }
      __syncthreads();

      const bool opens = t0 == 0, closes = t1 == b.span.count;
      if (active && wt == 0) {
        const float l = acc.l + xor32(acc.l);
        if (opens && closes) {
          if (wq * kTile + col < b.rows) {
            const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const u32x2 w{bf16_pair(acc.o[x][4 * j] * inv, acc.o[x][4 * j + 1] * inv),
                              bf16_pair(acc.o[x][4 * j + 2] * inv, acc.o[x][4 * j + 3] * inv)};
                *reinterpret_cast<u32x2*>(a.out + out_at * D + x * 32 + 8 * j + 4 * h) = w;
              }
            if (a.lse && h == 0) a.lse[out_at] = l != 0.f ? (acc.m + __builtin_amdgcn_logf(l)) * kLn2 : neg_inf();
          }
        } else {
          const int64_t slot = (static_cast<int64_t>(wg) * 2 + (opens ? 1 : 0)) * a.slot_tiles + wq;
          if (h == 0) a.ml[slot * kTile + col] = make_float2(acc.m, l);
          f32x4* dst = reinterpret_cast<f32x4*>(a.part) + slot * (NB * 4 * 64);
#pragma unroll
          for (int x = 0; x < NB; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              dst[(x * 4 + j) * 64 + lane] =
                  f32x4{acc.o[x][4 * j], acc.o[x][4 * j + 1], acc.o[x][4 * j + 2], acc.o[x][4 * j + 3]};
        }
      }
      if (opens && !closes) {
        const int64_t end = seg + b.span.count;  // the work group that holds unit end - 1 has the last part
        left = Desc{static_cast<int>((end * nb - 1) / N) - wg + 1, r, entry % a.blocks, hk};
      }
      u = seg + t1;
    }
  }
  if (threadIdx.x == 0) reinterpret_cast<Desc*>(a.desc)[wg] = left;
}

// Joins the parts of what work group blockIdx.x opened and did not close, in
// the order of the tokens.  A thread takes four output dims of one row.
template <int FMT, int D>
__global__ __launch_bounds__(256) void cache_attention_join(AttnArgs a) {
  constexpr int W = Shape<D>::kWaves, NB = D / 32;
  const int wg = blockIdx.x;
  const Desc d = reinterpret_cast<const Desc*>(a.desc)[wg];
  if (d.parts == 0) return;
  const Block b = block_of(a, d.r * a.blocks + d.block, W * kTile);
  const int piece = blockIdx.y * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wq = piece / (NB * 4), x = piece % (NB * 4);
  const int row = wq * kTile + (lane & 31);
  if (row >= b.rows) return;
  float m = neg_inf(), l = 0.f;
  f32x4 o{0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < d.parts; ++k) {
    const int64_t slot = (static_cast<int64_t>(wg + k) * 2 + (k == 0 ? 1 : 0)) * a.slot_tiles + wq;
    const float2 ml = a.ml[slot * kTile + (lane & 31)];
    const f32x4 y = reinterpret_cast<const f32x4*>(a.part)[slot * (NB * 4 * 64) + x * 64 + lane];
    const float top = fmaxf(m, ml.x), ref = top == neg_inf() ? 0.f : top;
    const float sa = __builtin_amdgcn_exp2f(m - ref), sb = __builtin_amdgcn_exp2f(ml.x - ref);
    m = top;
    l = l * sa + ml.y * sb;
#pragma unroll
    for (int z = 0; z < 4; ++z) o[z] = o[z] * sa + y[z] * sb;
  }
  const int G = a.Hq / a.Hkv;
  const int i = (b.m0 + row) / G, g = (b.m0 + row) % G;
  const int64_t first_row = a.row0 ? static_cast<int64_t>(a.row0[d.r]) : static_cast<int64_t>(d.r) * (a.gamma + 1);
  const int64_t out_at = (first_row + i) * a.Hq + d.head * G + g;
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const u32x2 w{bf16_pair(o[0] * inv, o[1] * inv), bf16_pair(o[2] * inv, o[3] * inv)};
  *reinterpret_cast<u32x2*>(a.out + out_at * D + (x / 4) * 32 + 8 * (x % 4) + 4 * (lane >> 5)) = w;
  if (a.lse && x == 0 && lane < 32) a.lse[out_at] = l != 0.f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : neg_inf();
}

// Work groups of the first launch: one per compute unit (the registers allow
// no second).
constexpr int kMaxGrid = 512;
int grid_of() {
  const int n = compute_units();
  return n < kMaxGrid ? n : kMaxGrid;
}

int slot_tiles_of(int gamma, int Hq, int Hkv, int D) {
  const int W = D == 256 ? 4 : 8;
  const int64_t rows = static_cast<int64_t>(gamma + 1) * (Hq / Hkv);
  return rows >= W * kTile ? W : ceil_div(rows, kTile);
}

template <int FMT, int D>
hipError_t run(AttnArgs& a, void* ws, hipStream_t s) {
  constexpr int W = Shape<D>::kWaves, NB = D / 32;
  const int G = a.Hq / a.Hkv;
  a.page_bytes = a.Hkv * PageLayout<FMT, D>::head_bytes(a.P);
  a.blocks = ceil_div(static_cast<int64_t>(a.gamma + 1) * G, W * kTile);
  a.slot_tiles = slot_tiles_of(a.gamma, a.Hq, a.Hkv, D);
  a.min_units = W;
  const int grid = grid_of();
  char* p = static_cast<char*>(ws);
  a.desc = reinterpret_cast<int32_t*>(p);
  a.ml = reinterpret_cast<float2*>(p + kMaxGrid * sizeof(Desc));
  a.part = reinterpret_cast<float*>(p + kMaxGrid * sizeof(Desc) +
                                    static_cast<size_t>(kMaxGrid) * 2 * a.slot_tiles * kTile * sizeof(float2));
  cache_attention_tiles<FMT, D><<<grid, W * 64, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  cache_attention_join<FMT, D><<<dim3(grid, a.slot_tiles * NB), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int FMT>
hipError_t run_d(int D, AttnArgs& a, void* ws, hipStream_t s) {
  return D == 64 ? run<FMT, 64>(a, ws, s) : D == 128 ? run<FMT, 128>(a, ws, s) : run<FMT, 256>(a, ws, s);
}

}  // namespace

size_t cache_attention_workspace_bytes(int R, int gamma, int Hq, int Hkv, int D) {
  (void)R;
  const size_t rows = static_cast<size_t>(kMaxGrid) * 2 * slot_tiles_of(gamma, Hq, Hkv, D) * kTile;
  return kMaxGrid * sizeof(Desc) + rows * (sizeof(float2) + static_cast<size_t>(D) * sizeof(float));
}

hipError_t cache_attention_launch(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages,
                                  int max_pages, const void* q, float scale, int window, int sinks,
                                  const int32_t* row0, const int32_t* ell, const int32_t* len, const int32_t* table,
                                  const void* pool, void* out, float* lse, void* ws, hipStream_t s) {
  AttnArgs a{};
  a.R = R, a.gamma = gamma, a.Hq = Hq, a.Hkv = Hkv, a.P = P, a.n_pages = n_pages, a.max_pages = max_pages;
  a.q = static_cast<const uint16_t*>(q);
  a.scale_log2 = scale == 0.f ? 1.f : (scale < 0.f ? -scale : scale) * kLog2e;
  a.q_keep = scale == 0.f ? 0u : 0xFFFFFFFFu;
  a.q_flip = scale < 0.f ? 0x80008000u : 0u;
  a.window = window, a.sinks = window > 0 ? sinks : 0;
  a.row0 = row0, a.ell = ell, a.len = len, a.table = table;
  a.pool = static_cast<const char*>(pool);
  a.out = static_cast<uint16_t*>(out), a.lse = lse;
  return fmt == DSPARK_CACHE_BF16 ? run_d<DSPARK_CACHE_BF16>(D, a, ws, s) : run_d<DSPARK_CACHE_FP4>(D, a, ws, s);
}

}  // namespace dspark
