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
// Pages hold both operands in 16-byte pieces, contiguous over the lanes that
// read them, so a tile goes straight into registers where every wave has
// tiles of its own (rows of one row tile; 4 bits), and past the registers into
// a ring in LDS where several waves multiply the same 16-bit tile.
//
// Work is split over tokens as well as rows.  The units (request, row block,
// head, tile) are numbered in that order, and every work group takes a
// contiguous run of them, whatever the requests' lengths, or a whole part of a
// head where heads are few and of one length.  A (request, row block, head)
// that lies in one run is finished there; of one that crosses runs, every part
// leaves (max, sum, unnormalised output) in the workspace, and a second launch
// joins them in order.
//
// What bounds it, with 8 heads of 128 dims: the pages' bytes for 16 bits (128
// requests of up to 17 rows x 7 query heads a head, ragged contexts up to
// 8192: 556 us, 4.7 TB/s; one request x 17 rows over 131072 tokens 123 us, 4.4
// TB/s) and mostly for single tokens of 4 bits (32 requests over 16384 tokens
// 97 us, 3.7 TB/s).  Many rows of 4 bits (the same 128 requests up to 16384
// tokens 505 us) are bound by the order inside a wave: vector instructions
// take 47 % of the issue slots and products 33 % of the matrix units' time,
// and with two waves a SIMD neither hides the other whole.  Heads of 256 dims
// have one wave a SIMD, where nothing but the wave itself does; 65 .. 96 query
// rows are three row tiles, and the fourth wave of the work group idles.
// Short contexts are bound by the two launches and the chain of loads before
// the first tile, 6 of 13 us (one token over 1023).
#include "cache.hpp"

namespace dspark {

namespace {

constexpr int kTile = 32;       // tokens of a tile, and query rows of a wave
constexpr int W = 4;            // waves of a work group
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
  int R, gamma, Hq, Hkv, G, P, n_pages, max_pages;
  int blocks;              // row blocks a request can have
  int slot_tiles;          // row tiles of a workspace slot
  int by_head;             // descriptors per (request, row block, head), not per work group
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

// What is left for the join: a (row block, head) that work group `wg` opened
// and did not close, in `parts` parts of as many work groups.
struct Desc {
  int parts;     // 0: nothing
  int rows, m0;  // the row block
  int head;
  int64_t first_row;  // the request's row 0 in q and out
  int wg;
};

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

// A request's row block: its query rows m0 .. m0 + rows - 1, and the tiles
// any of them can see: tiles 0 .. head - 1, then first .., count in all.
// Tokens past the table's reach do not exist, so positions fit 32 bits.
struct Block {
  int m0, rows;
  int len;               // the first new token, at most kFar
  int head, first, count;
  int shift;             // log2 of the waves along the rows (1, 2, 4)
};
constexpr int kFar = 1 << 29;  // past every table (2^20 pages of 128 tokens)

// Units of a tile by the log2 of the waves along the rows: the time it takes.
// 16-bit tiles come at the pace of memory until four waves share them; 4-bit
// ones at that of the vector units nearly from the start.  Measured with heads
// of 128 dims, as kRestart and kFavour below.
__device__ __forceinline__ int weight_of(int fmt, int shift) {
  return fmt == DSPARK_CACHE_BF16 ? 2 + shift : (shift == 0 ? 2 : shift == 1 ? 4 : 7);
}
constexpr int kMinUnits = 8;  // of a work group: a tile a wave; no less than any weight

__device__ __forceinline__ Block block_of(const AttnArgs& a, int entry, int rows_max) {
  const int r = entry / a.blocks, c = entry % a.blocks;
  const int n = rows_of(a.ell[r], a.gamma);
  const int len = a.len[r];
  Block b{c * rows_max, 0, min(len, kFar), 0, 0, 0, 0};
  b.rows = min(rows_max, n * a.G - b.m0);
  if (b.rows <= 0 || len < 0) {
    b.rows = 0;
    return b;
  }
  const int qt = (b.rows + kTile - 1) / kTile;
  b.shift = qt == 1 ? 0 : 32 - __clz(qt - 1);
  const int cap = a.max_pages * a.P;
  const int end = min(b.len + (b.m0 + b.rows - 1) / a.G + 1, cap);
  const int tiles = (end + kTile - 1) / kTile;
  b.count = tiles;
  if (a.window > 0) {
    const int low = b.len + b.m0 / a.G + 1 - a.window;
    b.first = low > 0 ? low / kTile : 0;
    b.head = min((min(a.sinks, end) + kTile - 1) / kTile, b.first);
    b.count = b.head + max(tiles - b.first, 0);
  }
  if (b.count == 0) {  // nothing to see: one tile, all of it masked, writes the empty result
    b.first = tiles - 1;
    b.count = 1;
  }
  return b;
}

// The same in every lane, so in scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ Block uniform(const Block& b) {
  return Block{uniform(b.m0),   uniform(b.rows),  uniform(b.len),  uniform(b.head),
               uniform(b.first), uniform(b.count), uniform(b.shift)};
}

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

// The operands of one tile, loaded ahead of their use.  K: this lane's row
// (token slot lane % 32 of the tile), the 8 dims of its half at every step.
// V: this lane's dim (lane % 32 of every block of 32), the 8 tokens of its
// half of each 16.  Addresses are a wave's base (the page's part for the head
// and the token in it, in scalar registers) and a lane's constant offset.
template <int FMT, int D>
struct KTile;
template <int FMT, int D>
struct VTile;

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

// Weights as two bf16 numbers each: the upper half of the bits, which is not
// above the weight, and the nearest to what that leaves and 2^-22 of the weight
// on top.  2^-15 of a weight is lost; both are positive where the weight is, so
// that an infinite value times them is infinite, and neither zero nor of the
// other sign.
struct Weights {
  u32x4 upper, rest;
  __device__ __forceinline__ void set(int j, float w0, float w1) {
    constexpr float kMore = 1.f + 0x1p-22f;
    const uint32_t b0 = __float_as_uint(w0), b1 = __float_as_uint(w1);
    upper[j] = __builtin_amdgcn_perm(b1, b0, 0x07060302u);
    rest[j] = bf16_pair(__builtin_fmaf(w0, kMore, -__uint_as_float(b0 & 0xFFFF0000u)),
                        __builtin_fmaf(w1, kMore, -__uint_as_float(b1 & 0xFFFF0000u)));
  }
};

// o += V^T W^T for two blocks of 32 dims, in turn so that no product waits
// for the one before it.
//
// One bf16 number a weight put as much error into the output as the output's
// own rounding: 2.3e-3 of it in all against float64 (up to 2.8e-3 where few
// tokens matter), 1.66e-3 so, as with fp32 weights.  What the second costs:
// 128 requests x up to 17 rows of 16 bits 547 -> 556 us, one request over
// 131055 tokens 119 -> 123, window 51.7 -> 56.8, 4 x 512 rows 111 -> 122, 16 x
// 17 rows with heads of 256 dims 192 -> 224; of 4 bits the 128 requests 424 ->
// 505, single tokens 89 -> 95.  fp16 weights in a unit that follows the row's
// largest took 446 for 4 bits, but lose tokens below 2^-24 of it, and with them
// the dims that nothing larger reaches; to choose by tile would let a row's
// bits depend on the rows beside it.
__device__ __forceinline__ void add_weighted(f32x16& o0, f32x16& o1, u32x4 v0, u32x4 v1, const Weights& w) {
  o0 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(v0), as_bf16(w.upper), o0, 0, 0, 0);
  o1 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(v1), as_bf16(w.upper), o1, 0, 0, 0);
  o0 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(v0), as_bf16(w.rest), o0, 0, 0, 0);
  o1 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16(v1), as_bf16(w.rest), o1, 0, 0, 0);
}

template <int D>
struct VTile<DSPARK_CACHE_BF16, D> {
  u32x4 x[2][D / 32];
  static __device__ __forceinline__ uint32_t lane_offset(int row, int h) { return (h * D + row) * 16; }
  // block s of the tile: 16 tokens from t of the page on
  __device__ __forceinline__ void load(int s, const char* head, int P, int t, uint32_t lane, int) {
    const char* p = head + 2 * P * D + static_cast<int64_t>(t >> 4) * (32 * D);
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
      x[s][b] = *reinterpret_cast<const u32x4*>(p + b * 512 + lane);
      keep_load_order();
    }
  }
  __device__ __forceinline__ u32x4 operand(int s, int b) const { return x[s][b]; }
  __device__ __forceinline__ float weight(int, float p) const { return p; }
  __device__ __forceinline__ void hide(int, bool) {}
};

// 4 bits: a token's scale goes into its weights.
template <int D>
struct VTile<DSPARK_CACHE_FP4, D> {
  static constexpr int E = D / 32;
  uint32_t x[2][E];
  f32x4 sc[2][2];
  static __device__ __forceinline__ uint32_t lane_offset(int row, int h) { return (h * 32 + row) * (4 * E); }
  __device__ __forceinline__ void load(int s, const char* head, int P, int t, uint32_t lane, int h) {
    const char* p = head + P * (D / 2 + E) + static_cast<int64_t>(t >> 4) * (8 * D) + lane;
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
    const f32x4* b = reinterpret_cast<const f32x4*>(head + P * (D + E) + t * 4 + static_cast<uint32_t>(h * 32));
    sc[s][0] = b[0];
    sc[s][1] = b[1];
  }
  __device__ __forceinline__ u32x4 operand(int s, int b) const { return fp4_octet(x[s][b], 1.f); }
  __device__ __forceinline__ float weight(int j, float p) const { return p * sc[j / 8][(j % 8) / 4][j % 4]; }
  // a hidden token's scale may be anything, its weight is zero
  __device__ __forceinline__ void hide(int j, bool see) {
    f32x4& x = sc[j / 8][(j % 8) / 4];
    x[j % 4] = see ? x[j % 4] : 0.f;
  }
};

// Running softmax of a lane's query row (m, what weights are relative to, is
// the row's, l the lane's own tokens') and its part of the output.
template <int D>
struct Acc {
  float m, l;
  f32x16 o[D / 32];
};

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

// What starting another head costs a work group, in units (5 us of them).
constexpr int kRestart = 16;

// Of two work groups on a compute unit the one that came first is served
// first.  Where the vector units set the pace (4-bit heads of 64 and 128 dims)
// it is through with an equal share after 85 % of the other's time, so it gets
// more, in 64ths of an equal share: 545 -> 511 us for 128 requests x up to 17
// rows over ragged contexts up to 16384, 142 -> 135 us for 32 x 17 rows over
// 8192.  At the pace of memory it makes no difference (16-bit pages: within 1
// %), and short runs lose: only from 4 kMinUnits a work group on.
constexpr int kFavour = 7;

// A head in `parts` parts of `tiles` tiles, the last ones perhaps empty; with
// `more` > 0 parts come in pairs, the first of a pair that much longer.
template <bool FAVOURED>
struct Parts {
  int count, tiles, more;
  __device__ __forceinline__ Parts(int count, int weight, int parts, bool paired)
      : count(count), tiles(max((count + parts - 1) / parts, (kMinUnits + weight - 1) / weight)),
        more(FAVOURED && paired ? tiles * kFavour / 64 : 0) {}
  __device__ __forceinline__ int begin(int j) const {
    return static_cast<int>(min(static_cast<int64_t>(j) * tiles + (FAVOURED ? (j & 1) * more : 0),
                                static_cast<int64_t>(count)));
  }
  // those that are not empty
  __device__ __forceinline__ int used() const {
    const int n = (count + tiles - 1) / tiles;
    return FAVOURED && begin(n - 1) == count ? n - 1 : n;
  }
};

// The range of units of work group wg: `first` for each of the first n,
// `share` for the others, of which the first `rest` get one more.
template <bool FAVOURED>
struct Deal {
  int64_t share, rest, first;
  int n;
  __device__ __forceinline__ int64_t begin(int wg) const {
    if (FAVOURED && wg < n) return wg * first;
    const int64_t x = FAVOURED ? wg - n : wg;
    return (FAVOURED ? n * first : 0) + share * x + (x < rest ? x : rest);
  }
  __device__ __forceinline__ int owner(int64_t unit) const {
    if (FAVOURED && unit < n * first) return static_cast<int>(quotient(unit, first));
    const int64_t x = FAVOURED ? unit - n * first : unit, big = rest * (share + 1);
    return static_cast<int>((FAVOURED ? n : 0) + (x < big ? quotient(x, share + 1) : rest + quotient(x - big, share)));
  }
};

// Waves along the tokens by the log2 of those along the rows.  Of 16-bit
// heads of 256 dims no tile fits the registers beside the output, so theirs
// all come through LDS, and the ring there holds two rounds of two.
__device__ __forceinline__ int waves_along(int fmt, int D, int shift) {
  return fmt == DSPARK_CACHE_BF16 && D == 256 ? min(2, W >> shift) : W >> shift;
}

// Moves a wave's 64 x 16 bytes from memory to LDS at byte `to`, lane by lane,
// past the registers.  Counts as an outstanding vector load; the compiler
// does not know of it, so its waits may be longer than they need to be, never
// shorter, and the reader's wait is written out below.  M0, which holds the
// address and which the compiler reserves for itself, is left as it was.
__device__ __forceinline__ void copy_to_lds(const char* from, uint32_t to) {
  uint32_t m0;
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, off\n\ts_mov_b32 m0, %0"
      : "=&s"(m0)
      : "s"(to), "v"(from)
      : "memory");
}

// Outstanding vector loads down to N, LDS reads down to none, then the work
// group's barrier: what every wave waited for is there for all, and what
// every wave read may be overwritten.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Four waves a work group.  256 registers a wave for heads of 64 and 128 dims:
// two work groups share a compute unit, and one's startup and joining hide
// behind the other's tiles (one of eight waves measured 3 to 15 % slower);
// 512 registers and one work group for 256 dims.
// TWO: pages of 16 tokens, two a tile.
template <int FMT, int D, bool TWO>
__global__ __launch_bounds__(W * 64, D == 256 ? 1 : 2) void cache_attention_tiles(AttnArgs a) {
  typedef PageLayout<FMT, D> L;
  constexpr int T = W * 64, NB = D / 32, KS = D / 16;
  // The weights' reference is put 8 (in base 2) beyond the maximum, and moves
  // again once a score passes it: weights are at most 1, so that sums stay as
  // far from overflow as those of a plain softmax, and few tiles rescale.
  constexpr float kSlack = 8.f;
  constexpr bool kShared = FMT == DSPARK_CACHE_BF16;
  // the waves' outputs, on their way to be joined; before that the ring of 16-bit tiles
  __shared__ f32x4 lds_own[W][NB * 4][64];
  __shared__ float2 lds_ml[W][64];
  static_assert((NB * 4) % W == 0, "waves share an output's pieces");
  __shared__ int64_t lds_scan[W];
  __shared__ int64_t lds_base, lds_run[2];
  __shared__ int2 lds_heads[W];
  __shared__ int lds_entry;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, col = lane & 31;
  constexpr int rows_max = W * kTile;
  const int wg = blockIdx.x;

  // Entries are (request, row block).  Up to one a thread they are dealt as
  // they are numbered; of more, only those that have rows: a block may be
  // declared for far more rows than most requests bring, and slots be idle.
  // 255 single tokens beside a chunk of 512 rows (8 query heads a head) take
  // 79 us so and 122 with every declared block gone through, 3 requests in
  // 4096 slots 121 and 884.
  int entries = a.R * a.blocks;
  const bool sparse = entries > T;
  int* const lds_live = reinterpret_cast<int*>(&lds_own[0][0][0]);  // row blocks of requests 0 .. r
  static_assert(sizeof(lds_own) >= kCacheMaxR * sizeof(int), "a count a request");
  if (sparse) {
    const int each = ceil_div(a.R, T);
    const int r0 = min(a.R, static_cast<int>(threadIdx.x) * each), r1 = min(a.R, r0 + each);
    int n = 0;
    for (int r = r0; r < r1; ++r) {
      n += a.len[r] < 0 ? 0 : ceil_div(rows_of(a.ell[r], a.gamma) * a.G, rows_max);
      lds_live[r] = n;
    }
    const int incl = wave_scan(n, [](int p, int q) { return p + q; });
    if (lane == 63) lds_heads[wave].x = incl;
    __syncthreads();
    int before = incl - n;
    entries = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int x = lds_heads[w].x;
      if (w < wave) before += x;
      entries += x;
    }
    for (int r = r0; r < r1; ++r) lds_live[r] += before;
    __syncthreads();
  }
  // the i-th entry that has rows, of request r or a later one
  auto entry_at = [&](int i, int& r) {
    if (!sparse) return i;
    int hi = lds_live[r] > i ? r : r + 1 < a.R && lds_live[r + 1] > i ? r + 1 : a.R - 1;
    if (r + 1 < hi) r += 2;
    while (r < hi) {
      const int mid = (r + hi) >> 1;
      if (lds_live[mid] > i) hi = mid;
      else r = mid + 1;
    }
    return r * a.blocks + i - (r > 0 ? lds_live[r - 1] : 0);
  };

  // Units before every entry: runs of entries per thread and a scan, with the
  // heads (an entry has a.Hkv) and the longest head beside it.  Then the
  // deal: equal runs of units whatever their owners, or, if the heads are few
  // and of one length, whole parts of heads, which a work group starts and
  // ends once.  A further pass looks up where this work group's run begins.
  const int per = ceil_div(entries, T);
  const int e0 = min(entries, static_cast<int>(threadIdx.x) * per), e1 = min(entries, e0 + per);
  if (threadIdx.x == 0) lds_run[0] = lds_run[1] = 0;
  constexpr bool kFavoured = FMT == DSPARK_CACHE_FP4 && D != 256;
  Deal<kFavoured> deal{0, 0, 0, 0};
  int64_t at = 0, u0 = 0;
  int nb = 0, parts = 0;  // parts of a head; 0: equal runs
  int heads_at = 0, my_head = 0, my_part = 0;
  int place_of = wg;  // its slots in the workspace: in the order of a head's parts
  bool paired = false;
  auto place = [&](int e, int64_t units_at, int first_head, int count, int weight) {
    const int64_t per_head = static_cast<int64_t>(count) * weight;
    if (parts > 0) {
      const int x = my_head - first_head;
      if (count == 0 || x < 0 || x >= a.Hkv) return;
      const Parts<kFavoured> split(count, weight, parts, paired);
      lds_entry = e;
      lds_base = units_at;
      lds_run[0] = units_at + x * per_head + static_cast<int64_t>(split.begin(my_part)) * weight;
      lds_run[1] = units_at + x * per_head + static_cast<int64_t>(split.begin(my_part + 1)) * weight;
    } else if (u0 >= units_at && u0 < units_at + per_head * a.Hkv) {
      lds_entry = e;
      lds_base = units_at;
      lds_run[0] = u0;
      lds_run[1] = wg < nb ? deal.begin(wg + 1) : u0;
    }
  };
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1 && per == 1) break;
    int64_t sum = 0;
    int heads = 0, longest = 0, count = 0, weight = 1, e = 0, r = 0;
#pragma unroll 1
    for (int i = e0; i < e1; ++i) {
      e = entry_at(i, r);
      const Block b = block_of(a, e, rows_max);
      count = b.count;
      weight = weight_of(FMT, b.shift);
      if (pass == 1) place(e, at + sum, heads_at + heads, count, weight);
      else if (count == 0 && a.by_head && wg == 0)  // nobody opens these
        for (int x = 0; x < a.Hkv; ++x) reinterpret_cast<Desc*>(a.desc)[e * a.Hkv + x].parts = 0;
      sum += static_cast<int64_t>(count) * weight * a.Hkv;
      heads += count > 0 ? a.Hkv : 0;
      longest = max(longest, count * weight);
    }
    if (pass == 0) {
      const int64_t incl = wave_scan(sum, [](int64_t p, int64_t q) { return p + q; });
      const int heads_incl = wave_scan(heads, [](int p, int q) { return p + q; });
      longest = wave_scan(longest, [](int p, int q) { return max(p, q); });
      if (lane == 63) {
        lds_scan[wave] = incl;
        lds_heads[wave] = make_int2(heads_incl, longest);
      }
      __syncthreads();
      int64_t before = 0, N = 0;
      int heads_before = 0, H = 0;
      longest = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const int64_t s = lds_scan[w];
        const int2 n = lds_heads[w];
        if (w < wave) before += s, heads_before += n.x;
        N += s;
        H += n.x;
        longest = max(longest, n.y);
      }
      at = before + incl - sum;
      heads_at = heads_before + heads_incl - heads;
      const int64_t useful = N / kMinUnits;
      nb = useful < 1 ? 1 : useful < gridDim.x ? static_cast<int>(useful) : static_cast<int>(gridDim.x);
      const int64_t equal = quotient(N, nb);
      deal.share = equal;
      deal.rest = N - equal * nb;
      if (kFavoured && nb == static_cast<int>(gridDim.x) && equal >= 4 * kMinUnits) {
        deal.n = nb / 2;
        deal.first = equal + equal * kFavour / 64;
        const int64_t others = N - deal.n * deal.first;
        deal.share = quotient(others, nb - deal.n);
        deal.rest = others - deal.share * (nb - deal.n);
      }
      u0 = deal.begin(wg);
      if (H > 0 && H <= static_cast<int>(gridDim.x)) {
        const int p = min(static_cast<int>(gridDim.x / H), ceil_div(longest, kMinUnits));
        if (longest / p <= equal + kRestart) {
          const int half = gridDim.x / 2;
          parts = p;
          paired = kFavoured && (p & 1) == 0 && H * p > half && longest / p >= 4 * kMinUnits;
          if (paired) place_of = wg < half ? 2 * wg : 2 * (wg - half) + 1;
          my_head = place_of / p;
          my_part = place_of - my_head * p;
        }
      }
      if (per == 1 && e0 < e1) place(e, at, heads_at, count, weight);
    }
  }
  __syncthreads();
  Desc left{};
  u0 = lds_run[0];
  const int64_t u1 = lds_run[1];
  int entry = u0 < u1 ? __builtin_amdgcn_readfirstlane(lds_entry) : 0;
  int64_t base = u0 < u1 ? lds_base : 0;

#pragma unroll 1
  for (int64_t u = u0; u < u1;) {
    const int r = entry / a.blocks;
    const Block b = uniform(block_of(a, entry, rows_max));
    const int weight = weight_of(FMT, b.shift);
    const int64_t per_head = static_cast<int64_t>(b.count) * weight;
    if (u >= base + per_head * a.Hkv) {
      base += per_head * a.Hkv;
      ++entry;
      if (b.rows == 0) {  // past a request's rows: the next that has some, 64 at a time
        rare();
        int x = r + 1;
        uint64_t live = 0;
        for (; x < a.R && !live; x += 64) {
          const int y = min(x + lane, a.R - 1);
          live = __ballot(x + lane < a.R && a.ell[y] >= 0 && a.len[y] >= 0);
        }
        if (!live) break;
        entry = uniform(x - 64 + __builtin_ctzll(live)) * a.blocks;
      }
      continue;
    }
    const int hk = uniform(static_cast<int>(quotient(u - base, per_head)));
    const int64_t seg = base + hk * per_head, seg_end = seg + per_head;
    // the tiles whose first unit is in this run
    const int t0 = uniform(static_cast<uint32_t>(u - seg + weight - 1) / weight);
    const int t1 = uniform(u1 < seg_end ? static_cast<uint32_t>(u1 - seg + weight - 1) / weight : b.count);
    u = seg_end;
    if (t0 >= t1) continue;
    const int qt = ceil_div(b.rows, kTile);
    const int WT = waves_along(FMT, D, b.shift);
    const int wt = uniform(wave / qt), wq = wave - wt * qt;
    const bool active = wt < WT;

    // this lane's query row
    const int row = min(wq * kTile + col, b.rows - 1);
    const int i = (b.m0 + row) / a.G, g = (b.m0 + row) - i * a.G;
    const int64_t first_row = a.row0 ? static_cast<int64_t>(a.row0[r]) : static_cast<int64_t>(r) * (a.gamma + 1);
    const int64_t out_at = (first_row + i) * a.Hq + hk * a.G + g;
    const int pos = b.len + i;
    const int low = a.window > 0 ? pos - a.window + 1 : 0;  // window < 2^31 and pos < 2^30: no overflow
    // the wave's first and last rows
    const int pos_a = b.len + (b.m0 + min(wq * kTile, b.rows - 1)) / a.G;
    const int pos_b = b.len + (b.m0 + min(wq * kTile + kTile, b.rows) - 1) / a.G;
    const int low_a = a.window > 0 ? pos_a - a.window + 1 : 0;
    const int low_b = a.window > 0 ? pos_b - a.window + 1 : 0;

    Acc<D> acc;
    acc.m = neg_inf();
    acc.l = 0.f;
    float minus_ref = 0.f;  // -m, or 0 while nothing was seen
#pragma unroll
    for (int x = 0; x < NB; ++x) acc.o[x] = f32x16{0.f};

    const int tiles = t1 - t0;
    const char* pool = a.pool + hk * L::head_bytes(a.P);
    const int32_t* table = a.table + static_cast<int64_t>(r) * a.max_pages;
    const int lp = TWO ? 4 : 31 - __clz(a.P);
    // tile t of the run: its first token
    auto token_at = [&](int t) {
      const int x = t0 + t;
      return (x < b.head ? x : x - b.head + b.first) * kTile;
    };
    // page ids of tiles t, t + WT, .. for 64 of them, a tile a lane (two pages
    // a tile when P is 16): -1 where the table has none
    struct Ids {
      int v0, v1;
    };
    auto fetch_ids = [&](int t) {
      const int tok = token_at(min(t + lane * WT, tiles - 1));
      const int s0 = tok >> lp, s1 = (tok + 16) >> lp;
      Ids x;
      x.v0 = s0 < a.max_pages ? page_or_none(table[s0], a.n_pages) : -1;
      x.v1 = !TWO ? x.v0 : s1 < a.max_pages ? page_or_none(table[s1], a.n_pages) : -1;
      return x;
    };
    // which of those tiles need no mask
    auto clear_of = [&](const Ids& x, int t) {
      const int tok = token_at(min(t + lane * WT, tiles - 1));
      return __ballot(x.v0 >= 0 && x.v1 >= 0 && tok + kTile - 1 <= pos_a && (tok >= low_b || tok + kTile <= a.sinks));
    };
    // the part for this head of a page; a missing page is read as page 0 and masked
    auto head_of = [&](int id) { return pool + max(id, 0) * a.page_bytes; };
    // a lane's offsets from its wave's bases; with two pages a tile the key
    // rows of the upper 16 tokens lie in the other one
    const uint32_t k_lane = KTile<FMT, D>::lane_offset(TWO ? col & 15 : col, h);
    const uint32_t v_lane = VTile<FMT, D>::lane_offset(col, h);

    // the query rows' operands
    u32x4 q[KS];
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      q[x] = *reinterpret_cast<const u32x4*>(a.q + out_at * D + KTile<FMT, D>::q_dim(x, h));
#pragma unroll
      for (int y = 0; y < 4; ++y) q[x][y] = (q[x][y] & a.q_keep) ^ a.q_flip;
    }

    // One tile: its scores s, its values, first token ct and pages c0, c1;
    // ahead(): what may run beside the exponentials.
    auto absorb = [&](f32x16 s, VTile<FMT, D>& vt, int ct, int c0, int c1, bool clear, auto ahead) {
      if (!clear) {
        rare();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int t = ct + 16 * (j / 8) + 8 * h + j % 8;
          const bool see = (j < 8 ? c0 : c1) >= 0 && t <= pos && (t >= low || t < a.sinks);
          s[j] = see ? s[j] : neg_inf();
          vt.hide(j, see);
        }
      }
      float top = s[0];
#pragma unroll
      for (int j = 1; j < 16; ++j) top = fmaxf(top, s[j]);
      top = fmaxf(top, xor32(top)) * a.scale_log2;
      if (__any(top > acc.m)) {
        const float m = top > acc.m ? top + kSlack : acc.m;
        const float keep = m == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(acc.m - m);
        acc.l *= keep;
        acc.m = m;
        minus_ref = m == neg_inf() ? 0.f : -m;
#pragma unroll
        for (int x = 0; x < NB; ++x)
#pragma unroll
          for (int j = 0; j < 16; ++j) acc.o[x][j] *= keep;
      }
      ahead();
      float p[16], sum = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j], a.scale_log2, minus_ref));
        sum += p[j];
      }
      acc.l += sum;
      bool odd = false;
      if constexpr (FMT == DSPARK_CACHE_BF16) {
        if (!clear) {
          // tokens that no row of the wave sees become zeros; of the others, values that are not finite too
          rare();
#pragma unroll
          for (int s2 = 0; s2 < 2; ++s2) {
            u32x4 keep{0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int t = ct + 16 * s2 + 8 * h + e;
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
      for (int s2 = 0; s2 < 2; ++s2) {
        Weights w;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const int t = 8 * s2 + j;
          w.set(j / 2, vt.weight(t, p[t]), vt.weight(t + 1, p[t + 1]));
        }
#pragma unroll
        for (int x = 0; x < NB; x += 2)
          add_weighted(acc.o[x], acc.o[x + 1], vt.operand(s2, x), vt.operand(s2, x + 1), w);
      }
      if constexpr (FMT == DSPARK_CACHE_BF16)
        if (__any(odd)) {
          uint32_t visible = 0;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int t = ct + 16 * (j / 8) + 8 * h + j % 8;
            const bool see = (j < 8 ? c0 : c1) >= 0 && t <= pos && (t >= low || t < a.sinks);
            visible |= static_cast<uint32_t>(see) << j;
          }
          add_non_finite<D>(acc.o, p, visible, head_of(c0), head_of(c1), a.P, ct & (a.P - 1), (ct + 16) & (a.P - 1), lane);
        }
    };

    const bool shared = kShared && (D == 256 || b.shift > 0);
    if constexpr (kShared) if (shared) {
      // Rounds of WT tiles through a ring of W tiles in LDS.  A wave copies
      // its share of every round, whole 1 KB operands in the order the lanes
      // read them, and multiplies its own tile of it.  Copies are issued
      // W / WT - 1 rounds ahead, past the run's end too (its last tile
      // again), so that what is outstanding is known.
      constexpr int F = D / 8;  // operands of a tile: D / 16 of K, as many of V
      static_assert(sizeof(lds_own) == W * F * 1024, "the ring lies under the outputs");
      const uint32_t ring = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
          (__attribute__((address_space(3))) char*)(&lds_own[0][0][0])));
      const int depth = W / WT, lw = __ffs(WT) - 1;
      const int rounds = (tiles + WT - 1) >> lw;
      const int n = F * WT / W;                   // operands a wave copies in a round
      const int mine = wave * n / F, f0 = wave * n - mine * F;
      const bool keys = f0 < KS;                  // all of them K, or all V
      Ids from{-1, -1}, own{-1, -1};
      unsigned long long clear_v = 0;
      auto copy = [&](int round) {
        if ((round & 63) == 0) {
          rare();
          from = fetch_ids((round << lw) + mine);
        }
        const int tok = token_at(min((round << lw) + mine, tiles - 1));
        const char* p0 = head_of(__builtin_amdgcn_readlane(from.v0, round & 63));
        const char* p1 = TWO ? head_of(__builtin_amdgcn_readlane(from.v1, round & 63)) : p0;
        const int t = TWO ? 0 : (tok & (a.P - 1)) >> 4;
        uint32_t to = ring + ((((round & (depth - 1)) << lw) + mine) * F + f0) * 1024;
        if (keys) {
          const char* p = (TWO && col >= 16 ? p1 : p0) + t * (32 * D) + f0 * 512 + k_lane;
#pragma unroll 1
          for (int j = 0; j < n; ++j) copy_to_lds(p + j * 512, to + j * 1024);
        } else {
          const int g = f0 - KS;
          const int64_t v0 = 2 * a.P * D + t * (32 * D) + v_lane;
#pragma unroll 1
          for (int j = g; j < g + n; ++j) {
            const int s2 = j / NB;
            copy_to_lds((TWO && s2 ? p1 : p0 + (TWO ? 0 : s2 * (32 * D))) + v0 + (j - s2 * NB) * 512, to);
            to += 1024;
          }
        }
      };
      for (int round = 0; round < depth - 1; ++round) copy(round);
#pragma unroll 1
      for (int round = 0; round < rounds; ++round) {
        // this round's copies are there: those of the depth - 2 after it may be on their way
        if (depth == 2) wait_and_meet<0>();
        else wait_and_meet<2 * F / W>();
        copy(round + depth - 1);
        if ((round & 63) == 0) {
          rare();
          own = fetch_ids((round << lw) + wt);
          clear_v = clear_of(own, (round << lw) + wt);
        }
        const int t = (round << lw) + wt;
        if (active && t < tiles) {
          const u32x4* tile = reinterpret_cast<const u32x4*>(&lds_own[0][0][0]) +
                              (((round & (depth - 1)) << lw) + wt) * (F * 64) + lane;
          KTile<FMT, D> kt;
          VTile<FMT, D> vt;
#pragma unroll
          for (int u = 0; u < KS; ++u) kt.x[u] = tile[u * 64];
          const f32x16 s = kt.scores(q, h);
#pragma unroll
          for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
            for (int x = 0; x < NB; ++x) vt.x[s2][x] = tile[(KS + s2 * NB + x) * 64];
          const int c0 = __builtin_amdgcn_readlane(own.v0, round & 63);
          const int c1 = TWO ? __builtin_amdgcn_readlane(own.v1, round & 63) : c0;
          absorb(s, vt, token_at(t), c0, c1, (clear_v >> (round & 63)) & 1u, [] {});
        }
      }
      wait_and_meet<0>();
    }
    if constexpr (D != 256 || !kShared) if (!shared && active && wt < tiles) {
      // Every wave for itself, straight into registers, a tile ahead.  4-bit
      // tiles leave room for the next one's scores, whose products then run
      // beside this one's exponentials (128 requests x up to 17 rows over
      // ragged contexts up to 16384: 550 -> 511 us with it; 64 x 17 rows, heads
      // of 256 dims, up to 4096: 363 -> 322).
      constexpr bool kAhead = FMT == DSPARK_CACHE_FP4;
      const int steps = uniform((tiles - wt + WT - 1) >> (__ffs(WT) - 1));
      const int k_token = (TWO ? 0 : col & 16) + token_of_slot(col & 15);
      KTile<FMT, D> kt;
      VTile<FMT, D> vt;
      Ids ids{-1, -1};
      unsigned long long clear_v = 0;
      int id0 = 0, id1 = 0, tok = 0;
      auto fetch = [&](int k) {
        ids = fetch_ids(wt + k * WT);
        clear_v = clear_of(ids, wt + k * WT);
      };
      auto aim = [&](int k) {
        id0 = __builtin_amdgcn_readlane(ids.v0, k & 63);
        id1 = TWO ? __builtin_amdgcn_readlane(ids.v1, k & 63) : id0;
        tok = token_at(wt + k * WT);
      };
      auto load_k = [&]() {
        kt.load(head_of(TWO && col >= 16 ? id1 : id0), TWO ? 16 : a.P, TWO ? 0 : tok & (a.P - 1), k_lane, k_token);
      };
      auto load_v = [&](VTile<FMT, D>& v) {
        const int t = TWO ? 0 : tok & (a.P - 1);
        v.load(0, head_of(id0), TWO ? 16 : a.P, t, v_lane, h);
        v.load(1, head_of(id1), TWO ? 16 : a.P, TWO ? 0 : t + 16, v_lane, h);
      };
      fetch(0);
      aim(0);
      load_k();
      // tile k, or after the last tile that one again (loaded, not used)
      auto next = [&](int k) {
        if ((k & 63) == 0 && k < steps) {
          rare();
          fetch(k);
        }
        aim(min(k, steps - 1));
      };
      if constexpr (!kAhead) {
        load_v(vt);
#pragma unroll 1
        for (int k = 0; k < steps; ++k) {
          const f32x16 s = kt.scores(q, h);
          const int c0 = id0, c1 = id1, ct = tok;
          const bool clear = (clear_v >> (k & 63)) & 1u;
          next(k + 1);
          load_k();
          absorb(s, vt, ct, c0, c1, clear, [] {});
          load_v(vt);
        }
      } else {
        VTile<FMT, D> vu;
        load_v(vt);
        f32x16 s = kt.scores(q, h);
        int c0 = id0, c1 = id1, ct = tok;
        bool clear = clear_v & 1u;
        next(1);
        load_k();
        // tile k with its scores in s, values in `now`; kt has the next one's keys
        auto turn = [&](VTile<FMT, D>& now, VTile<FMT, D>& then, int k) {
          load_v(then);
          f32x16 ahead;
          absorb(s, now, ct, c0, c1, clear, [&] { ahead = kt.scores(q, h); });
          s = ahead;
          c0 = id0, c1 = id1, ct = tok;
          clear = (clear_v >> ((k + 1) & 63)) & 1u;
          next(k + 2);
          load_k();
        };
#pragma unroll 1
        for (int k = 0; k < steps; k += 2) {
          turn(vt, vu, k);
          if (k + 1 < steps) turn(vu, vt, k + 1);
        }
      }
    }

    // Write, or leave a part.  Waves along the tokens are joined first: every
    // wave leaves its output in LDS and takes an equal share of its rows' dims
    // from all of them.  A wave that has its rows for itself writes from its
    // registers (32 x 17 rows x 4 query heads a head, over 4096 tokens 112 us
    // through LDS, 106 so; of 4 bits over 8192 140 and 135).
    const bool opens = t0 == 0, closes = t1 == b.count;
    const bool valid = wq * kTile + col < b.rows;
    const int64_t slot = (static_cast<int64_t>(place_of) * 2 + (opens ? 1 : 0)) * a.slot_tiles + wq;
    const bool whole = opens && closes;
    float m = acc.m, l = 0.f;
    // piece x: dims 32 (x / 4) + 8 (x % 4) + 4 h .. of the lane's row
    auto write = [&](int x, const f32x4& o) {
      if (!whole) {
        if (valid) reinterpret_cast<f32x4*>(a.part)[(slot * (NB * 4) + x) * 64 + lane] = o;
      } else if (valid) {
        const u32x2 w{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
        *reinterpret_cast<u32x2*>(a.out + out_at * D + (x / 4) * 32 + 8 * (x % 4) + 4 * h) = w;
      }
    };
    auto piece = [&](int x, float f) {
      const f32x16& y = acc.o[x / 4];
      const int j = 4 * (x % 4);
      return f32x4{y[j] * f, y[j + 1] * f, y[j + 2] * f, y[j + 3] * f};
    };
    if (WT == 1) {
      if (active) {
        l = acc.l + xor32(acc.l);
        const float f = !whole ? 1.f : l != 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int x = 0; x < NB * 4; ++x) write(x, piece(x, f));
      }
    } else {
      if (active) lds_ml[wave][lane] = make_float2(acc.m, acc.l);
      __syncthreads();
      if (active) {
        float2 ml[W];
#pragma unroll
        for (int k = 0; k < W; ++k) ml[k] = k < WT ? lds_ml[wq + k * qt][lane] : make_float2(neg_inf(), 0.f);
#pragma unroll
        for (int k = 0; k < W; ++k) m = fmaxf(m, ml[k].x);
        const float ref = m == neg_inf() ? 0.f : m;
#pragma unroll
        for (int k = 0; k < W; ++k) l += ml[k].y * __builtin_amdgcn_exp2f(ml[k].x - ref);
        l += xor32(l);
        const float f = __builtin_amdgcn_exp2f(acc.m - ref) * (!whole ? 1.f : l != 0.f ? 1.f / l : 0.f);
#pragma unroll
        for (int x = 0; x < NB * 4; ++x) lds_own[wave][x][lane] = piece(x, f);
      }
      __syncthreads();
      if (active) {
        const int share = NB * 4 >> (__ffs(WT) - 1);
#pragma unroll 2
        for (int x = wt * share; x < (wt + 1) * share; ++x) {
          f32x4 o{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < W; ++k)
            if (k < WT) {
              const f32x4 y = lds_own[wq + k * qt][x][lane];
#pragma unroll
              for (int z = 0; z < 4; ++z) o[z] += y[z];
            }
          write(x, o);
        }
      }
      __syncthreads();  // before the next segment's waves write there
    }
    if (active && wt == 0 && h == 0) {
      if (!whole) a.ml[slot * kTile + col] = make_float2(m, l);
      else if (a.lse && valid) a.lse[out_at] = l != 0.f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : neg_inf();
    }
    if (opens) {  // the work group that holds the last tile's first unit has the last part
      const int n = closes ? 0
                    : parts > 0 ? Parts<kFavoured>(b.count, weight, parts, paired).used()
                                : deal.owner(seg_end - weight) - wg + 1;
      left = Desc{n, b.rows, b.m0, hk, first_row, place_of};
      if (a.by_head && threadIdx.x == 0) reinterpret_cast<Desc*>(a.desc)[entry * a.Hkv + hk] = left;
    }
  }
  if (!a.by_head && threadIdx.x == 0) reinterpret_cast<Desc*>(a.desc)[wg] = left;
}

// Joins the parts of a descriptor in the order of the tokens.  A piece is 4
// output dims of 32 rows per half of a wave, as the parts were stored.
// Few parts (SPLIT 1): a block per row tile, NB pieces a wave, their loads
// together.  Many (SPLIT 4): a block per piece, each wave a quarter of the
// parts, joined in LDS.
template <int D, int SPLIT>
__global__ __launch_bounds__(256) void cache_attention_join(AttnArgs a) {
  constexpr int NB = D / 32, PIECES = SPLIT == 1 ? NB : 1;
  __shared__ f32x4 lds_o[SPLIT == 1 ? 1 : 4][64];
  __shared__ float2 lds_ml[SPLIT == 1 ? 1 : 4][64];
  const int per_desc = a.slot_tiles * (SPLIT == 1 ? 1 : NB * 4);
  const Desc d = reinterpret_cast<const Desc*>(a.desc)[blockIdx.x / per_desc];
  if (d.parts == 0) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int at = blockIdx.x % per_desc;
  const int wq = SPLIT == 1 ? at : at / (NB * 4);
  const int x0 = SPLIT == 1 ? wave * NB : at % (NB * 4);
  const int row = wq * kTile + (lane & 31);
  if (wq * kTile >= d.rows) return;
  const int each = SPLIT == 1 ? d.parts : ceil_div(d.parts, SPLIT);
  const int k_first = SPLIT == 1 ? 0 : wave * each, k_end = min(d.parts, k_first + each);
  float m = neg_inf(), l = 0.f;
  f32x4 o[PIECES];
#pragma unroll
  for (int x = 0; x < PIECES; ++x) o[x] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto add = [&](float2 ml, const f32x4* y) {
    const float top = fmaxf(m, ml.x), ref = top == neg_inf() ? 0.f : top;
    const float sa = __builtin_amdgcn_exp2f(m - ref), sb = __builtin_amdgcn_exp2f(ml.x - ref);
    m = top;
    l = l * sa + ml.y * sb;
#pragma unroll
    for (int x = 0; x < PIECES; ++x)
#pragma unroll
      for (int z = 0; z < 4; ++z) o[x][z] = o[x][z] * sa + y[x][z] * sb;
  };
  // several parts' loads at a time: the loop is a chain of latencies otherwise
  constexpr int kBatch = SPLIT == 1 ? 2 : 4;
#pragma unroll 1
  for (int k0 = k_first; k0 < k_end; k0 += kBatch) {
    float2 ml[kBatch];
    f32x4 y[kBatch][PIECES];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int k = k0 + j;
      ml[j] = make_float2(neg_inf(), 0.f);
#pragma unroll
      for (int x = 0; x < PIECES; ++x) y[j][x] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (k < k_end && row < d.rows) {
        const int64_t slot = (static_cast<int64_t>(d.wg + k) * 2 + (k == 0 ? 1 : 0)) * a.slot_tiles + wq;
        ml[j] = a.ml[slot * kTile + (lane & 31)];
#pragma unroll
        for (int x = 0; x < PIECES; ++x)
          y[j][x] = reinterpret_cast<const f32x4*>(a.part)[slot * (NB * 4 * 64) + (x0 + x) * 64 + lane];
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) add(ml[j], y[j]);
  }
  if constexpr (SPLIT > 1) {
    lds_ml[wave][lane] = make_float2(m, l);
    lds_o[wave][lane] = o[0];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int k = 1; k < SPLIT; ++k) add(lds_ml[k][lane], &lds_o[k][lane]);
  }
  if (row >= d.rows) return;
  const int i = (d.m0 + row) / a.G, g = (d.m0 + row) - i * a.G;
  const int64_t out_at = (d.first_row + i) * a.Hq + d.head * a.G + g;
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int j = 0; j < PIECES; ++j) {
    const int x = x0 + j;
    const u32x2 w{bf16_pair(o[j][0] * inv, o[j][1] * inv), bf16_pair(o[j][2] * inv, o[j][3] * inv)};
    *reinterpret_cast<u32x2*>(a.out + out_at * D + (x / 4) * 32 + 8 * (x % 4) + 4 * (lane >> 5)) = w;
  }
  if (a.lse && x0 == 0 && lane < 32) a.lse[out_at] = l != 0.f ? (m + __builtin_amdgcn_logf(l)) * kLn2 : neg_inf();
}

// Work groups at most: two on each of a gfx950's 256 compute units.
constexpr int kMaxGrid = 512;

int slot_tiles_of(int gamma, int Hq, int Hkv) {
  const int64_t rows = static_cast<int64_t>(gamma + 1) * (Hq / Hkv);
  return rows >= W * kTile ? W : ceil_div(rows, kTile);
}

// Work groups: as many as the device holds at once.
int grid_of(int D) {
  const int per_unit = D == 256 ? 1 : 2;
  const int n = compute_units() * per_unit, most = kMaxGrid / 2 * per_unit;
  return n < most ? n : most;
}

template <int FMT, int D, bool TWO>
hipError_t run(AttnArgs& a, void* ws, hipStream_t s) {
  constexpr int NB = D / 32;
  a.page_bytes = a.Hkv * PageLayout<FMT, D>::head_bytes(a.P);
  a.blocks = ceil_div(static_cast<int64_t>(a.gamma + 1) * a.G, W * kTile);
  a.slot_tiles = slot_tiles_of(a.gamma, a.Hq, a.Hkv);
  const int grid = grid_of(D);
  // few heads and requests: many parts each
  const int64_t heads = static_cast<int64_t>(a.R) * a.blocks * a.Hkv;
  a.by_head = heads * 4 <= grid;
  char* p = static_cast<char*>(ws);
  a.desc = reinterpret_cast<int32_t*>(p);
  a.ml = reinterpret_cast<float2*>(p + kMaxGrid * sizeof(Desc));
  a.part = reinterpret_cast<float*>(p + kMaxGrid * sizeof(Desc) +
                                    static_cast<size_t>(grid) * 2 * a.slot_tiles * kTile * sizeof(float2));
  cache_attention_tiles<FMT, D, TWO><<<grid, W * 64, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.by_head) cache_attention_join<D, 4><<<heads * a.slot_tiles * NB * 4, 256, 0, s>>>(a);
  else cache_attention_join<D, 1><<<grid * a.slot_tiles, 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int FMT, int D>
hipError_t run_p(AttnArgs& a, void* ws, hipStream_t s) {
  return a.P == 16 ? run<FMT, D, true>(a, ws, s) : run<FMT, D, false>(a, ws, s);
}

template <int FMT>
hipError_t run_d(int D, AttnArgs& a, void* ws, hipStream_t s) {
  return D == 64 ? run_p<FMT, 64>(a, ws, s) : D == 128 ? run_p<FMT, 128>(a, ws, s) : run_p<FMT, 256>(a, ws, s);
}

}  // namespace

size_t cache_attention_workspace_bytes(int gamma, int Hq, int Hkv, int D) {
  // sized for the largest grid: the size does not depend on the device
  const size_t grid = D == 256 ? kMaxGrid / 2 : kMaxGrid;
  const size_t rows = grid * 2 * slot_tiles_of(gamma, Hq, Hkv) * kTile;
  return kMaxGrid * sizeof(Desc) + rows * (sizeof(float2) + static_cast<size_t>(D) * sizeof(float));
}

hipError_t cache_attention_launch(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages,
                                  int max_pages, const void* q, float scale, int window, int sinks,
                                  const int32_t* row0, const int32_t* ell, const int32_t* len, const int32_t* table,
                                  const void* pool, void* out, float* lse, void* ws, hipStream_t s) {
  AttnArgs a{};
  a.R = R, a.gamma = gamma, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv, a.P = P, a.n_pages = n_pages, a.max_pages = max_pages;
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
