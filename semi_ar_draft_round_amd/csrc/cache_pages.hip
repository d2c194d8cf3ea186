// Who owns the cache's pages: reserve, commit, evict, fork, compact, copy, reset
// (include/dspark_cache.h).
//
// The free pages are a bitmap, so that which ids come next depends on the set
// of free pages alone and not on the order in which they were released: every
// call gives the same table whatever order its atomics ran in (reference
// counts and bits only ever see commuting adds and ors).  2^20 pages are
// 128 KB of bitmap: one work group counts and searches it in one pass.
#include "cache.hpp"

namespace dspark {

namespace {

constexpr int kT = 1024;  // threads of the single-work-group kernels

// Exclusive prefix sum of one int per thread over the work group; *total gets the sum.
__device__ int block_exclusive_scan(int v, int* lds, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int x = wave_scan(v, [](int p, int q) { return p + q; });
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kT / 64; ++w) {
    const int s = lds[w];
    if (w < wave) before += s;
    sum += s;
  }
  __syncthreads();
  *total = sum;
  return before + x - v;
}

__device__ __forceinline__ void release(int id, int n_pages, int32_t* ref, uint32_t* bits) {
  if (page_or_none(id, n_pages) < 0) return;
  if (atomicSub(&ref[id], 1) == 1) atomicOr(&bits[id >> 5], 1u << (id & 31));
}

constexpr int kEvicted = -2;  // table entry of a page that dspark_cache_evict let go
__device__ __forceinline__ int page_or_mark(int id, int n_pages) {
  return id == kEvicted ? kEvicted : page_or_none(id, n_pages);
}

// Bits of word w that stand for pages below n.
__device__ __forceinline__ uint32_t bits_below(int w, int n) {
  const int k = n - w * 32;
  return k >= 32 ? 0xFFFFFFFFu : k <= 0 ? 0u : (1u << k) - 1u;
}

__global__ void cache_reset_kernel(int64_t n_table, int R, int n_pages, int32_t* table, int32_t* len, int32_t* ref,
                                   uint32_t* bits) {
  const int words = (n_pages + 31) / 32;
  for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < n_table || i < n_pages || i < R; i += gridDim.x * 256LL) {
    if (i < n_table) table[i] = -1;
    if (i < R) len[i] = 0;
    if (i < n_pages) ref[i] = 0;
    if (i < words) bits[i] = bits_below(static_cast<int>(i), n_pages);
  }
}

// What a request asks for: its pages first .. last - 1, the shared page it must leave.
struct Ask {
  int n, first, last;  // rows, page range
  int tail;            // page of token len - 1 if it is to be written too and others hold it, else -1
  int missing;         // entries of the range that are -1
};

__device__ Ask ask_of(int r, int gamma, int P, int n_pages, int max_pages, const int32_t* ell, const int32_t* len,
                      const int32_t* table, const int32_t* ref) {
  Ask a{rows_of(ell[r], gamma), 0, 0, -1, 0};
  const int64_t at = len[r];
  const int64_t last = (at + a.n + P - 1) / P;
  if (a.n == 0 || at < 0 || last > max_pages) {
    a.n = 0;
    return a;
  }
  a.first = static_cast<int>(at / P);
  a.last = static_cast<int>(last);
  const int32_t* row = table + static_cast<int64_t>(r) * max_pages;
  for (int i = a.first; i < a.last; ++i) {
    const int id = page_or_none(row[i], n_pages);
    if (id < 0) ++a.missing;
    else if (i == a.first && at % P != 0 && ref[id] > 1) a.tail = id;
  }
  return a;
}

// One work group.  Requests are dealt to threads in contiguous runs, so one
// scan over the threads' sums orders them; what a request asks for is looked
// up again where it is needed (its few table entries are in cache by then).
__global__ __launch_bounds__(kT) void cache_reserve_kernel(int R, int gamma, int P, int n_pages, int max_pages,
                                                           const int32_t* ell, const int32_t* len, int32_t* table,
                                                           int32_t* ref, uint32_t* bits, int32_t* ell_out,
                                                           int32_t* pairs, int32_t* n_pairs, int32_t* status,
                                                           int32_t* ids) {
  __shared__ int lds[kT / 64];
  __shared__ int s_tail[kCacheMaxR];
  __shared__ int s_alloc, s_refused;
  const int per = ceil_div(R, kT);
  const int r0 = min(R, static_cast<int>(threadIdx.x) * per), r1 = min(R, r0 + per);
  if (threadIdx.x == 0) s_alloc = s_refused = 0;

  Ask a[4];
  bool copy[4], exempt[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (r0 + j < r1) {
      a[j] = ask_of(r0 + j, gamma, P, n_pages, max_pages, ell, len, table, ref);
      s_tail[r0 + j] = a[j].tail;
    }
  // free pages per thread: contiguous words
  const int words = (n_pages + 31) / 32;
  const int wper = ceil_div(words, kT);
  const int w0 = min(words, static_cast<int>(threadIdx.x) * wper), w1 = min(words, w0 + wper);
  int mine = 0;
  for (int w = w0; w < w1; ++w) mine += __popc(bits[w] & bits_below(w, n_pages));
  __syncthreads();

  int want = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    copy[j] = exempt[j] = false;
    if (r0 + j < r1 && a[j].tail >= 0) {
      int before = 0;
      for (int q = 0; q < r0 + j; ++q) before += s_tail[q] == a[j].tail;
      copy[j] = ref[a[j].tail] - before > 1;
      exempt[j] = !copy[j];
    }
    if (r0 + j < r1) want += a[j].missing + copy[j];
  }
  int all, n_free;
  const int base0 = block_exclusive_scan(want, lds, &all);
  const int free0 = block_exclusive_scan(mine, lds, &n_free);

  bool ok[4];
  int base[4], at = base0, n_copies = 0, alloc = 0;
  bool refused = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    ok[j] = false;
    base[j] = at;
    if (r0 + j < r1) {
      const int cnt = a[j].missing + copy[j];
      const bool none_failed = at <= n_free;  // nobody before this request was refused for want of pages
      at += cnt;
      ok[j] = a[j].n > 0 && (cnt > 0 ? at <= n_free : true) && (!exempt[j] || none_failed);
      if (ok[j] && cnt > 0) alloc = at;
      if (!ok[j] && rows_of(ell[r0 + j], gamma) > 0) refused = true;
      n_copies += ok[j] && copy[j];
    }
  }
  // requests that got pages are a prefix of those that asked: ranks below s_alloc are theirs
  if (alloc > 0) atomicMax(&s_alloc, alloc);
  if (refused) atomicOr(&s_refused, 1);
  int copies;
  int pair = block_exclusive_scan(n_copies, lds, &copies);  // its barriers also publish s_alloc
  const int n_alloc = s_alloc;
  for (int w = w0, rank = free0; w < w1 && rank < n_alloc; ++w) {
    uint32_t b = bits[w] & bits_below(w, n_pages);
    const uint32_t was = b;
    uint32_t taken = 0;
    while (b && rank < n_alloc) {
      const uint32_t low = b & (~b + 1u);
      ids[rank++] = w * 32 + __ffs(b) - 1;
      taken |= low;
      b ^= low;
    }
    if (taken) bits[w] = was & ~taken;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (r0 + j < r1) {
      const int r = r0 + j;
      int32_t* row = table + static_cast<int64_t>(r) * max_pages;
      ell_out[r] = ok[j] ? a[j].n - 1 : -1;
      if (!ok[j]) continue;
      int k = base[j];
      if (copy[j]) {
        const int id = ids[k++];
        pairs[2 * pair] = a[j].tail;
        pairs[2 * pair + 1] = id;
        ++pair;
        atomicSub(&ref[a[j].tail], 1);
        ref[id] = 1;
        row[a[j].first] = id;
      }
      for (int i = a[j].first; i < a[j].last; ++i)
        if (page_or_none(row[i], n_pages) < 0) {
          const int id = ids[k++];
          ref[id] = 1;
          row[i] = id;
        }
    }
  if (threadIdx.x == 0) {
    *n_pairs = copies;
    if (status) *status = s_refused ? DSPARK_ENOPAGES : DSPARK_OK;
  }
}

// One wave per request.  Pages in use are contiguous in a row (released ones
// lie before them, free entries behind) but for those that dspark_cache_evict
// let go, which read kEvicted: both searches end at another entry that is no
// page, and the second one's way is marked -1 as far as it came.
__global__ __launch_bounds__(256) void cache_commit_kernel(int R, int gamma, int P, int n_pages, int max_pages,
                                                           int window, int sinks, const int32_t* ell,
                                                           const int32_t* n_acc, int32_t* len, int32_t* table,
                                                           int32_t* ref, uint32_t* bits) {
  const int r = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (r >= R) return;
  const int n = rows_of(ell[r], gamma);
  if (n == 0) return;
  const int64_t cap = static_cast<int64_t>(max_pages) * P;
  int64_t end = static_cast<int64_t>(len[r]) + min(max(n_acc[r], 0), n - 1) + 1;
  if (end > cap) end = cap;
  if (end < 0) end = 0;
  if (lane == 0) len[r] = static_cast<int32_t>(end);
  int32_t* row = table + static_cast<int64_t>(r) * max_pages;
  for (int64_t i = (end + P - 1) / P + lane; ; i += 64) {
    const int id = i < max_pages ? row[i] : -1;
    if (id >= 0) {
      row[i] = -1;
      release(id, n_pages, ref, bits);
    }
    if (__ballot(id < 0)) break;
  }
  if (window <= 0) return;
  // a later row sees nothing at or before end - window: pages up to dead - 1 hold nothing else
  const int64_t dead = (end - window + 1) >= P ? (end - window + 1) / P : 0;
  const int64_t keep = (static_cast<int64_t>(sinks) + P - 1) / P;
  for (int64_t i = dead - 1 - lane; ; i -= 64) {
    const int id = i >= keep ? row[i] : -1;
    if (id >= 0 || id == kEvicted) {
      row[i] = -1;
      release(id, n_pages, ref, bits);
    }
    if (__ballot(id < 0 && id != kEvicted)) break;
  }
}

__device__ __forceinline__ int fork_source(int r, int R, const int32_t* from) {
  const int s = from[r];
  return s < -1 || s >= R ? r : s;
}

// First launch: every new row is gathered into the workspace and its pages
// counted, from rows nobody has changed yet.  Second launch: the old rows'
// pages are let go.  All increments come before all decrements, so a page
// that one request drops and another takes never looks free in between.
__global__ __launch_bounds__(256) void cache_fork_take(int R, int P, int n_pages, int max_pages, const int32_t* from,
                                                       const int32_t* len, const int32_t* table, int32_t* ref,
                                                       int32_t* new_table, int32_t* new_len) {
  const int r = blockIdx.x, s = fork_source(r, R, from);
  if (s == r || s < 0) return;
  int64_t pages = (static_cast<int64_t>(max(len[s], 0)) + P - 1) / P;
  if (pages > max_pages) pages = max_pages;
  if (threadIdx.x == 0) new_len[r] = len[s];
  const int32_t* src = table + static_cast<int64_t>(s) * max_pages;
  int32_t* dst = new_table + static_cast<int64_t>(r) * max_pages;
  for (int i = threadIdx.x; i < max_pages; i += 256) {
    const int id = i < pages ? page_or_mark(src[i], n_pages) : -1;
    dst[i] = id;
    if (id >= 0) atomicAdd(&ref[id], 1);
  }
}

__global__ __launch_bounds__(256) void cache_fork_drop(int R, int n_pages, int max_pages, const int32_t* from,
                                                       int32_t* len, int32_t* table, int32_t* ref, uint32_t* bits,
                                                       const int32_t* new_table, const int32_t* new_len) {
  const int r = blockIdx.x, s = fork_source(r, R, from);
  if (s == r) return;
  int32_t* row = table + static_cast<int64_t>(r) * max_pages;
  for (int i = threadIdx.x; i < max_pages; i += 256) {
    release(row[i], n_pages, ref, bits);
    row[i] = s < 0 ? -1 : new_table[static_cast<int64_t>(r) * max_pages + i];
  }
  if (threadIdx.x == 0) len[r] = s < 0 ? 0 : new_len[r];
}

// Both in one launch of one work group for tables of at most 4 kT entries,
// a thread's four in registers: a round's bookkeeping (fork, reserve, copy,
// commit) of 128 requests x 18 pages takes the GPU 23.2 us with it and 22.8
// with two launches, and the host 35.5 us instead of 38.7.
constexpr int kForkPer = 4;
__global__ __launch_bounds__(kT) void cache_fork_small(int R, int P, int n_pages, int max_pages, const int32_t* from,
                                                       int32_t* len, int32_t* table, int32_t* ref, uint32_t* bits) {
  const int n = R * max_pages;
  int id[kForkPer], old[kForkPer], new_len[kForkPer];
  bool mine[kForkPer];
#pragma unroll
  for (int j = 0; j < kForkPer; ++j) {
    const int e = j * kT + threadIdx.x;
    mine[j] = e < n;
    id[j] = old[j] = -1;
    new_len[j] = 0;
    if (!mine[j]) continue;
    const int r = e / max_pages, i = e - r * max_pages, s = fork_source(r, R, from);
    mine[j] = s != r;
    if (s == r) continue;
    old[j] = page_or_none(table[e], n_pages);
    if (s < 0) continue;
    new_len[j] = len[s];
    const int64_t pages = (static_cast<int64_t>(max(new_len[j], 0)) + P - 1) / P;
    if (i < pages) id[j] = page_or_mark(table[s * max_pages + i], n_pages);
  }
#pragma unroll
  for (int j = 0; j < kForkPer; ++j)
    if (id[j] >= 0) atomicAdd(&ref[id[j]], 1);
  // all increments before all decrements, all reads before all writes; one
  // work group, so its barrier orders them
  __syncthreads();
  int was[kForkPer];
#pragma unroll
  for (int j = 0; j < kForkPer; ++j) was[j] = old[j] >= 0 ? atomicSub(&ref[old[j]], 1) : 0;
#pragma unroll
  for (int j = 0; j < kForkPer; ++j)
    if (mine[j]) {
      const int e = j * kT + threadIdx.x;
      if (was[j] == 1) atomicOr(&bits[old[j] >> 5], 1u << (old[j] & 31));
      table[e] = id[j];
      if (e % max_pages == 0) len[e / max_pages] = new_len[j];
    }
}

// Eviction, a work group a request: the k-th smallest mass of the pages that
// may go is found a byte at a time from the top (at most four passes over keys,
// their counts in LDS), as far down as it takes until all pages up to some key
// go; then they do, and of equal masses that cannot all go the first by entry.
// Keys of up to kEvictPer a thread stay in registers, of longer tables they are
// made again from memory in every pass.
//
// Bound by its chain of loads and, where many pages go, by the writes that let
// go of them: 4.2 us for a request of 63 pages; 64 requests of up to 8192 pages
// of 16 tokens, 4096 of which stay, 27 us: 2 for the passes, 13 for the pages
// that go (7 of them the bitmap's atomics), the rest to load the table and the
// masses.
constexpr int kEvictPer = 8;

// Smaller mass, smaller key; -0 as 0, NaN above all.
__device__ __forceinline__ uint32_t mass_key(float m) {
  return m != m ? 0xFFFFFFFFu : ordered_bits(m + 0.f);
}

// As release, for a kernel in which counts only fall: a page that nobody else
// holds (`holders`, read before) is nobody else's to count.
__device__ __forceinline__ void release_own(int id, int holders, int32_t* ref, uint32_t* bits) {
  if (holders == 1) ref[id] = 0;
  else if (atomicSub(&ref[id], 1) != 1) return;
  atomicOr(&bits[id >> 5], 1u << (id & 31));
}

template <int T, bool LONG>
__global__ __launch_bounds__(T) void cache_evict_kernel(int P, int n_pages, int max_pages, int sinks, int recent,
                                                        const int32_t* budget, const int32_t* len, float* mass,
                                                        int32_t* table, int32_t* ref, uint32_t* bits, int32_t* freed) {
  constexpr int W = T / 64;
  __shared__ int2 sums[W];
  __shared__ int count[256];
  __shared__ int s_digit, s_left, s_inside;
  const int r = blockIdx.x, most = budget[r];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t n = len[r];
  int32_t* row = table + static_cast<int64_t>(r) * max_pages;
  float* weight = mass + static_cast<int64_t>(r) * max_pages;
  const int used = n <= 0 ? 0 : static_cast<int>(min((n + P - 1) / P, static_cast<int64_t>(max_pages)));
  if (most < 0 || used <= most) {  // the same for all threads
    if (threadIdx.x == 0 && freed) freed[r] = 0;
    return;
  }
  // entries that may go: first .. end - 1
  const int first = static_cast<int>(min((static_cast<int64_t>(sinks) + P - 1) / P, static_cast<int64_t>(used)));
  const int end = n > recent ? static_cast<int>(min((n - recent) / P, static_cast<int64_t>(used))) : 0;
  const int rounds = ceil_div(used, T);
  int id[kEvictPer];       // -1: may not go
  uint32_t key[kEvictPer];
  int held = 0, able = 0;
  auto look = [&](int i, int& page, uint32_t& k) {
    const int s = i * T + threadIdx.x;
    page = s < used ? page_or_none(row[s], n_pages) : -1;
    const float m = s < used ? weight[s] : 0.f;
    held += page >= 0;
    if (s < first || s >= end) page = -1;
    able += page >= 0;
    k = mass_key(m);
  };
  // f(round, page, key) for this thread's entries, all of one round at a time
  auto all = [&](auto f) {
    if constexpr (LONG) {
#pragma unroll 1
      for (int i = 0; i < rounds; ++i) {
        look(i, id[0], key[0]);
        f(i, id[0], key[0]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kEvictPer; ++i)
        if (i < rounds) f(i, id[i], key[i]);
    }
  };
  if constexpr (LONG) {
    all([](int, int, uint32_t) {});
  } else {
#pragma unroll
    for (int i = 0; i < kEvictPer; ++i) look(i, id[i], key[i]);
  }
  auto sum = [](int p, int q) { return p + q; };
  const int held_w = wave_scan(held, sum), able_w = wave_scan(able, sum);
  if (lane == 63) sums[wave] = make_int2(held_w, able_w);
  for (int i = threadIdx.x; i < 256; i += T) count[i] = 0;
  __syncthreads();
  held = able = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) held += sums[w].x, able += sums[w].y;
  const int k = min(held - most, able);
  if (threadIdx.x == 0 && freed) freed[r] = max(k, 0);
  if (k <= 0) return;
  // keys whose bits under `mask` are below `prefix` go, and `left` of those that
  // equal it, which are `inside` in all
  uint32_t prefix = 0, mask = 0;
  int left = k, inside = able;
#pragma unroll 1
  for (int shift = 24; shift >= 0 && left < inside; shift -= 8) {
    all([&](int, int page, uint32_t x) {
      if (page >= 0 && (x & mask) == prefix) atomicAdd(&count[(x >> shift) & 255], 1);
    });
    __syncthreads();
    if (wave == 0) {  // four counts a lane, cleared for the next pass
      int c[4], before = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[j] = count[lane * 4 + j];
        before += c[j];
        count[lane * 4 + j] = 0;
      }
      before = wave_scan(before, sum) - before;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (before < left && left <= before + c[j]) s_digit = lane * 4 + j, s_left = left - before, s_inside = c[j];
        before += c[j];
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    mask |= 0xFFu << shift;
    left = s_left;
    inside = s_inside;
  }
  int before = 0;  // equal ones in the rounds so far
  auto goes = [&](int page, uint32_t x) {
    const uint32_t y = x & mask;
    if (left == inside) return page >= 0 && y <= prefix;
    const bool tie = page >= 0 && y == prefix;
    const int incl = wave_scan(static_cast<int>(tie), sum);
    __syncthreads();
    if (lane == 63) sums[wave].x = incl;
    __syncthreads();
    int at = before + incl - tie;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < wave) at += sums[w].x;
      before += sums[w].x;
    }
    return page >= 0 && (y < prefix || (tie && at < left));
  };
  auto drop = [&](int i, int page, int holders) {
    const int s = i * T + threadIdx.x;
    release_own(page, holders, ref, bits);
    row[s] = kEvicted;
    weight[s] = 0.f;
  };
  if constexpr (LONG) {
    all([&](int i, int page, uint32_t x) {
      if (goes(page, x)) drop(i, page, ref[page]);
    });
  } else {
    // all counts on their way before the first is used
    int holders[kEvictPer];
    all([&](int i, int page, uint32_t x) {
      if (!goes(page, x)) id[i] = -1;
      holders[i] = id[i] >= 0 ? ref[id[i]] : 0;
    });
    all([&](int i, int page, uint32_t) {
      if (page >= 0) drop(i, page, holders[i]);
    });
  }
}

// ws: word 0 = U, then the new id of every page that moves.
__global__ __launch_bounds__(kT) void cache_compact_plan(int n_pages, uint32_t* bits, int32_t* pairs,
                                                         int32_t* n_pairs, int32_t* used, int32_t* map) {
  __shared__ int lds[kT / 64];
  const int words = (n_pages + 31) / 32;
  const int wper = ceil_div(words, kT);
  const int w0 = min(words, static_cast<int>(threadIdx.x) * wper), w1 = min(words, w0 + wper);
  int n = 0, free_pages;
  for (int w = w0; w < w1; ++w) n += __popc(bits[w] & bits_below(w, n_pages));
  block_exclusive_scan(n, lds, &free_pages);
  const int U = n_pages - free_pages;
  int movers = 0, holes = 0;
  for (int w = w0; w < w1; ++w) {
    const uint32_t low = bits_below(w, U), valid = bits_below(w, n_pages), b = bits[w] & valid;
    holes += __popc(b & low);
    movers += __popc(~b & valid & ~low);
  }
  int total;
  int h = block_exclusive_scan(holes, lds, &total);
  int m = block_exclusive_scan(movers, lds, &total);
  for (int w = w0; w < w1; ++w) {
    const uint32_t low = bits_below(w, U), valid = bits_below(w, n_pages), b = bits[w] & valid;
    for (uint32_t x = b & low; x; x &= x - 1) pairs[2 * h++ + 1] = w * 32 + __ffs(x) - 1;
    for (uint32_t x = ~b & valid & ~low; x; x &= x - 1) pairs[2 * m++] = w * 32 + __ffs(x) - 1;
    bits[w] = valid & ~low;
  }
  if (threadIdx.x == 0) {
    *n_pairs = total;
    *used = U;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += kT) map[pairs[2 * i]] = pairs[2 * i + 1];
}

__global__ __launch_bounds__(256) void cache_compact_apply(int64_t n_table, int n_pages, int32_t* table, int32_t* ref,
                                                           const int32_t* pairs, const int32_t* n_pairs,
                                                           const int32_t* used, const int32_t* map) {
  const int U = *used, n = *n_pairs;
  for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < n_table || i < n; i += gridDim.x * 256LL) {
    if (i < n) {
      ref[pairs[2 * i + 1]] = ref[pairs[2 * i]];
      ref[pairs[2 * i]] = 0;
    }
    if (i < n_table) {
      const int id = page_or_none(table[i], n_pages);
      if (id >= U) table[i] = map[id];
    }
  }
}

// Work groups take 16 KB pieces in turn; a thread moves four 16-byte words,
// all loads ahead of the stores.
constexpr int kPiece = 16384;
__global__ __launch_bounds__(256) void cache_copy_kernel(int layers, int64_t layer_bytes, int64_t page_bytes,
                                                         int n_pages, const int32_t* pairs, const int32_t* n_pairs,
                                                         int max_pairs, char* pool) {
  const int n = min(max(*n_pairs, 0), max_pairs);
  const int per_page = ceil_div(page_bytes, kPiece);
  const int64_t pieces = static_cast<int64_t>(n) * layers * per_page;
  for (int64_t i = blockIdx.x; i < pieces; i += gridDim.x) {
    const int64_t page = i / per_page;
    const int pair = static_cast<int>(page / layers), layer = static_cast<int>(page % layers);
    const int src = page_or_none(pairs[2 * pair], n_pages), dst = page_or_none(pairs[2 * pair + 1], n_pages);
    if (src < 0 || dst < 0) continue;
    const int64_t off = (i % per_page) * kPiece;
    const int64_t left = page_bytes - off;
    char* base = pool + layer * layer_bytes + off;
    const char* from = base + src * page_bytes;
    char* to = base + dst * page_bytes;
    u32x4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t b = (j * 256 + threadIdx.x) * 16LL;
      if (b < left) x[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from + b));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t b = (j * 256 + threadIdx.x) * 16LL;
      if (b < left) __builtin_nontemporal_store(x[j], reinterpret_cast<u32x4*>(to + b));
    }
  }
}

}  // namespace

hipError_t cache_reset_launch(int R, int n_pages, int max_pages, int32_t* table, int32_t* len, int32_t* ref,
                              uint32_t* bits, hipStream_t s) {
  const int64_t n_table = static_cast<int64_t>(R) * max_pages;
  const int64_t n = n_table > n_pages ? n_table : n_pages;
  const int blocks = n / 256 + 1 > 2048 ? 2048 : static_cast<int>(n / 256 + 1);
  cache_reset_kernel<<<blocks, 256, 0, s>>>(n_table, R, n_pages, table, len, ref, bits);
  return hipGetLastError();
}

hipError_t cache_reserve_launch(int R, int gamma, int P, int n_pages, int max_pages, const int32_t* ell,
                                const int32_t* len, int32_t* table, int32_t* ref, uint32_t* bits, int32_t* ell_out,
                                int32_t* pairs, int32_t* n_pairs, int32_t* status, void* ws, hipStream_t s) {
  cache_reserve_kernel<<<1, kT, 0, s>>>(R, gamma, P, n_pages, max_pages, ell, len, table, ref, bits, ell_out, pairs,
                                        n_pairs, status, static_cast<int32_t*>(ws));
  return hipGetLastError();
}

hipError_t cache_commit_launch(int R, int gamma, int P, int n_pages, int max_pages, int window, int sinks,
                               const int32_t* ell, const int32_t* n_acc, int32_t* len, int32_t* table, int32_t* ref,
                               uint32_t* bits, hipStream_t s) {
  cache_commit_kernel<<<ceil_div(R, 4), 256, 0, s>>>(R, gamma, P, n_pages, max_pages, window, sinks, ell, n_acc, len,
                                                     table, ref, bits);
  return hipGetLastError();
}

hipError_t cache_evict_launch(int R, int P, int n_pages, int max_pages, int sinks, int recent, const int32_t* budget,
                              const int32_t* len, float* mass, int32_t* table, int32_t* ref, uint32_t* bits,
                              int32_t* freed, hipStream_t s) {
  auto launch = [&](auto kernel, int threads) {
    kernel<<<R, threads, 0, s>>>(P, n_pages, max_pages, sinks, recent, budget, len, mass, table, ref, bits, freed);
  };
  // few entries: a small work group, whose barriers cost less.  A request of 128
  // pages takes 5.1 us (1024 threads 5.9), of 256 5.9 (6.2), 64 of 256 8.6 (9.1), of
  // 512 9.5 (9.8), 256 of 512 11.6 (11.9); but a lone one of 400 pages 7.6 (6.9 ..
  // 7.1), of 512 7.0 (6.9), and 64 of 768 would take 11.9 (10.9).  Long tables are read again in each pass: 64 of up to
  // 8192 would take 38 so, 30 with their keys in registers.
  if (max_pages <= 4 * 128) launch(cache_evict_kernel<128, false>, 128);
  else if (max_pages <= kEvictPer * kT) launch(cache_evict_kernel<kT, false>, kT);
  else launch(cache_evict_kernel<kT, true>, kT);
  return hipGetLastError();
}

hipError_t cache_fork_launch(int R, int P, int n_pages, int max_pages, const int32_t* from, int32_t* len,
                             int32_t* table, int32_t* ref, uint32_t* bits, void* ws, hipStream_t s) {
  if (static_cast<int64_t>(R) * max_pages <= kForkPer * kT) {
    cache_fork_small<<<1, kT, 0, s>>>(R, P, n_pages, max_pages, from, len, table, ref, bits);
    return hipGetLastError();
  }
  int32_t* new_len = static_cast<int32_t*>(ws);
  int32_t* new_table = new_len + (R + 63) / 64 * 64;
  cache_fork_take<<<R, 256, 0, s>>>(R, P, n_pages, max_pages, from, len, table, ref, new_table, new_len);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  cache_fork_drop<<<R, 256, 0, s>>>(R, n_pages, max_pages, from, len, table, ref, bits, new_table, new_len);
  return hipGetLastError();
}

hipError_t cache_compact_launch(int R, int n_pages, int max_pages, int32_t* table, int32_t* ref, uint32_t* bits,
                                int32_t* pairs, int32_t* n_pairs, void* ws, hipStream_t s) {
  int32_t* used = static_cast<int32_t*>(ws);
  int32_t* map = used + 64;
  cache_compact_plan<<<1, kT, 0, s>>>(n_pages, bits, pairs, n_pairs, used, map);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t n_table = static_cast<int64_t>(R) * max_pages;
  const int64_t n = n_table > n_pages / 2 ? n_table : n_pages / 2;
  const int blocks = n / 256 + 1 > 2048 ? 2048 : static_cast<int>(n / 256 + 1);
  cache_compact_apply<<<blocks, 256, 0, s>>>(n_table, n_pages, table, ref, pairs, n_pairs, used, map);
  return hipGetLastError();
}

hipError_t cache_copy_launch(int layers, int64_t layer_bytes, int64_t page_bytes, int n_pages, const int32_t* pairs,
                             const int32_t* n_pairs, int max_pairs, void* pool, hipStream_t s) {
  const int64_t pieces = static_cast<int64_t>(max_pairs) * layers * ceil_div(page_bytes, kPiece);
  const int64_t most = 8LL * compute_units();
  cache_copy_kernel<<<static_cast<int>(pieces < most ? pieces : most), 256, 0, s>>>(
      layers, layer_bytes, page_bytes, n_pages, pairs, n_pairs, max_pairs, static_cast<char*>(pool));
  return hipGetLastError();
}

}  // namespace dspark
