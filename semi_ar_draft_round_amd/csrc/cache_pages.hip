// Who owns the cache's pages: reserve, commit, fork, compact, copy, reset
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

// One wave per request.  Pages in use are contiguous in a row (evicted ones
// lie before them, free entries behind), so both searches end at a -1.
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
    if (id >= 0) {
      row[i] = -1;
      release(id, n_pages, ref, bits);
    }
    if (__ballot(id < 0)) break;
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
    const int id = i < pages ? page_or_none(src[i], n_pages) : -1;
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
    if (i < pages) id[j] = page_or_none(table[s * max_pages + i], n_pages);
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
