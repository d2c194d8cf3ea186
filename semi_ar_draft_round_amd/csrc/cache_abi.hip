// The C ABI of the paged cache (include/dspark_cache.h): argument checks and
// workspace sizes.  Every check that needs no device data happens here.
#include <math.h>

#include "cache.hpp"

namespace dspark {
// cache_append.hip
hipError_t cache_append_launch(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages, int max_pages,
                               const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                               const void* wq, const void* wk, float eps, const double* freq, int rot, int adjacent,
                               const int32_t* row0, const int32_t* ell, const int32_t* len, const int32_t* table,
                               void* q_out, void* pool, hipStream_t s);
hipError_t cache_read_launch(int fmt, int R, int T, int Hkv, int D, int P, int n_pages, int max_pages,
                             const int32_t* start, const int32_t* count, const int32_t* table, const void* pool,
                             void* k, void* v, hipStream_t s);
// cache_attention.hip
size_t cache_attention_workspace_bytes(int gamma, int Hq, int Hkv, int D);
hipError_t cache_attention_launch(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages,
                                  int max_pages, const void* q, float scale, int window, int sinks,
                                  const int32_t* row0, const int32_t* ell, const int32_t* len, const int32_t* table,
                                  const void* pool, void* out, float* lse, void* ws, hipStream_t s);
// cache_weigh.hip
hipError_t cache_weigh_launch(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages, int max_pages,
                              const void* q, float scale, int window, int sinks, const float* lse,
                              const int32_t* row0, const int32_t* ell, const int32_t* len, const int32_t* table,
                              const void* pool, float keep, float* mass, hipStream_t s);
// cache_pages.hip
hipError_t cache_evict_launch(int R, int P, int n_pages, int max_pages, int sinks, int recent, const int32_t* budget,
                              const int32_t* len, float* mass, int32_t* table, int32_t* ref, uint32_t* bits,
                              int32_t* freed, hipStream_t s);
hipError_t cache_reset_launch(int R, int n_pages, int max_pages, int32_t* table, int32_t* len, int32_t* ref,
                              uint32_t* bits, hipStream_t s);
hipError_t cache_reserve_launch(int R, int gamma, int P, int n_pages, int max_pages, const int32_t* ell,
                                const int32_t* len, int32_t* table, int32_t* ref, uint32_t* bits, int32_t* ell_out,
                                int32_t* pairs, int32_t* n_pairs, int32_t* status, void* ws, hipStream_t s);
hipError_t cache_commit_launch(int R, int gamma, int P, int n_pages, int max_pages, int window, int sinks,
                               const int32_t* ell, const int32_t* n_acc, int32_t* len, int32_t* table, int32_t* ref,
                               uint32_t* bits, hipStream_t s);
hipError_t cache_fork_launch(int R, int P, int n_pages, int max_pages, const int32_t* from, int32_t* len,
                             int32_t* table, int32_t* ref, uint32_t* bits, void* ws, hipStream_t s);
hipError_t cache_compact_launch(int R, int n_pages, int max_pages, int32_t* table, int32_t* ref, uint32_t* bits,
                                int32_t* pairs, int32_t* n_pairs, void* ws, hipStream_t s);
hipError_t cache_copy_launch(int layers, int64_t layer_bytes, int64_t page_bytes, int n_pages, const int32_t* pairs,
                             const int32_t* n_pairs, int max_pairs, void* pool, hipStream_t s);

namespace {

bool format_ok(int fmt) { return fmt == DSPARK_CACHE_BF16 || fmt == DSPARK_CACHE_FP4 || fmt == DSPARK_CACHE_FP8; }
bool page_ok(int P) { return P == 16 || P == 32 || P == 64 || P == 128; }
bool dim_ok(int D) { return D == 64 || D == 128 || D == 256; }
bool heads_ok(int H) { return H >= 1 && H <= kCacheMaxHeads; }
bool batch_ok(int R, int gamma) { return R >= 1 && R <= kCacheMaxR && gamma >= 0 && gamma <= kCacheMaxGamma; }
bool pages_ok(int R, int n_pages, int max_pages) {
  return R >= 1 && R <= kCacheMaxR && n_pages >= 1 && n_pages <= kCacheMaxPages && max_pages >= 1 &&
         max_pages <= kCacheMaxPages && static_cast<int64_t>(R) * max_pages < (1LL << 31);
}

// Pointers that the kernels read or write in 16-byte words.
template <typename... T>
bool aligned(const T*... p) {
  return ((reinterpret_cast<uintptr_t>(p) % 16 == 0) && ...);
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

dspark_status launched(hipError_t e) { return e == hipSuccess ? DSPARK_OK : DSPARK_ELAUNCH; }

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

size_t dspark_cache_page_bytes(int fmt, int Hkv, int D, int P) {
  if (!format_ok(fmt) || !heads_ok(Hkv) || !dim_ok(D) || !page_ok(P)) return 0;
  if (fmt == DSPARK_CACHE_FP8) return (2 * static_cast<size_t>(P) * D + 16) * Hkv;
  const size_t token = fmt == DSPARK_CACHE_BF16 ? 4 * static_cast<size_t>(D) : static_cast<size_t>(D) + D / 32 + 4;
  return token * P * Hkv;
}

size_t dspark_cache_workspace_size(dspark_cache_ws_kind kind, int R, int gamma, int a, int b, int c) {
  switch (kind) {
    case DSPARK_CACHE_WS_ATTENTION:
      if (!batch_ok(R, gamma) || !heads_ok(a) || !heads_ok(b) || a % b != 0 || !dim_ok(c)) return 0;
      return round256(cache_attention_workspace_bytes(gamma, a, b, c));
    case DSPARK_CACHE_WS_RESERVE:  // the ids handed out
      if (!pages_ok(R, b, a)) return 0;
      return round256(4 * static_cast<size_t>(b));
    case DSPARK_CACHE_WS_FORK:  // the new lengths and rows
      if (!pages_ok(R, b, a)) return 0;
      return round256(4 * static_cast<size_t>(R)) + round256(4 * static_cast<size_t>(R) * a);
    case DSPARK_CACHE_WS_COMPACT:  // the number of pages in use and the new ids
      if (!pages_ok(R, b, a)) return 0;
      return 256 + round256(4 * static_cast<size_t>(b));
  }
  return 0;
}

dspark_status dspark_cache_append(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages,
                                  int max_pages, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                  const void* v, int64_t ldv, const void* wq, const void* wk, float eps,
                                  const double* freq, int rot, int adjacent, const int32_t* row0, const int32_t* ell,
                                  const int32_t* len, const int32_t* table, void* q_out, void* pool, void* stream) {
  if (!format_ok(fmt)) return DSPARK_EDTYPE;
  if (!batch_ok(R, gamma) || !heads_ok(Hq) || !heads_ok(Hkv) || !dim_ok(D) || !page_ok(P) ||
      !pages_ok(R, n_pages, max_pages))
    return DSPARK_EINVAL;
  if (ldq < static_cast<int64_t>(Hq) * D || ldk < static_cast<int64_t>(Hkv) * D ||
      ldv < static_cast<int64_t>(Hkv) * D || ldq % 8 != 0 || ldk % 8 != 0 || ldv % 8 != 0 ||
      ldq >= (1LL << 31) || ldk >= (1LL << 31) || ldv >= (1LL << 31))
    return DSPARK_EINVAL;
  if (rot < 0 || rot > D || rot % 2 != 0 || (!adjacent && rot % 16 != 0) || (rot > 0 && !freq)) return DSPARK_EINVAL;
  if (!(eps >= 0.f) || isinf(eps)) return DSPARK_EINVAL;
  if (!q || !k || !v || !ell || !len || !table || !q_out || !pool) return DSPARK_EINVAL;
  if (!aligned(static_cast<const char*>(q), static_cast<const char*>(k), static_cast<const char*>(v),
               static_cast<const char*>(wq), static_cast<const char*>(wk), static_cast<const char*>(q_out),
               static_cast<const char*>(pool)))
    return DSPARK_EINVAL;
  dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(cache_append_launch(fmt, R, gamma, Hq, Hkv, D, P, n_pages, max_pages, q, ldq, k, ldk, v, ldv, wq, wk,
                                      eps, freq, rot, adjacent, row0, ell, len, table, q_out, pool,
                                      static_cast<hipStream_t>(stream)));
}

dspark_status dspark_cache_attention(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages,
                                     int max_pages, const void* q, float scale, int window, int sinks,
                                     const int32_t* row0, const int32_t* ell, const int32_t* len,
                                     const int32_t* table, const void* pool, void* out, float* lse, void* ws,
                                     size_t ws_bytes, void* stream) {
  if (!format_ok(fmt)) return DSPARK_EDTYPE;
  if (!batch_ok(R, gamma) || !heads_ok(Hq) || !heads_ok(Hkv) || Hq % Hkv != 0 || !dim_ok(D) || !page_ok(P) ||
      !pages_ok(R, n_pages, max_pages))
    return DSPARK_EINVAL;
  if (window < 0 || sinks < 0 || !(fabsf(scale) <= 0x1p126f)) return DSPARK_EINVAL;  // times log2 e: still finite
  if (!q || !ell || !len || !table || !pool || !out) return DSPARK_EINVAL;
  if (!aligned(static_cast<const char*>(q), static_cast<const char*>(pool), static_cast<const char*>(out),
               static_cast<const char*>(ws)))
    return DSPARK_EINVAL;
  if (!ws || ws_bytes < round256(cache_attention_workspace_bytes(gamma, Hq, Hkv, D))) return DSPARK_EWORKSPACE;
  dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(cache_attention_launch(fmt, R, gamma, Hq, Hkv, D, P, n_pages, max_pages, q, scale, window, sinks,
                                         row0, ell, len, table, pool, out, lse, ws,
                                         static_cast<hipStream_t>(stream)));
}

dspark_status dspark_cache_read(int fmt, int R, int T, int Hkv, int D, int P, int n_pages, int max_pages,
                                const int32_t* start, const int32_t* count, const int32_t* table, const void* pool,
                                void* k, void* v, void* stream) {
  if (!format_ok(fmt)) return DSPARK_EDTYPE;
  if (!heads_ok(Hkv) || !dim_ok(D) || !page_ok(P) || !pages_ok(R, n_pages, max_pages) || T < 1 || T > kCacheMaxT)
    return DSPARK_EINVAL;
  if (!count || !table || !pool || !k || !v) return DSPARK_EINVAL;
  if (!aligned(static_cast<const char*>(pool), static_cast<const char*>(k), static_cast<const char*>(v)))
    return DSPARK_EINVAL;
  dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(cache_read_launch(fmt, R, T, Hkv, D, P, n_pages, max_pages, start, count, table, pool, k, v,
                                    static_cast<hipStream_t>(stream)));
}

dspark_status dspark_cache_weigh(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages,
                                 int max_pages, const void* q, float scale, int window, int sinks, const float* lse,
                                 const int32_t* row0, const int32_t* ell, const int32_t* len, const int32_t* table,
                                 const void* pool, float keep, float* mass, void* stream) {
  if (!format_ok(fmt)) return DSPARK_EDTYPE;
  if (!batch_ok(R, gamma) || !heads_ok(Hq) || !heads_ok(Hkv) || Hq % Hkv != 0 || !dim_ok(D) || !page_ok(P) ||
      !pages_ok(R, n_pages, max_pages))
    return DSPARK_EINVAL;
  if (window < 0 || sinks < 0 || !(fabsf(scale) <= 0x1p126f)) return DSPARK_EINVAL;  // times log2 e: still finite
  if (!(keep >= 0.f) || isinf(keep)) return DSPARK_EINVAL;
  if (!q || !lse || !ell || !len || !table || !pool || !mass) return DSPARK_EINVAL;
  if (!aligned(static_cast<const char*>(q), static_cast<const char*>(pool))) return DSPARK_EINVAL;
  dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(cache_weigh_launch(fmt, R, gamma, Hq, Hkv, D, P, n_pages, max_pages, q, scale, window, sinks, lse,
                                     row0, ell, len, table, pool, keep, mass, static_cast<hipStream_t>(stream)));
}

dspark_status dspark_cache_evict(int R, int P, int n_pages, int max_pages, int sinks, int recent,
                                 const int32_t* budget, const int32_t* len, float* mass, int32_t* table,
                                 int32_t* ref, uint32_t* bits, int32_t* freed, void* stream) {
  if (!page_ok(P) || !pages_ok(R, n_pages, max_pages) || sinks < 0 || recent < 0) return DSPARK_EINVAL;
  if (!budget || !len || !mass || !table || !ref || !bits) return DSPARK_EINVAL;
  dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(cache_evict_launch(R, P, n_pages, max_pages, sinks, recent, budget, len, mass, table, ref, bits,
                                     freed, static_cast<hipStream_t>(stream)));
}

dspark_status dspark_cache_reset(int R, int n_pages, int max_pages, int32_t* table, int32_t* len, int32_t* ref,
                                 uint32_t* bits, void* stream) {
  if (!pages_ok(R, n_pages, max_pages) || !table || !len || !ref || !bits) return DSPARK_EINVAL;
  dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(cache_reset_launch(R, n_pages, max_pages, table, len, ref, bits, static_cast<hipStream_t>(stream)));
}

dspark_status dspark_cache_reserve(int R, int gamma, int P, int n_pages, int max_pages, const int32_t* ell,
                                   const int32_t* len, int32_t* table, int32_t* ref, uint32_t* bits,
                                   int32_t* ell_out, int32_t* pairs, int32_t* n_pairs, int32_t* status, void* ws,
                                   size_t ws_bytes, void* stream) {
  if (!batch_ok(R, gamma) || !page_ok(P) || !pages_ok(R, n_pages, max_pages)) return DSPARK_EINVAL;
  if (!ell || !len || !table || !ref || !bits || !ell_out || !pairs || !n_pairs ||
      !aligned(static_cast<const char*>(ws)))
    return DSPARK_EINVAL;
  if (!ws || ws_bytes < dspark_cache_workspace_size(DSPARK_CACHE_WS_RESERVE, R, gamma, max_pages, n_pages, 0))
    return DSPARK_EWORKSPACE;
  dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(cache_reserve_launch(R, gamma, P, n_pages, max_pages, ell, len, table, ref, bits, ell_out, pairs,
                                       n_pairs, status, ws, static_cast<hipStream_t>(stream)));
}

dspark_status dspark_cache_commit(int R, int gamma, int P, int n_pages, int max_pages, int window, int sinks,
                                  const int32_t* ell, const int32_t* n_acc, int32_t* len, int32_t* table,
                                  int32_t* ref, uint32_t* bits, void* stream) {
  if (!batch_ok(R, gamma) || !page_ok(P) || !pages_ok(R, n_pages, max_pages)) return DSPARK_EINVAL;
  if (window < 0 || sinks < 0) return DSPARK_EINVAL;
  if (!ell || !n_acc || !len || !table || !ref || !bits) return DSPARK_EINVAL;
  dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(cache_commit_launch(R, gamma, P, n_pages, max_pages, window, sinks, ell, n_acc, len, table, ref,
                                      bits, static_cast<hipStream_t>(stream)));
}

dspark_status dspark_cache_fork(int R, int P, int n_pages, int max_pages, const int32_t* from, int32_t* len,
                                int32_t* table, int32_t* ref, uint32_t* bits, void* ws, size_t ws_bytes,
                                void* stream) {
  if (!page_ok(P) || !pages_ok(R, n_pages, max_pages)) return DSPARK_EINVAL;
  if (!from || !len || !table || !ref || !bits || !aligned(static_cast<const char*>(ws))) return DSPARK_EINVAL;
  if (!ws || ws_bytes < dspark_cache_workspace_size(DSPARK_CACHE_WS_FORK, R, 0, max_pages, n_pages, 0))
    return DSPARK_EWORKSPACE;
  dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(cache_fork_launch(R, P, n_pages, max_pages, from, len, table, ref, bits, ws,
                                    static_cast<hipStream_t>(stream)));
}

dspark_status dspark_cache_compact(int R, int n_pages, int max_pages, int32_t* table, int32_t* ref, uint32_t* bits,
                                   int32_t* pairs, int32_t* n_pairs, void* ws, size_t ws_bytes, void* stream) {
  if (!pages_ok(R, n_pages, max_pages)) return DSPARK_EINVAL;
  if (!table || !ref || !bits || !pairs || !n_pairs || !aligned(static_cast<const char*>(ws))) return DSPARK_EINVAL;
  if (!ws || ws_bytes < dspark_cache_workspace_size(DSPARK_CACHE_WS_COMPACT, R, 0, max_pages, n_pages, 0))
    return DSPARK_EWORKSPACE;
  dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(cache_compact_launch(R, n_pages, max_pages, table, ref, bits, pairs, n_pairs, ws,
                                       static_cast<hipStream_t>(stream)));
}

dspark_status dspark_cache_copy(int layers, int64_t layer_bytes, int64_t page_bytes, int n_pages,
                                const int32_t* pairs, const int32_t* n_pairs, int max_pairs, void* pool,
                                void* stream) {
  if (layers < 1 || layers > (1 << 16) || page_bytes < 16 || page_bytes % 16 != 0 || page_bytes >= (1LL << 31) ||
      n_pages < 1 || n_pages > kCacheMaxPages || max_pairs < 1 || max_pairs > kCacheMaxPages)
    return DSPARK_EINVAL;
  if (layers > 1 && (layer_bytes % 16 != 0 || layer_bytes < n_pages * page_bytes)) return DSPARK_EINVAL;
  if (!pairs || !n_pairs || !pool || !aligned(static_cast<const char*>(pool))) return DSPARK_EINVAL;
  dspark_status st = check_device();
  if (st != DSPARK_OK) return st;
  return launched(cache_copy_launch(layers, layer_bytes, page_bytes, n_pages, pairs, n_pairs, max_pairs, pool,
                                    static_cast<hipStream_t>(stream)));
}

}  // extern "C"
