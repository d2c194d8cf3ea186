/*
 * dspark_cache.h — the paged key/value cache of a verification round.
 *
 * A round (dspark.h) admits ell[r] drafts of request r; the target then runs
 * over rows row0[r] .. row0[r] + ell[r] (the anchor and the admitted drafts,
 * caijizhuo section 四 step 5; notes, the flattened ragged verify batch), and
 * after dspark_verify the rows past n_acc[r] leave the cache again
 * (caijizhuo, rollback_kv).  These entry points are what that pass does to
 * the cache of one attention layer, and who owns its pages:
 *
 *   dspark_cache_append     per-head norm of queries and keys and the position
 *                           rotation in one pass; K and V go into the pages
 *   dspark_cache_attention  the rows' attention over the pages, optionally
 *                           with a sliding window and visible first tokens
 *   dspark_cache_read       cached tokens as dense rows
 *   dspark_cache_weigh      the attention weights that the tokens of every
 *                           page got from the rows, added up
 *   dspark_cache_reset      an empty cache
 *   dspark_cache_reserve    pages for a round's rows (copy on write)
 *   dspark_cache_commit     keep the accepted rows, release the other pages
 *   dspark_cache_fork       requests take over other requests' caches (beams,
 *                           shared prompts), or let go of their own
 *   dspark_cache_evict      pages of least weight let go, down to a budget
 *   dspark_cache_compact    the pages in use drawn together at the low ids
 *   dspark_cache_copy       the page copies the calls above ask for
 *
 * A round over one layer's pool, in stream order:
 *   dspark_schedule (ell) -> reserve (ell_out) -> copy -> for each layer
 *   append and attention (ell_out) -> dspark_verify (n_acc) -> commit; with a
 * budget of pages, weigh after every layer's attention and evict after commit.
 *
 * The conventions of dspark.h hold (device pointers, 16-byte aligned, owned
 * by the caller; nothing allocated, synchronised or read on the host; safe to
 * capture; host-checkable preconditions first; results do not depend on the
 * order in which anything ran).  Calls that write the same table or pool are
 * ordered by the caller (one stream, or events).
 *
 * Requests and rows.  R requests; len[r] >= 0 tokens of request r are
 * committed; ell[r] in -1 .. gamma says that its rows this time are the
 * ell[r] + 1 tokens at positions len[r] .. len[r] + ell[r] (-1: none; values
 * outside are clamped).  In row arrays they are rows row0[r] .. row0[r] +
 * ell[r], or r (gamma + 1) .. when row0 is NULL.  Other rows of an output
 * are left as they were.
 *
 * Pages.  A pool holds n_pages pages of P tokens for every key/value head;
 * request r's token t is in page table[r][t / P] at t % P.  A table entry
 * outside [0, n_pages) is no page: its tokens are invisible, and rows
 * written there are dropped.  Page layout (E = D / 32; blocks of 16 tokens):
 *   DSPARK_CACHE_BF16   [Hkv][2][P/16]: K blocks [D/8][16 tokens][8 dims],
 *                       V blocks [2][D][8 tokens], bf16
 *   DSPARK_CACHE_FP4    [Hkv] of: K codes [P/16][E][16 tokens][32 dims / 2],
 *                       K scales [P][E] u8 (2^(b - 127); 255: NaN), V codes
 *                       [P/16][2][32][E][8 tokens / 2] (dim e * 32 + i at
 *                       [i][e]), V scales [P] f32.  Two codes a byte, low
 *                       nibble first; a code is e2m1: a sign bit and the
 *                       magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.
 *   DSPARK_CACHE_FP8    [Hkv] of: K codes [P/16][D/16][16 tokens][16 dims], V
 *                       codes [P/16][2][32][E][8 tokens] (dim e * 32 + i at
 *                       [i][e]), K scales [8] u8, V scales [8] u8, one for
 *                       each block of 16 tokens (2^(b - 127); those past P/16
 *                       unused).  A code is e4m3: a sign, four exponent bits
 *                       (bias 7), three of the magnitude; 0x7F and 0xFF are
 *                       NaN, there are no infinities, the largest is 448.
 *
 * 4-bit rounding: codes are the nearest, ties to the even code.  K: a scale
 * 2^e per 32 dims, the smallest that brings them to at most 7 (7 rounds to 6
 * within half of the last step), -126 <= e <= 125; computed in fp64 from the
 * bf16 inputs, so a code does not depend on the order of a sum.  V: one scale
 * per token and head, max|v| / 6 in fp32; codes by exact comparison.  A group
 * with a NaN, or a value at or past 2^128, has a NaN scale.
 *
 * 8-bit rounding: a block's scale for K, and for V, is the smallest 2^e, -117
 * <= e <= 119, that brings what the block holds to at most 448 (larger values
 * are held as 448 2^119); codes are the nearest, ties to the even code,
 * computed in fp64 from the bf16 inputs.  Tokens join a block as they are
 * appended, and the scale only grows: where it does, the codes of the block's
 * committed tokens are rounded again, which is exact but for values below
 * 2^-6 of the scale.  So a token that is appended and rolled back can leave a
 * larger scale behind, up to the next block.  Infinities and NaN are held as
 * NaN and have no part in the scale.
 */
#ifndef DSPARK_CACHE_H
#define DSPARK_CACHE_H

#include "dspark.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device status of dspark_cache_reserve: a request got no pages. */
#define DSPARK_ENOPAGES 7

typedef enum { DSPARK_CACHE_BF16 = 1, DSPARK_CACHE_FP4 = 2, DSPARK_CACHE_FP8 = 4 } dspark_cache_format;

/* Workspace selectors for dspark_cache_workspace_size. */
typedef enum {
  DSPARK_CACHE_WS_ATTENTION = 0,  /* a = Hq, b = Hkv, c = D                   */
  DSPARK_CACHE_WS_RESERVE = 1,    /* a = max_pages, b = n_pages               */
  DSPARK_CACHE_WS_FORK = 2,       /* a = max_pages, b = n_pages               */
  DSPARK_CACHE_WS_COMPACT = 3     /* a = max_pages, b = n_pages               */
} dspark_cache_ws_kind;

/* Bytes of one page of all heads (a multiple of 16); 0 for an invalid shape.
 * Limits of every call: fmt as above; 1 <= Hkv <= 1024; D in {64, 128, 256};
 * P in {16, 32, 64, 128}. */
size_t dspark_cache_page_bytes(int fmt, int Hkv, int D, int P);

/* Bytes of workspace a call needs; 0 for an invalid shape.  gamma is used by
 * the attention only. */
size_t dspark_cache_workspace_size(dspark_cache_ws_kind kind, int R, int gamma, int a, int b, int c);

/*
 * dspark_cache_append — norms of queries and keys per head, the position
 * rotation in the same pass, and the new rows' K and V into the pages.
 *
 * For a head x of D values of a row at position p:
 *   y = x * (mean(x^2) + eps)^(-1/2) * w          (w NULL: y = x)
 *   (y_a, y_b) <- (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
 * for the rot / 2 pairs i, t = p * freq[i]: a = i, b = i + rot / 2, or with
 * adjacent != 0 a = 2 i, b = 2 i + 1; dims rot .. D - 1 are not rotated.
 * q heads use wq and go to q_out, k heads wk; v is stored as it is.  Angles
 * are fp64 (reduced to a turn before the fp32 sine and cosine), the rest
 * fp32 (the norm of a head in fp64 where its squares leave fp32's range),
 * rounded once; keys of 4-bit and 8-bit pages are fp64 throughout.
 *
 *   q      bf16, row i at q + i * ldq: [Hq][D]; ldq >= Hq * D; likewise k, v
 *          with [Hkv][D] (views of one fused projection are fine); ldq, ldk
 *          and ldv multiples of 8
 *   wq, wk [D] bf16 or NULL
 *   freq   [rot / 2] f64, radians per position; rot even, 0 .. D, with
 *          adjacent == 0 a multiple of 16 (NULL allowed when rot = 0)
 *   row0 [R] i32 or NULL, ell [R] i32, len [R] i32, table [R][max_pages] i32
 *   q_out  [rows][Hq][D] bf16 out
 *   pool   out: pages of format fmt
 *
 * Limits: 1 <= R <= 4096, 0 <= gamma <= 1023, 1 <= Hq <= 1024, 1 <= n_pages
 * <= 2^20, 1 <= max_pages <= 2^20, R * max_pages < 2^31, len[r] <= 2^29 (past
 * every table: 2^20 pages of 128 tokens).  Two rows never fall on one token
 * unless two requests' tables name one page for it: reserve sees to that.
 */
dspark_status dspark_cache_append(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages,
                                  int max_pages, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                  const void* v, int64_t ldv, const void* wq, const void* wk, float eps,
                                  const double* freq, int rot, int adjacent, const int32_t* row0,
                                  const int32_t* ell, const int32_t* len, const int32_t* table, void* q_out,
                                  void* pool, void* stream);

/*
 * dspark_cache_attention — grouped-head attention of the new rows over the
 * cache, with what append has just written in it.
 *
 * The row of request r at position p sees token j iff j <= p, j's page
 * exists, and (window == 0, or j > p - window, or j < sinks).  With
 * s_j = scale * q . k_j over the visible tokens,
 *   out = sum_j exp(s_j) v_j / sum_j exp(s_j),  lse = ln sum_j exp(s_j);
 * a row that sees nothing gives out = 0 and lse = -inf.  Query head h reads
 * key/value head h / (Hq / Hkv).  What an invisible token holds, infinities
 * and NaN too, has no effect.  Scores, maxima and sums are fp32; the weights
 * exp(s_j - m), m at most 8 ln 2 above the running maximum and never below it,
 * are carried as two bf16 numbers each (2^-15 of a weight is lost) into the
 * product with v, 4-bit V with its token's scale multiplied into the weight
 * first; the output is rounded once.  Weights are at most 1: out is finite
 * where the scores are and the visible tokens' |v| of a dim (4 bits: of a
 * head's largest) add up to less than 2^127.  How the tokens are cut into
 * parts follows from the whole batch, so a row's last bits do too; the same
 * call gives the same bits.
 *
 *   q    [rows][Hq][D] bf16 (q_out of append); out [rows][Hq][D] bf16 out
 *   lse  [rows][Hq] f32 out, or NULL
 *   window >= 0, sinks >= 0 (ignored without a window)
 *   ws   dspark_cache_workspace_size(DSPARK_CACHE_WS_ATTENTION, R, gamma, Hq,
 *        Hkv, D) bytes, 16-byte aligned; contents on entry are irrelevant
 *
 * Limits: as append; Hq a multiple of Hkv; |scale| <= 2^126.
 */
dspark_status dspark_cache_attention(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages,
                                     int max_pages, const void* q, float scale, int window, int sinks,
                                     const int32_t* row0, const int32_t* ell, const int32_t* len,
                                     const int32_t* table, const void* pool, void* out, float* lse, void* ws,
                                     size_t ws_bytes, void* stream);

/*
 * dspark_cache_read — cached tokens as dense bf16 rows (to move a request to
 * another pool or format, or to look at a 4-bit cache).
 *
 * Token start[r] + i, i < min(count[r], T), goes to k[r][i] and v[r][i]
 * ([Hkv][D]); other rows are left as they were, tokens without a page read as
 * zero.  8-bit values are exact in bf16, 4-bit values for K, and rounded once
 * for V.
 *
 *   start NULL: 0.  Limits: as append; 1 <= T <= 2^26.
 */
dspark_status dspark_cache_read(int fmt, int R, int T, int Hkv, int D, int P, int n_pages, int max_pages,
                                const int32_t* start, const int32_t* count, const int32_t* table, const void* pool,
                                void* k, void* v, void* stream);

/*
 * dspark_cache_weigh — how much attention every page gets: for a request with
 * rows, for each entry s of its table,
 *   mass[r][s] <- keep * mass[r][s] + sum exp(scale * q . k_j - lse)
 * over the rows, the query heads and the tokens j of page s that the row sees
 * (dspark_cache_attention's rule and its lse).  Requests without rows are left
 * as they were.  Every row and head shares out 1 over the pages it sees.  Drafts
 * count whether they are accepted or not; called with n_acc in the place of ell,
 * before commit, only the rows that stay do.
 * The layers of a model share a table, so a round calls it once per layer with
 * one mass: keep < 1 (older rounds fade) for the first, 1 for the others.
 * The entries of rejected drafts are weighed like the others, and no other call
 * but dspark_cache_evict writes mass: after dspark_cache_commit the caller sets
 * it to 0 where the table has no page, or a later page of that entry would start
 * with what the released one got, and after dspark_cache_fork it moves rows of
 * mass as the call moved rows of the table.
 *
 * Scores and sums are fp32, the sum in an order that follows from the batch
 * (the same call gives the same bits).  What an invisible token holds has no
 * effect; a row that sees nothing (lse -inf) adds nothing; a NaN among the
 * visible keys, in q or in lse makes the page's mass NaN, which it stays until
 * a call with keep = 0: that takes the old mass for 0 whatever it is.
 *
 *   q, scale, window, sinks, row0, ell, len, table, pool  as in
 *        dspark_cache_attention (values are not read)
 *   lse  [rows][Hq] f32, dspark_cache_attention's
 *   keep finite and >= 0
 *   mass [R][max_pages] f32 in/out (with keep = 0 out, but for requests without rows)
 *
 * Limits: as dspark_cache_attention.
 */
dspark_status dspark_cache_weigh(int fmt, int R, int gamma, int Hq, int Hkv, int D, int P, int n_pages,
                                 int max_pages, const void* q, float scale, int window, int sinks,
                                 const float* lse, const int32_t* row0, const int32_t* ell, const int32_t* len,
                                 const int32_t* table, const void* pool, float keep, float* mass, void* stream);

/*
 * Ownership of the pages.  Per pool (the layers of a model share it):
 *   table [R][max_pages] i32   page ids, -1 = none, -2 = evicted
 *   len   [R] i32              committed tokens
 *   ref   [n_pages] i32        table entries that name the page
 *   bits  [ceil(n_pages / 32)] u32, bit p % 32 of word p / 32 set iff ref[p]
 *         is 0 (bits past n_pages are 0)
 * The calls keep these consistent; they are in/out arguments of all of them.
 * New pages are always the lowest free ids, in request order.
 * Limits: 1 <= R <= 4096, n_pages <= 2^20, R * max_pages < 2^31.
 */

/* Every table entry -1, every len and ref 0, every page free. */
dspark_status dspark_cache_reset(int R, int n_pages, int max_pages, int32_t* table, int32_t* len, int32_t* ref,
                                 uint32_t* bits, void* stream);

/*
 * dspark_cache_reserve — pages for rows len[r] .. len[r] + ell[r].
 *
 * Entries that are no page get new pages.  If the page that holds token
 * len[r] - 1 is also to be written (len[r] % P != 0) and other requests hold it
 * too, r gets a copy of it instead: pairs gets (old, new), and the old page
 * loses a reference; of several such requests of one call the last keeps the
 * old page if nobody else holds it.  ell_out[r] = ell[r], or -1 for a request that was
 * refused: its rows would pass max_pages, or the free pages were used up by
 * the requests before it (then every later request that needs pages, or whose
 * page an earlier one should have left, is refused too); nothing of a refused
 * request changes.
 *
 *   ell_out [R] i32 out; pairs [R][2] i32 out (the first n_pairs);
 *   n_pairs [1] i32 out; status [1] i32 out or NULL: DSPARK_OK, or
 *   DSPARK_ENOPAGES if a request was refused
 *   ws      DSPARK_CACHE_WS_RESERVE bytes, 16-byte aligned
 * ell_out may be ell.
 */
dspark_status dspark_cache_reserve(int R, int gamma, int P, int n_pages, int max_pages, const int32_t* ell,
                                   const int32_t* len, int32_t* table, int32_t* ref, uint32_t* bits,
                                   int32_t* ell_out, int32_t* pairs, int32_t* n_pairs, int32_t* status, void* ws,
                                   size_t ws_bytes, void* stream);

/*
 * dspark_cache_commit — after verification: len[r] += min(n_acc[r], ell[r]) + 1
 * for every r with ell[r] >= 0 (negative n_acc count as 0; len stops at
 * max_pages P), and the pages past the new end are released.  With window > 0
 * so are the pages that no later row can see: those with every token at or
 * before len[r] - window, from the first page that begins at or past `sinks`.
 * Requests with ell[r] < 0 are left alone.
 */
dspark_status dspark_cache_commit(int R, int gamma, int P, int n_pages, int max_pages, int window, int sinks,
                                  const int32_t* ell, const int32_t* n_acc, int32_t* len, int32_t* table,
                                  int32_t* ref, uint32_t* bits, void* stream);

/*
 * dspark_cache_fork — every request r takes over what request from[r] had
 * before the call: its committed tokens and their pages, shared.  from[r] = r
 * leaves r alone, -1 empties it; values outside [-1, R) leave it alone.  Any
 * map is allowed (a permutation, one source for many, chains): all sources
 * are read as they were.
 *
 *   from [R] i32; ws DSPARK_CACHE_WS_FORK bytes, 16-byte aligned
 */
dspark_status dspark_cache_fork(int R, int P, int n_pages, int max_pages, const int32_t* from, int32_t* len,
                                int32_t* table, int32_t* ref, uint32_t* bits, void* ws, size_t ws_bytes,
                                void* stream);

/*
 * dspark_cache_evict — request r keeps at most budget[r] pages of committed
 * tokens: while it has more, the page of least mass among those it may lose is
 * let go (ties: the lower entry; NaN counts as the largest), its entry becomes
 * -2 and its mass 0.  It may lose a page whose tokens are all at or past
 * `sinks` and before len[r] - recent; if these are too few, all of them go.
 * A page that other requests hold stays theirs.  budget[r] < 0 leaves r alone.
 * No page may be reserved and not committed.
 *
 *   mass [R][max_pages] f32 in/out (dspark_cache_weigh's, or any ranking)
 *   budget [R] i32; freed [R] i32 out or NULL: how many pages r lost
 *
 * Limits: sinks >= 0, recent >= 0.
 */
dspark_status dspark_cache_evict(int R, int P, int n_pages, int max_pages, int sinks, int recent,
                                 const int32_t* budget, const int32_t* len, float* mass, int32_t* table,
                                 int32_t* ref, uint32_t* bits, int32_t* freed, void* stream);

/*
 * dspark_cache_compact — moves pages so that the U pages in use are 0 .. U-1:
 * the k-th page in use at or past U goes to the k-th free id below U.  The
 * table, ref and bits say so at once; pairs (old, new) tell
 * dspark_cache_copy what to move before the cache is used again.
 *
 *   pairs [n_pages / 2][2] i32 out (the first n_pairs), n_pairs [1] i32 out
 *   ws    DSPARK_CACHE_WS_COMPACT bytes, 16-byte aligned
 */
dspark_status dspark_cache_compact(int R, int n_pages, int max_pages, int32_t* table, int32_t* ref, uint32_t* bits,
                                   int32_t* pairs, int32_t* n_pairs, void* ws, size_t ws_bytes, void* stream);

/*
 * dspark_cache_copy — page pairs[i][0] to page pairs[i][1], i < min(*n_pairs,
 * max_pairs), in each of `layers` pools, layer_bytes apart.  No page may be
 * the target of two pairs or both source and target (reserve and compact see
 * to that); a pair with an id outside [0, n_pages) is skipped.
 *
 * Limits: page_bytes and layer_bytes multiples of 16, layer_bytes >= n_pages *
 * page_bytes when layers > 1; 1 <= max_pairs <= 2^20.
 */
dspark_status dspark_cache_copy(int layers, int64_t layer_bytes, int64_t page_bytes, int n_pages,
                                const int32_t* pairs, const int32_t* n_pairs, int max_pairs, void* pool,
                                void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_CACHE_H */
