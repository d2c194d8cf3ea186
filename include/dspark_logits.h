/*
 * dspark_logits.h — conditions on the target's logits in a verification round.
 *
 * Between the target's forward pass and dspark_verify (caijizhuo section 四,
 * steps 5 and 6) the rows of a request get what the user asked for: penalties
 * for tokens that are there already, biases, and the tokens that a grammar
 * allows.  Row i of request r follows its history, the anchor x0 and the
 * drafts x_1 .. x_i, so the rows of one round differ in what they penalise.
 * Verified against such rows, the round's tokens are distributed as if they had
 * been drawn from them one at a time (notes, lossless verification), and none is
 * one that its row does not allow.
 *
 *   dspark_logits         the rows' logits with all of it applied
 *   dspark_logits_prompt  a slot's history: a new prompt
 *   dspark_logits_commit  the history after a round
 *
 * The conventions of dspark.h hold (device pointers, 16-byte aligned; nothing
 * allocated, synchronised or read on the host; safe to capture; host-checkable
 * preconditions first).  ell, gamma and row0 as in dspark_cache.h: the rows of
 * request r are row0[r] .. row0[r] + ell[r], or r (gamma + 1) .. when row0 is
 * NULL, none with ell[r] = -1, and values outside -1 .. gamma are clamped.
 *
 * State: [R][V] u16, one word a token: bit 15 says that it is in the prompt,
 * the others how often it was answered with (at most 32767).
 * Limits of every call: 1 <= R <= 4096, 0 <= gamma <= 1023, 2 <= V < 2^24.
 */
#ifndef DSPARK_LOGITS_H
#define DSPARK_LOGITS_H

#include "dspark.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * dspark_logits — for a row that follows token v n times in the answer:
 *   l <- l / repetition if l > 0, else l * repetition   if n > 0 or v is in
 *                                                       the prompt
 *   l <- l - (frequency * n + presence)                 if n > 0
 *   l <- l + bias
 *   l <- -inf                                           if v is not allowed
 * in fp32, rounded once to dt.  Rows of nobody are left as they were.  A row
 * that allows nothing is -inf throughout (dspark_verify then accepts no draft
 * there, and what it draws is any token).
 *
 *   logits   [rows][V] dt;  out [rows][V] dt out (may be logits)
 *   state    [R][V] u16 or NULL (no history: x0 and x are not counted either)
 *   x0       [R] i32, x [R][gamma] i32 or NULL: the anchor and the drafts; a
 *            token outside [0, V) is none.  x NULL: rows follow no drafts.
 *   repetition, presence, frequency  [R] f32 or NULL (1, 0, 0); repetition > 0
 *   nb, bias_tok [R][nb] i32, bias [R][nb] f32: request r's biases; a token
 *            outside [0, V) is none, one that is there twice gets both, in
 *            their order.  nb = 0: none (both ignored).
 *   mask     [rows][ceil(V / 32)] u32 or NULL: bit v % 32 of word v / 32 is
 *            set where the row allows token v
 *
 * Limits: 0 <= nb <= 2^20.
 */
dspark_status dspark_logits(dspark_dtype dt, int R, int gamma, int V, const void* logits, const int32_t* row0,
                            const int32_t* ell, const int32_t* x0, const int32_t* x, const uint16_t* state,
                            const float* repetition, const float* presence, const float* frequency, int nb,
                            const int32_t* bias_tok, const float* bias, const uint32_t* mask, void* out,
                            void* stream);

/*
 * dspark_logits_prompt — slot r's history becomes the prompt tokens[start[r]]
 * .. tokens[start[r] + count[r] - 1], with nothing answered yet; count[r] < 0
 * leaves the slot as it is.  Tokens outside [0, V), and places outside
 * [0, n), are none.
 *
 *   tokens [n] i32; start, count [R] i32; state [R][V] u16 in/out
 *
 * Limits: 0 <= n < 2^31 (n = 0: tokens may be NULL).
 */
dspark_status dspark_logits_prompt(int R, int V, int64_t n, const int32_t* tokens, const int32_t* start,
                                   const int32_t* count, uint16_t* state, void* stream);

/*
 * dspark_logits_commit — after verification the anchor and the accepted drafts
 * join the history: x0[r] and the first min(n_acc[r], ell[r]) tokens of x[r],
 * for every r with ell[r] >= 0 (negative n_acc count as 0, as in
 * dspark_cache_commit).  Counts stop at 32767.
 *
 *   ell, n_acc [R] i32; x0, x as in dspark_logits; state [R][V] u16 in/out
 */
dspark_status dspark_logits_commit(int R, int gamma, int V, const int32_t* ell, const int32_t* n_acc,
                                   const int32_t* x0, const int32_t* x, uint16_t* state, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_LOGITS_H */
