/*
 * draft.h -- verification of drafted tokens, of libwkv7, on AMD Instinct MI355X
 * (gfx950).  It stands between the verify step of speculative decoding (wkv7_step or
 * gdr_step with per-position states, run over the last token and its drafts) and
 * wkv7_state_commit, which keeps the states of the accepted prefix.
 *
 * Memory, asynchrony and status codes are those of wkv7.h.
 */
#ifndef DRAFT_H
#define DRAFT_H

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits (WKV7_ERR_SHAPE beyond them). */
#define DRAFT_MAX_ROWS 4000000
#define DRAFT_MAX_DRAFTS 1024
#define DRAFT_MAX_VOCAB 16777216

/*
 * draft_verify -- accept drafted tokens against the target's probabilities and draw
 * the token that follows, from given random numbers.
 *
 *   target   : [B, N+1, vocab] probabilities of dtype (WKV7_F32 | WKV7_BF16):
 *              target[b, j] is the target's distribution for the place of draft j,
 *              target[b, N] the one behind the last.
 *   draft    : [B, N, vocab] the drafter's probabilities, of dtype, or NULL for a
 *              drafter that is sure of its token (all mass on it).
 *   tokens   : [B, N] int32, the drafted tokens.
 *   n_draft  : [B] int32, the drafts of each row (clamped to [0, N]), or NULL (N).
 *   u        : [B, N] fp32 in [0, 1), one number for each acceptance.
 *   u_draw   : [B] fp32 in [0, 1), for the drawn token.
 *   out      : [B, N+1] int32: the accepted drafts, the drawn token, then -1.
 *   kept     : [B] int32: 1 + accepted drafts, the number of tokens in out[b] and of
 *              the verify step's tokens whose states stand, as wkv7_state_commit
 *              takes it.
 *
 * Per row, with p = target, q = draft and x = tokens[b, j]:
 *   - draft j is accepted iff u[j] q_j[x] < p_j[x] (the product in 64 bits, exact);
 *     n is the first draft that is not, or the row's number of drafts.
 *   - the weights are max(p_n - q_n, 0) at a refused draft and p_n behind the last;
 *     where all of the former are 0, p_n stands in for them.
 *   - the drawn token is the lowest with (sum of the weights up to it) > u_draw times
 *     the sum of all, or the last of positive weight if there is none.  The sums are
 *     in 64 bits, in a fixed order (no atomics: the same call gives the same token).
 *     A row without any weight draws -1.
 * A probability that is no positive finite number (NaN, an infinity, below 0) weighs
 * nothing.  A drafted token outside [0, vocab) is refused.
 * N may be 0 (tokens, u and draft may then be NULL): a plain draw from target[b, 0].
 * target, draft: 16-byte aligned; the other pointers 4-byte.  No output may overlap
 * another buffer.
 */
int draft_verify(const void *target, const void *draft, int dtype, const int *tokens, const int *n_draft,
                 const float *u, const float *u_draw, int *out, int *kept, int B, int N, int vocab, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DRAFT_H */
