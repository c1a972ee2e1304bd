/*
 * gdr.h -- the gated delta rule of libwkv7, on AMD Instinct MI355X (gfx950).
 *
 * THE OPERATION.  Per batch row b and value head h the library carries a K x V
 * fp32 state S, row i a key channel and column j a value channel (as the WKV-7
 * state in wkv7.h).  Groups of H / Hk value heads share one query / key head,
 * kh = h / (H / Hk).  For each token t, with alpha = exp(g_t):
 *
 *     R[j]    = v_t[j] - alpha * sum_i k_t[i] * S[i][j]     (the residual)
 *     S[i][j] = alpha * S[i][j] + beta_t * k_t[i] * R[j]
 *     o_t[j]  = scale * sum_i q_t[i] * S[i][j]              (state after the step)
 *
 * i.e. S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T and
 * o_t = scale S_t^T q_t.  It is the WKV-7 recurrence with one decay per head and
 * the erased direction tied to the key (w = alpha, a = -alpha beta k, b = k), for
 * wider heads and shared keys.  q and k are taken as given: a caller whose model
 * normalises them does so before.
 *
 * LAYOUTS (row-major, contiguous, no padding):
 *   q, k                : [B, T, Hk, K]     of in_dtype
 *   v                   : [B, T, H, V]      of in_dtype
 *   g, beta             : [B, T, H]         fp32; g is the LOG of the decay
 *                         (-inf: the state before the token is dropped)
 *   o                   : [B, T, H, V]      of o_dtype
 *   state_in, state_out : [B, H, K, V]      fp32
 *   state_pos           : [B, T, H, K, V]   fp32, [b,t,h] = S after token t
 *   ckpt, work          : [B, ceil(T/64), H, K*V] fp32, opaque
 * K is 64 or 128; V is a multiple of 64 up to GDR_MAX_V; Hk divides H.
 * in_dtype and o_dtype are WKV7_F32 or WKV7_BF16.
 *
 * Memory, asynchrony, status codes and aliasing are those of wkv7.h: device
 * pointers on the current HIP device, 16-byte aligned (lengths: 4), owned by the
 * caller; calls enqueue on `stream` and return; state_out may equal state_in
 * exactly, and any other overlap of an output with another buffer is refused.
 *
 * wkv7_state_commit and wkv7_state_reset serve these states too: a K x V state is
 * K V / 4096 consecutive blocks of 64 x 64 floats, so pass H * K * V / 4096 as
 * their H (and 64 as N).
 *
 * NUMERICS.  The state and every accumulation are fp32.  Results match
 * an fp64 evaluation to a relative L2 error below 1e-6 (plus the rounding of a bf16 o)
 * for g <= 0; where positive g make the state grow, a few times that.
 * Value channels stay independent: a NaN or Inf in v[b,t,h,j] reaches only column j of
 * that head, from token t on, except that gdr_forward forms the outputs of 32 tokens
 * together, so there it can also reach the earlier tokens of the same 32-token chunk.
 */
#ifndef GDR_H
#define GDR_H

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits (WKV7_ERR_SHAPE beyond them): V <= GDR_MAX_V; T <= GDR_MAX_T; H * K and H * V <= GDR_MAX_ROW (the rows
 * of 64 tokens are addressed with 32-bit offsets from the first); B * H * V <= GDR_MAX_COLUMNS and
 * B * ceil(T/64) * H <= GDR_MAX_BLOCKS (a launch holds fewer than 2^32 threads; the latter
 * for the training pair).  Tensor offsets are 64-bit. */
#define GDR_MAX_V 512
#define GDR_MAX_ROW 8388608
#define GDR_MAX_T 1073741824
#define GDR_MAX_BLOCKS 8000000
#define GDR_MAX_COLUMNS 268435456

/*
 * gdr_forward -- the parallel (prefill) pass over T tokens.
 *
 *   state_in : fp32 state entering token 0; NULL = all zeros.
 *   lengths  : [B] int32 on the device, or NULL (every row runs T tokens).  Row b
 *              runs its first L_b = lengths[b] tokens, clamped to [0, T]: o[b, t]
 *              for t >= L_b is left untouched, the inputs behind are not used, and
 *              state_out[b] is the state after L_b tokens.  May not overlap o or
 *              state_out.
 *   scale    : multiplies o.
 * T = 0 copies state_in to state_out (zeros if NULL).
 */
int gdr_forward(const void *q, const void *k, const void *v, const float *g, const float *beta, int in_dtype,
                const float *state_in, void *o, int o_dtype, float *state_out, const int *lengths, float scale,
                int B, int T, int Hk, int H, int K, int V, void *stream);

/*
 * gdr_step -- the recurrent (decode / speculative-verify) pass, token by token.
 *
 *   state_pos : [B,T,H,K,V] fp32 or NULL; [b,t,h] = the state after token t.  With
 *               it given and T > 0, state_out may be NULL.
 * Everything else as gdr_forward.  Meant for small T, correct for any T >= 0.
 */
int gdr_step(const void *q, const void *k, const void *v, const float *g, const float *beta, int in_dtype,
             const float *state_in, void *o, int o_dtype, float *state_out, float *state_pos, float scale,
             int B, int T, int Hk, int H, int K, int V, void *stream);

/*
 * gdr_forward_ckpt -- the forward pass of training: gdr_forward (fp32 o, every row T
 * tokens) that also keeps what gdr_backward_ckpt reads.
 *
 *   ckpt  : the state entering every 64 tokens, [B, ceil(T/64), H, K*V] fp32.
 *   resid : the residuals R of every token, [B, T, H, V] fp32.
 * Both may be NULL only when T = 0.
 */
int gdr_forward_ckpt(const void *q, const void *k, const void *v, const float *g, const float *beta, int in_dtype,
                     const float *state_in, float *o, float *state_out, float *ckpt, float *resid, float scale,
                     int B, int T, int Hk, int H, int K, int V, void *stream);

/*
 * gdr_backward_ckpt -- the gradients, given what gdr_forward_ckpt kept from the same
 * inputs.  For a loss L with dL/do = d_o and dL/dS_T = d_state_out:
 *
 *   d_o         : [B,T,H,V] fp32.
 *   d_state_out : [B,H,K,V] fp32, or NULL (zeros).
 *   dq, dk      : [B,T,Hk,K] fp32, summed over the value heads of a group in a fixed
 *                 order (no atomics: the same call gives the same bits).
 *   dv          : [B,T,H,V] fp32.     dg, dbeta : [B,T,H] fp32.
 *   d_state_in  : [B,H,K,V] fp32; may equal d_state_out.
 *   work        : scratch of ckpt's size; what it holds afterwards is unspecified.
 * v itself is not read (resid stands for it).  With T = 0 only d_state_in is written.
 */
int gdr_backward_ckpt(const void *q, const void *k, const float *g, const float *beta, int in_dtype,
                      const float *ckpt, const float *resid, const float *d_o, const float *d_state_out,
                      float *dq, float *dk, float *dv, float *dg, float *dbeta, float *d_state_in, float *work,
                      float scale, int B, int T, int Hk, int H, int K, int V, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H */
