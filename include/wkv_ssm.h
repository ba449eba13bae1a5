/*
 * wkv_ssm.h -- C ABI of the state-space operators of libwkv_b200.so: the short
 * causal convolution, the per-head norm with position rotation, and the
 * selective scan, each with its backward pass and its serving forms (packed
 * variable-length slots, one token per slot). wkv.h gives the conventions
 * that hold here too (memory, layout, alignment, sizes, dtype, C granularity,
 * streams, errors, threads); the status, dtype and device-error codes are
 * those of wkv.h, and failures are read with wkv_last_error() and
 * wkv_device_error(). Outputs must not overlap inputs unless stated. The
 * current device must be the tensors' device; C is at most 2^26.
 */
#ifndef WKV_B200_SSM_H
#define WKV_B200_SSM_H

#include <stddef.h>
#include <stdint.h>

#include "wkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Steps between two scan state checkpoints (see wkv_scan_forward). */
#define WKV_SCAN_CKPT_LEN 16

/* ------------------------------------------------------------------------ */
/* Short causal convolution                                                  */
/* ------------------------------------------------------------------------ */

/*
 * Depthwise causal convolution over the last W tokens, the W-tap relative of
 * wkv4_time_shift_mix:
 *
 *     pre_t[c] = bias[c] + sum_{j<W} weight[j][c] * x_{t-W+1+j}[c]
 *     y_t[c]   = silu(pre_t[c]) = pre_t[c] * sigmoid(pre_t[c]),  or pre_t[c]
 *
 *   W           number of taps, 2..4 (else WKV_ERR_UNSUPPORTED);
 *               weight[W-1] meets the current token.
 *   silu        nonzero: apply silu; zero: y = pre.
 *   x, y        [B][T][C] of `dtype`.
 *   weight      [W][C] float32.      bias  [C] float32 or NULL (zero).
 *   x_prev      [B][W-1][C] of `dtype` or NULL (zeros): the tokens before x,
 *               oldest first.
 * One float32 multiply-add chain per output, rounded once at the end, so a
 * sequence cut in pieces (the last W-1 tokens passed on as x_prev) gives the
 * same bits as one call.
 */
wkv_status wkv_conv_forward(int64_t B, int64_t T, int64_t C, int dtype, int64_t W, int silu,
                            const void *x, const float *weight, const float *bias, const void *x_prev,
                            void *y, void *stream);

/* Bytes of device workspace wkv_conv_backward needs. */
size_t wkv_conv_backward_workspace_bytes(int64_t B, int64_t T, int64_t C, int dtype, int64_t W);

/*
 * Gradients of L = sum(gy * y) for y = wkv_conv_forward(...), with
 * gpre = gy * d(y)/d(pre) (the pre-activations are recomputed):
 *   gx          [B][T][C] of `dtype`: sum_j weight[j] gpre_{t+W-1-j}.
 *   gweight     [W][C] float32: sum over b, t of gpre_t x_{t-W+1+j}.
 *   gbias       [C] float32 or NULL; if given, written: sum of gpre_t.
 *   gx_prev     [B][W-1][C] of `dtype` or NULL; if given, written.
 *   workspace   at least wkv_conv_backward_workspace_bytes(...) bytes,
 *               16-byte aligned; its contents on entry are ignored.
 * Parameter sums are taken in a fixed order (run-to-run deterministic), in
 * float32 over at most 256 tokens and in float64 beyond.
 */
wkv_status wkv_conv_backward(int64_t B, int64_t T, int64_t C, int dtype, int64_t W, int silu,
                             const void *x, const float *weight, const float *bias, const void *x_prev,
                             const void *gy, void *gx, float *gweight, float *gbias, void *gx_prev,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * The convolution over S slots of packed tokens (slots as in wkv4_chunk_step).
 *   x, y        [n_tokens][C] of `dtype`, all slots back to back.
 *   cu_tokens   DEVICE int32 [S+1], as for wkv4_chunk_step: an empty slot is
 *               skipped; one whose range is decreasing or outside n_tokens is
 *               skipped too and WKV_DEVERR_BAD_SLOT is recorded. Rows of y
 *               that no slot covers are not written.
 *   state       [S][W-1][C] of `dtype`, read and written in place: the last
 *               W-1 tokens of each slot, oldest first (zeros to begin with).
 * Gives the same bits as wkv_conv_forward on the same tokens. The launch is
 * sized for the mean length; one slot far longer than the others takes as long
 * as few CTAs need for it (wkv_conv_forward with x_prev does it at once).
 */
wkv_status wkv_conv_chunk_step(int64_t S, int64_t C, int dtype, int64_t W, int silu,
                               const void *x, const float *weight, const float *bias,
                               void *y, int64_t n_tokens, const int32_t *cu_tokens, void *state,
                               void *stream);

/* One token for every slot: x, y [S][C]; the same bits as wkv_conv_chunk_step
 * with cu_tokens = {0, 1, ..., S}. */
wkv_status wkv_conv_decode_step(int64_t S, int64_t C, int dtype, int64_t W, int silu,
                                const void *x, const float *weight, const float *bias,
                                void *y, void *state, void *stream);

/* ------------------------------------------------------------------------ */
/* Per-head norm with position rotation                                      */
/* ------------------------------------------------------------------------ */

/*
 * Root-mean-square norm of every head of the queries and of the keys, and the
 * rotation by position, in one pass: the prologue of the head-state
 * recurrences (r and k of wkv6_forward and wkv7_forward; C and B of
 * wkv_scan_forward, whose groups are the heads). Per token and head, with
 * v = x / sqrt(mean(x^2) + eps) * weight, the first R entries of v are turned
 * in pairs by the angle p * inv_freq[i], i < R/2, p the token's position:
 *
 *     (v_a, v_b) -> (v_a cos - v_b sin, v_a sin + v_b cos),
 *     (a, b) = (i, i + R/2), or (2i, 2i + 1) if interleaved.
 *
 * (weight = 1/sqrt(K) with eps divided by K gives the Euclidean norm.)
 *   Hq, Hk      heads of q and of k; either may be 0 (its pointers are then
 *               not read).
 *   K           head size, a multiple of 8, 8..256 (else UNSUPPORTED).
 *   R           rotated entries of each head, 0..K: a multiple of 16, or of
 *               2 if interleaved (else UNSUPPORTED). R = 0: norm only.
 *   q, k        [B][T][Hq*K], [B][T][Hk*K] of `dtype`.
 *   q_weight, k_weight  [K] float32 or NULL (ones).
 *   eps         >= 0.
 *   inv_freq    [R/2] float32, required if R > 0.
 *   positions   DEVICE int32 [B][T] or NULL: p = pos_offset + t, which must
 *               stay within 2^53 either way if R > 0 (else UNSUPPORTED). With
 *               positions pos_offset is not read.
 *   q_out, k_out  like q and k; q_out = q and k_out = k (in place) is allowed.
 * Angles are reduced in two parts of 64 bits, so that no position loses
 * anything (up to angles of 2^65); the rest is float32, rounded once at the
 * end. The mean of squares must fit float32: entries above 1e18 overflow it,
 * and with eps = 0 a head below 1e-19 is lost to it. A single token of S slots
 * is B = S, T = 1 with one position per slot.
 */
wkv_status wkv_norm_rotate(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t K, int64_t R, int dtype,
                           const void *q, const void *k, const float *q_weight, const float *k_weight,
                           float eps, const float *inv_freq, const int32_t *positions, int64_t pos_offset,
                           int interleaved, void *q_out, void *k_out, void *stream);

/* Bytes of device workspace wkv_norm_rotate_backward needs. */
size_t wkv_norm_rotate_backward_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t K);

/*
 * Gradients of L = sum(gq_out * q_out) + sum(gk_out * k_out) for
 * wkv_norm_rotate with the same arguments:
 *   gq, gk      like q and k, written; gq = gq_out and gk = gk_out (in place)
 *               is allowed.
 *   gq_weight, gk_weight  [K] float32 or NULL; if given, written: summed over
 *               tokens and heads in a fixed order (deterministic), in float32
 *               over about 256 heads and in float64 beyond.
 *   workspace   at least wkv_norm_rotate_backward_workspace_bytes(...) bytes,
 *               16-byte aligned; its contents on entry are ignored.
 */
wkv_status wkv_norm_rotate_backward(int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t K, int64_t R, int dtype,
                                    const void *q, const void *k, const void *gq_out, const void *gk_out,
                                    const float *q_weight, const float *k_weight, float eps,
                                    const float *inv_freq, const int32_t *positions, int64_t pos_offset,
                                    int interleaved, void *gq, void *gk, float *gq_weight, float *gk_weight,
                                    void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------ */
/* Selective scan                                                            */
/* ------------------------------------------------------------------------ */

/*
 * Selective state-space scan. Every channel c carries a state h[c][n] of N
 * float32 numbers; the step size dt and the vectors B, C come with the token
 * (G groups of channels share B and C: channel c belongs to group
 * c / (C/G)). With d_t = dt_t + dt_bias, put through softplus if dt_softplus:
 *
 *     h_t[c][n] = e^{d_t[c] A[c][n]} h_{t-1}[c][n] + d_t[c] x_t[c] B_t[g][n]
 *     s_t[c]    = sum_n C_t[g][n] h_t[c][n] + D[c] x_t[c]
 *     y_t[c]    = s_t[c] * silu(z_t[c])          (s_t[c] if z is NULL)
 *
 *   N           state size, a multiple of 4, 4..64 (else UNSUPPORTED). It is
 *               worked on as 8, 16, 32 or 64, whichever holds it.
 *   G           groups, >= 1; C/G must be whole and follow the C granularity.
 *   x, dt, z, y [B][T][C] of `dtype` (z may be NULL).
 *   A           [C][N] float32 (negative for a decay).
 *   Bm, Cm      [B][T][G*N] of `dtype`.
 *   D, dt_bias  [C] float32 or NULL (zero).
 *   init_state  [B][C][N] float32 or NULL (zero).
 *   final_state NULL or [B][C][N] float32, written: h after the last token.
 *               final_state = init_state (in place) is allowed.
 *   ckpt        NULL or [B][ceil(T/WKV_SCAN_CKPT_LEN)][C][N] float32, written:
 *               entry [b][m] is h before token m * WKV_SCAN_CKPT_LEN.
 *               wkv_scan_backward reads it.
 *   y may be NULL if ckpt or final_state is given.
 *   workspace   at least wkv_scan_forward_workspace_bytes(...) bytes (NULL
 *               where that is 0), 16-byte aligned.
 * A batch with too few channels to fill the GPU is cut along T: a first
 * kernel finds what each piece does to a state (in the workspace), a second
 * runs all pieces at once. The cut depends on B, T, C, N and G alone.
 * An infinity reaches the y and the states that the formulas say, and no others.
 */
wkv_status wkv_scan_forward(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G, int dtype,
                            const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                            const float *D, const void *z, const float *dt_bias, int dt_softplus,
                            const float *init_state, void *y, float *final_state, float *ckpt,
                            void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of device workspace wkv_scan_forward needs (0 for an uncut launch). */
size_t wkv_scan_forward_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G);

/* Number of floats of the checkpoint buffer. */
size_t wkv_scan_ckpt_floats(int64_t B, int64_t T, int64_t C, int64_t N);

/* Bytes of device workspace wkv_scan_backward needs (has_ckpt: ckpt != NULL). */
size_t wkv_scan_backward_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G, int has_ckpt);

/*
 * Gradients of L = sum(gy * y) + sum(g_final * final_state) for
 * wkv_scan_forward with the same arguments. With gs = gy silu(z) (gy without
 * z), a_t = e^{d_t A} and Q_t = dL/dh_t walked down,
 *     Q_t = gs_t C_t + a_{t+1} Q_{t+1}:
 *   gx, gdt     [B][T][C] of `dtype`: d_t sum_n Q B + gs D, and
 *               (x sum_n Q B + sum_n A Q a h_{t-1}) times the softplus's
 *               derivative.
 *   gz          [B][T][C] of `dtype`, required if z is given: gy s silu'(z).
 *   gB, gC      [B][T][G*N] of `dtype`: sums over the group's channels of
 *               Q d x and of gs h.
 *   gA          [C][N] float32: sum over b, t of d Q a h_{t-1}.
 *   gD, gdt_bias  [C] float32 or NULL; if given, written.
 *   g_final     [B][C][N] float32 or NULL (zero).
 *   g_init      [B][C][N] float32 or NULL; if given, written: dL/dh_{-1}.
 *   ckpt        the checkpoints wkv_scan_forward wrote for the same inputs,
 *               or NULL (then they are regenerated inside `workspace`).
 *   workspace   at least wkv_scan_backward_workspace_bytes(...) bytes,
 *               16-byte aligned; its contents on entry are ignored.
 * All sums are taken in a fixed order (run-to-run deterministic); those of the
 * parameters in float32 over at most 256 tokens and in float64 beyond. Like
 * the forward, a launch may be cut along T, here also for its last sequences
 * alone: equal sequences of one batch may then differ in the last bits. The
 * cut depends on B, T, C, N and G.
 * Most of the workspace holds gB and gC of every CTA: 8 G N bytes per token for
 * each of a group's CTAs (of 64, 32, 32, 16 channels for N up to 8, 16, 32,
 * 64), i.e. 1, 4, 8 and 32 bytes per token and channel.
 * Where a state, B or C is infinite, a gradient that the formulas make infinite
 * may be NaN.
 */
wkv_status wkv_scan_backward(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G, int dtype,
                             const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                             const float *D, const void *z, const float *dt_bias, int dt_softplus,
                             const float *init_state, const void *gy, const float *g_final, const float *ckpt,
                             void *gx, void *gdt, float *gA, void *gB, void *gC, float *gD, void *gz,
                             float *gdt_bias, float *g_init,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * The scan over S slots of packed tokens (slots as in wkv4_chunk_step).
 *   x, dt, z, y [n_tokens][C], Bm, Cm [n_tokens][G*N] of `dtype`.
 *   cu_tokens   as for wkv_conv_chunk_step.
 *   state       [S][C][N] float32, read and written in place (zeros to begin
 *               with).
 * Feeding a slot's tokens in several calls gives the same bits as one call,
 * and as wkv_scan_forward where that is not cut along T. A slot never is, so a
 * long one takes as long as its walk: for few long prompts wkv_scan_forward with
 * init_state and final_state is faster (8,192 tokens, C=1536 N=16 bf16: 162
 * against 555 us).
 */
wkv_status wkv_scan_chunk_step(int64_t S, int64_t C, int64_t N, int64_t G, int dtype,
                               const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                               const float *D, const void *z, const float *dt_bias, int dt_softplus,
                               void *y, int64_t n_tokens, const int32_t *cu_tokens, float *state,
                               void *stream);

/* One token for every slot: x, dt, z, y [S][C], Bm, Cm [S][G*N]; the same
 * bits as wkv_scan_chunk_step with cu_tokens = {0, 1, ..., S}. */
wkv_status wkv_scan_decode_step(int64_t S, int64_t C, int64_t N, int64_t G, int dtype,
                                const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                                const float *D, const void *z, const float *dt_bias, int dt_softplus,
                                void *y, float *state, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* WKV_B200_SSM_H */
