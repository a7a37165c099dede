/*
 * gdn_lin.h -- C ABI of linear attention with a decay for each head (part of
 * libgdn.so; status codes and dtypes from gdn.h, conventions from gdn_layer.h).
 * The recurrence of gdn.h without its delta correction:
 *
 *     S_t = e^{g_t} S_{t-1} + k_t v_t^T   [dk, dv],      o_t = scale S_t^T q_t
 *
 *   gdn_lin_fwd/bwd   whole sequences (prompts, training chunks linked by their
 *                     fp32 boundary state, packed sequences)
 *   gdn_lin_step      token by token over a cache of states (generation,
 *                     verification of drafted tokens)
 *
 * The StateFlow pages name no such layer; the formulas above are the definition.
 *
 * The log-decay is either g, one value for each token and head (of dtype), or
 * decay [H] fp32, one for each head: exactly one of the two is not NULL. It is
 * meant to be <= 0; g = -inf (the state is forgotten) gives factors of 0. Positive
 * values are taken as they are, and overflow where e^g over a sequence does.
 *
 * Sums, states and decay factors are fp32; each chunk (64 tokens of F32, 128 of BF16)
 * that a state passes rounds it by 2^-22 of itself at most. With GDN_DTYPE_F32 products
 * are taken on the tensor cores with each operand as two TF32 parts: operands are held
 * to 2^-23, products good to 2^-21.6 of themselves. With GDN_DTYPE_BF16, where rows lie
 * ld >= H * d apart (others take the fp32 kernels), products of inputs are exact; what
 * a state receives, and a state before it meets a row for dg, is taken as two bf16
 * parts (3 2^-16 of a term's magnitude, so S_out and dS_in are good to that of the sums
 * of magnitudes, and to the chunks' roundings); a masked product (q k^T) L or
 * (dout v^T) L, and the state in o and dv, is rounded to bf16 once before it meets its
 * other factor, as the result itself is.
 *
 * dg_t is the sum over s < t <= u of the tokens' (and states') products
 * scale (q_u . k_s) (dout_u . v_s) times the decay between them. Each is summed for
 * itself: dg_t, and ddecay as the sum of dg, are good to 2^-16 (F32) or 2^-13 (BF16)
 * of the magnitudes of their own terms before they are stored (and to the roundings of
 * the chunks between the tokens), whatever the rest of the sequence holds.
 *
 * Whole sequences work on chunks of 64 (fp32) or 128 (bf16) tokens by products with
 * zeros above the diagonal: a NaN or an infinity in a token reaches the results of
 * its chunk's earlier tokens too, and an infinite operand may come out as NaN. It
 * stays within its sequence.
 */
#ifndef GDN_LIN_H_
#define GDN_LIN_H_

#include <stddef.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ whole sequences
 * q, k [B, T, H, dk], v, o [B, T, H, dv], g [B, T, H]; states [nseq, H, dk, dv]
 * fp32, nseq = B. q, k, v are vector rows (gdn_layer.h) with the strides below
 * between the B * T token rows; g needs its type's alignment; o, dout and the
 * gradients are contiguous and 16-byte aligned.
 * Packed sequences (cu_seqlens, DEVICE int32 [nseq + 1], not NULL): B = 1, sequence
 * s owns rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1, 0 <= cu_seqlens[0] <= .. <=
 * cu_seqlens[nseq] <= T. Rows that belong to no sequence are neither read for
 * another's result nor written. An array that is not so is reported by
 * gdn_workspace_status as GDN_ERR_INVALID_ARG, and of that call's outputs only
 * ddecay is written (zeros). More than 65535 sequences x heads are
 * GDN_ERR_UNSUPPORTED. */
typedef struct {
  int B, T, H;
  int dk, dv;   /* 64 or 128 */
  int dtype;    /* gdn_dtype of q, k, v, g, o and their gradients */
  int nseq;     /* sequences; without cu_seqlens B */
  long long ldq, ldk, ldv, ldg; /* strides of the token rows, in elements */
  float scale;
} gdn_lin_shape;

/* Workspace bytes of gdn_lin_fwd (is_bwd = 0) or gdn_lin_bwd (is_bwd = 1); 0 if the
 * shape is invalid or unsupported. With F32 it holds an fp32 state for every 64
 * tokens of a head (the backward's two), with BF16 the backward's one for every 128.
 * 256-byte aligned; not shared by calls that may
 * run at the same time. A kernel's wait that ran out is reported by
 * gdn_workspace_status as GDN_ERR_TIMEOUT. */
size_t gdn_lin_workspace_bytes(const gdn_lin_shape* shape, int is_bwd);

/* S_in NULL: zero states. S_out NULL: not written; it may be S_in. */
gdn_status gdn_lin_fwd(const gdn_lin_shape* shape, const void* q, const void* k, const void* v,
                       const void* g, const float* decay, const float* S_in,
                       const int* cu_seqlens, void* o, float* S_out, void* workspace,
                       size_t workspace_bytes, void* stream);

/* From dout [B, T, H, dv] and dS_out (NULL: zero): dq, dk, dv, dg (with g) or ddecay [H]
 * (with decay; summed over the tokens in a fixed order), dS_in (NULL: not written; it
 * may be dS_out). With R_t the gradient of S_t:
 *     R_t = e^{g_{t+1}} R_{t+1} + scale q_t dout_t^T      (dS_out behind the last token)
 *     dq_t = scale S_t dout_t,  dk_t = R_t v_t,  dv_t = R_t^T k_t,
 *     dg_t = <R_t, e^{g_t} S_{t-1}>,   dS_in = e^{g_1} R_1. */
gdn_status gdn_lin_bwd(const gdn_lin_shape* shape, const void* q, const void* k, const void* v,
                       const void* g, const float* decay, const float* S_in,
                       const int* cu_seqlens, const void* dout, const float* dS_out, void* dq,
                       void* dk, void* dv, void* dg, float* ddecay, float* dS_in,
                       void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------- token by token
 * The sequences, slots, packed tokens and committed tokens of gdn_step
 * (gdn_layer.h). q, k [n_tok, Hk, dk], v [n_tok, H, dv], g [n_tok, H], rows
 * strided; value head h uses key head h / (H / Hk). S: cache [n_slots, H, dk, dv]
 * fp32, 16-byte aligned, updated in place. o [n_tok, H, dv] contiguous. All
 * arithmetic is fp32 multiply-adds, the same for any number of tokens. */
typedef struct {
  int N;         /* sequences */
  int n_tok;     /* rows of q, k, v, g, o */
  int n_slots;   /* slots of the cache */
  int H;         /* value heads */
  int Hk;        /* key heads, a divisor of H */
  int dk, dv;    /* 64 or 128 */
  int dtype;     /* gdn_dtype of q, k, v, g, o */
  long long ldq, ldk, ldv, ldg;
  float scale;
} gdn_lin_step_shape;

gdn_status gdn_lin_step(const gdn_lin_step_shape* shape, const void* q, const void* k,
                        const void* v, const void* g, const float* decay, float* S,
                        const int* slot_in, const int* slot_out, const int* cu_seqlens,
                        const int* n_commit, void* o, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LIN_H_ */
