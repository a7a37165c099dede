/*
 * gdn_layer.h -- C ABI of the operators a Gated DeltaNet layer runs around the
 * chunk transition (part of libgdn.so; status codes and dtypes from gdn.h).
 * The StateFlow pages name the layer but give no formula for these; the
 * formulas are stated below.
 *
 *   gdn_step           the gated delta rule token by token over a cache of
 *                      states (generation, verification of drafted tokens)
 *   gdn_conv_step      the short convolution of gdn_conv.h over a cache of its
 *                      last W - 1 inputs, for the same sequences
 *   gdn_prep_fwd/bwd   the maps before the recurrence: unit-norm q and k
 *                      (key heads shared by several value heads), the
 *                      log-decay and the write strength
 *   gdn_gate_norm_*    RMS norm of each head's output, times its gate
 *   gdn_res_norm_*     block boundary: norm of the block's output, residual
 *                      scale, addition, norm before the next block
 *
 * Conventions
 * -----------
 * - dtype: GDN_DTYPE_F32 or GDN_DTYPE_BF16 of the activations and their
 *   gradients. Parameters (rate, bias, w, ...), their gradients and cached
 *   recurrence states are fp32. Arithmetic, sums and statistics are fp32 (the
 *   products of gdn_step with several tokens: see there); a result is rounded
 *   once, when it is stored.
 * - Row strides (ld*) are in elements. "Vector rows" are rows read or written
 *   16 bytes at a time: their pointer must be 16-byte aligned and their stride
 *   a multiple of 16 bytes. Gate inputs (one value per head) need only their
 *   type's alignment. Tensors without a stride are contiguous.
 * - Outputs must not alias inputs except where it is said that they may.
 * - Counts of rows, sequences and channels that pass what the kernels' 32-bit
 *   indices hold (2^31 - 2^16 of any; gdn_step 2^28 sequences x heads; prep and
 *   the gated norm 2^30 and 2^31 rows x heads) are GDN_ERR_UNSUPPORTED.
 * - Ownership, execution and errors as in gdn.h: caller-owned buffers, work
 *   enqueued on `stream` without synchronising, every argument checked on the
 *   host before any launch, GDN_ERR_CUDA if a launch fails. Calls with nothing
 *   to do (no tokens, no rows) still write their parameter gradients (zeros).
 *   One condition shows on the device only: the CTAs that share a wide row of
 *   gdn_res_norm_* wait for each other's sums, and a wait that runs out (after
 *   about two seconds) leaves NaN in that call's outputs and is reported by
 *   gdn_layer_status.
 * - Parameter gradients are summed in a fixed order: results are the same from
 *   run to run.
 */
#ifndef GDN_LAYER_H_
#define GDN_LAYER_H_

#include <stddef.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* --------------------------------------------------- sequences over a cache
 * gdn_step and gdn_conv_step process N sequences with a few new tokens each.
 * The new tokens of all sequences are packed: sequence s owns rows
 * cu_seqlens[s] .. cu_seqlens[s + 1] - 1 (DEVICE int32 [N + 1]; NULL: one
 * token each, row s, and n_tok = N). Its state before them is cache slot
 * slot_in[s] (DEVICE int32 [N]; a value outside [0, n_slots) means the zero
 * state of a new sequence; NULL: slot s), and the state after its first
 * n_commit[s] tokens (DEVICE int32 [N], clamped to its token count; NULL: all
 * of them) is written to slot_out[s] (DEVICE int32 [N]; a value outside
 * [0, n_slots) means that it is not kept; NULL: slot s). So
 *   - drafted tokens are verified with n_commit = 0 (the slot stays as it is)
 *     and the accepted ones passed again, committed, ahead of the next draft;
 *   - slot_out != slot_in branches a sequence off (with no new tokens the slot
 *     is copied).
 * The cache is read and written in place. A slot written by one sequence must
 * not be read or written by another sequence of the same call. A sequence
 * whose cu_seqlens entries are negative, decreasing or past n_tok is treated
 * as having no tokens; rows that belong to no sequence are not written, and of a
 * row that several claim either's output may be stored. */

typedef struct {
  int N;         /* sequences */
  int n_tok;     /* rows of q, k, v, g, beta, o */
  int n_slots;   /* slots of the cache */
  int H;         /* value heads */
  int Hk;        /* key heads, a divisor of H: value head h uses key head h / (H / Hk) */
  int dk;        /* 64 or 128 */
  int dv;        /* 64, 128 or 256 */
  int dtype;     /* gdn_dtype of q, k, v, g, beta, o */
  long long ldq, ldk, ldv; /* strides of the token rows of q, k [n_tok, Hk, dk], v [n_tok, H, dv] */
  long long ldg, ldb;      /* strides of the token rows of g and beta [n_tok, H] */
  float q_scale; /* with rate: factor of q after its normalisation */
  float eps;     /* with rate: > 0, added to the squared norms */
} gdn_step_shape;

/* For each token, with S [dk, dv] as stored (gdn.h):
 *     S <- alpha (S - beta k (k^T S)) + beta k v^T,   o = S^T q,
 * alpha = e^g. rate and bias NULL: q, k, g, beta are used as they are.
 * Otherwise ([H] fp32 each) they are the inputs of the maps of gdn_prep_fwd,
 * which are applied here. S: cache [n_slots, H, dk, dv] fp32, 16-byte aligned.
 * o [n_tok, H, dv]. q, k, v are vector rows.
 * The tokens of a sequence are taken up to 8 at a time. One token takes fp32
 * multiply-adds. Several take their products on the tensor cores, each fp32
 * operand (the state; with GDN_DTYPE_F32 also q and k) as the sum of two TF32
 * values: an operand is held to 2^-23 of itself, a product is good to 2^-21.6,
 * sums and the state are fp32. The bits of a result thus depend on how many
 * tokens a call passes for its sequence, and an infinite operand may come out as
 * NaN. A token behind the committed ones reaches neither the state nor the
 * outputs before it, whatever it holds. */
gdn_status gdn_step(const gdn_step_shape* shape, const void* q, const void* k, const void* v,
                    const void* g, const void* beta, const float* rate, const float* bias,
                    float* S, const int* slot_in, const int* slot_out, const int* cu_seqlens,
                    const int* n_commit, void* o, void* stream);

typedef struct {
  int N, n_tok, n_slots;
  int C;         /* channels, a multiple of 4 */
  int W;         /* kernel width (2..8) */
  int dtype;     /* gdn_dtype of x, y and the cache */
  int act;       /* GDN_CONV_ACT_NONE or GDN_CONV_ACT_SILU (gdn_conv.h) */
  long long ldx; /* stride of the token rows of x: a multiple of 4 */
} gdn_conv_step_shape;

/* y [n_tok, C] and the cache [n_slots, W - 1, C] of the last inputs, with
 * w [C, W], b [C] (may be NULL) as in gdn_conv.h, 16-byte aligned. x: 4 elements
 * aligned. */
gdn_status gdn_conv_step(const gdn_conv_step_shape* shape, const void* x, const float* w,
                         const float* b, void* state, const int* slot_in, const int* slot_out,
                         const int* cu_seqlens, const int* n_commit, void* y, void* stream);

/* ------------------------------------------------ maps before the recurrence
 *     qn[h] = q_scale q[hk] / sqrt(|q[hk]|^2 + eps),   hk = h / (H / Hk)
 *     kn[h] =         k[hk] / sqrt(|k[hk]|^2 + eps)
 *     g = -exp(rate) softplus(xg + bias),   beta = sigmoid(xb)
 * q, k [rows, Hk, dk] vector rows; xg, xb [rows, H]; rate, bias [H];
 * qn, kn [rows, H, dk] and g, beta [rows, H] contiguous, as gdn_chunk_fwd takes
 * them. rows = B * T tokens. */
typedef struct {
  int rows, H, Hk;
  int dk;        /* 64 or 128 */
  int dtype;
  long long ldq, ldk, ldg, ldb; /* strides of the rows of q, k, xg, xb */
  float q_scale, eps;
} gdn_prep_shape;

gdn_status gdn_prep_fwd(const gdn_prep_shape* shape, const void* q, const void* k, const void* xg,
                        const void* xb, const float* rate, const float* bias, void* qn, void* kn,
                        void* g, void* beta, void* stream);

/* Workspace bytes of gdn_prep_bwd; 0 if the shape is invalid or unsupported. */
size_t gdn_prep_workspace_bytes(const gdn_prep_shape* shape);

/* From dqn, dkn [rows, H, dk] and dg, dbeta [rows, H]: dq, dk [rows, Hk, dk]
 * (summed over the value heads of a key head), dxg, dxb [rows, H],
 * drate, dbias [H] fp32. */
gdn_status gdn_prep_bwd(const gdn_prep_shape* shape, const void* q, const void* k, const void* xg,
                        const void* xb, const float* rate, const float* bias, const void* dqn,
                        const void* dkn, const void* dg, const void* dbeta, void* dq, void* dk,
                        void* dxg, void* dxb, float* drate, float* dbias, void* workspace,
                        size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------- gated norm
 *     y = o / sqrt(mean(o^2) + eps) * w * act(z)      per row of d values
 * o, y, dy, do [rows, H, d] contiguous; z [rows, H, d] with row stride ldz, dz
 * contiguous; w, dw [d] fp32 (one weight for every head). */
#define GDN_GATE_SILU 1
#define GDN_GATE_SIGMOID 2

typedef struct {
  int rows, H;
  int d;         /* multiple of 8, 8..256 */
  int dtype;
  int act;       /* GDN_GATE_SILU or GDN_GATE_SIGMOID */
  long long ldz; /* stride of the token rows of z */
  float eps;     /* > 0 */
} gdn_gate_norm_shape;

gdn_status gdn_gate_norm_fwd(const gdn_gate_norm_shape* shape, const void* o, const void* z,
                             const float* w, void* y, void* stream);

size_t gdn_gate_norm_workspace_bytes(const gdn_gate_norm_shape* shape);

gdn_status gdn_gate_norm_bwd(const gdn_gate_norm_shape* shape, const void* o, const void* z,
                             const float* w, const void* dy, void* dout, void* dz, float* dw,
                             void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------- block boundary
 *     p     = x / sqrt(mean(x^2) + eps) * w_post   (w_post NULL: p = x)
 *     h_out = h + scale * p                        (scale NULL: h + p)
 *     y     = h_out / sqrt(mean(h_out^2) + eps) * w
 * h, h_out (the residual stream) [rows, C] of res_dtype; x (the block's
 * output), y [rows, C] of dtype; w, w_post, scale [C] fp32. res_dtype is dtype
 * or GDN_DTYPE_F32. h_out may be h. x NULL (first block): y is the norm of h;
 * h_out, w_post and scale must then be NULL too. */
typedef struct {
  int rows;
  int C;         /* multiple of 8, 8..16384 */
  int dtype, res_dtype;
  float eps;     /* > 0 */
} gdn_res_norm_shape;

gdn_status gdn_res_norm_fwd(const gdn_res_norm_shape* shape, const void* h, const void* x,
                            const float* w, const float* w_post, const float* scale, void* h_out,
                            void* y, void* stream);

size_t gdn_res_norm_workspace_bytes(const gdn_res_norm_shape* shape);

/* The gradient at the stored h_out: from dy and dh_out (NULL: zero) dh (of
 * res_dtype), dx, and dw, dw_post, dscale [C] fp32 (those of absent parameters
 * NULL). x may be NULL where w_post and scale are NULL: the block's gradient
 * is then dh, and dx (dh in dtype) may be NULL. dh may be dh_out. */
gdn_status gdn_res_norm_bwd(const gdn_res_norm_shape* shape, const void* h_out, const void* x,
                            const float* w, const float* w_post, const float* scale,
                            const void* dy, const void* dh_out, void* dh, void* dx, float* dw,
                            float* dw_post, float* dscale, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Synchronises `stream`, then returns what the calls of this header have
 * recorded on the current device since the last such query (GDN_OK, or
 * GDN_ERR_TIMEOUT for a wait that ran out) and resets it. One word for all
 * streams of a device. */
gdn_status gdn_layer_status(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LAYER_H_ */
