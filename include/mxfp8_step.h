/*
 * mxfp8_step.h — C ABI of the operators of a training step around the products
 * of an expert layer: tokens sorted by expert and back (with the router's
 * weights, and the gradients of both directions), and the global norm of many
 * gradients with clipping. They lead from token order to the operands of
 * mxfp8_grouped_gemm, mxfp8_quantize_transpose_bf16 and mxfp8_wgrad_grouped
 * and back, and from the latter's output to mxfp8_muon_update. Status codes,
 * mxfp8_last_error(), mxfp8_device_status() and the conventions on pointers,
 * streams and errors are those of mxfp8_wgrad.h. Outputs overlap no input and
 * no other output unless that is said to be allowed. Under stream capture: a
 * first call in a context loads kernels, so make one before capturing.
 */
#ifndef MXFP8_STEP_H
#define MXFP8_STEP_H

#include "mxfp8_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* More bits of the device status word (mxfp8_device_status). */
#define MXFP8_DEV_TOKENS_ROWS 16   /* a plan had more (padded) pairs than rows: the last ones were dropped */
#define MXFP8_DEV_TOKENS_RANGE 32  /* a slot or src entry out of range; treated as absent (-1) */

/* Largest top_k, group alignment and pair count (T * top_k) of the token operators. */
#define MXFP8_TOKENS_MAX_TOPK 64
#define MXFP8_TOKENS_MAX_ALIGN 1024
#define MXFP8_TOKENS_MAX_PAIRS (1 << 30)

/* Types of expert indices (mxfp8_token_plan, `id_type`). */
#define MXFP8_ID_I32 0
#define MXFP8_ID_I64 1

/*
 * The plan of a routing: which row of the sorted buffers belongs to which
 * (token, choice) pair. Pair p = t * top_k + j chose expert ids[t][j]; it is
 * here when first <= ids[t][j] < first + local (one rank's experts), otherwise
 * (other ranks' experts, negative entries of padding tokens, anything else) it
 * is absent. Expert e of the n_e pairs here takes rows
 *
 *   start_e = sum over e' < e of align * ceil(n_e' / align),
 *   slot(p) = start_e(p) + number of earlier pairs of the same expert,
 *   offs[e] = start_e + align * ceil(n_e / align),
 *
 * so that rows keep the tokens' order inside a group, a token may choose an
 * expert more than once, and the rows between a group's last pair and its end
 * are padding. align = 32 gives the offsets that mxfp8_wgrad_grouped asks for;
 * mxfp8_grouped_gemm takes any.
 *
 *   ids  [T][top_k] int32 or int64 (id_type), aligned to its element size
 *   T >= 0, 1 <= top_k <= MXFP8_TOKENS_MAX_TOPK, T * top_k <= MXFP8_TOKENS_MAX_PAIRS
 *   first >= 0; 1 <= local <= MXFP8_MAX_EXPERTS; 1 <= align <= MXFP8_TOKENS_MAX_ALIGN
 *   rows of the sorted buffers: 0 <= rows < 2^31, a multiple of align.
 *        mxfp8_token_plan_rows() rows hold every routing. With fewer, the pairs
 *        whose slot would be rows or more are dropped (their slot is -1), offs
 *        is cut to rows, and MXFP8_DEV_TOKENS_ROWS is set.
 *   offs [local] int32, inclusive group ends (multiples of align)
 *   slot [T][top_k] int32, the pair's row, or -1
 *   src  [rows] int32, the row's pair, or -1 (padding, and rows from offs[local-1] on)
 * All 4-byte aligned; every element is written. No scratch, one launch.
 */
int mxfp8_token_plan(const void* ids, int id_type, int64_t T, int top_k, int first, int local, int align, int64_t rows,
                     int32_t* offs, int32_t* slot, int32_t* src, void* stream);

/* The fewest rows that hold every routing of T tokens: at most align - 1 padding
 * rows for each expert that can have a pair. -1 if the sizes are invalid or the
 * result is 2^31 or more. Host-only. */
int64_t mxfp8_token_plan_rows(int64_t T, int top_k, int local, int align);

/*
 * The operators below take a plan (slot [T][top_k] and src [rows], which belong
 * together, as mxfp8_token_plan writes them). Entries outside [0, rows) and
 * [0, T * top_k) count as -1 (MXFP8_DEV_TOKENS_RANGE is set for those below -1
 * or too large), so no plan makes an access leave the buffers. H is at most
 * 32768. Sizes T and rows may be 0.
 *
 * Rows in sorted order:
 *   out[r] = x[src[r] / top_k], exact zeros where src[r] = -1
 *   x [T][H] bf16, out [rows][H] bf16; H % 8 == 0; both 16-byte aligned
 * Every row of out is written once (a row whose pair is in src but not in slot
 * would be left out: plans of mxfp8_token_plan have none).
 */
int mxfp8_token_dispatch(const uint16_t* x, int64_t T, int H, int top_k, const int32_t* slot, const int32_t* src,
                         int64_t rows, uint16_t* out, void* stream);

/*
 * The same rows quantised along H by the rule of mxfp8_quantize_tokenwise (the
 * operand X of mxfp8_grouped_gemm): q [rows][H] E4M3 (16-byte aligned), s
 * [rows][H/32] E8M0; padding rows hold q = 0, s = 0. H % 32 == 0.
 */
int mxfp8_token_dispatch_mxfp8(const uint16_t* x, int64_t T, int H, int top_k, const int32_t* slot, const int32_t* src,
                               int64_t rows, uint8_t* q, uint8_t* s, void* stream);

/*
 * The gradient of mxfp8_token_dispatch with respect to x:
 *   dx[t] = bf16_rne( sum over j with a slot of dxs[slot[t][j]] )   (fp32, ascending j)
 *   dxs [rows][H] bf16, dx [T][H] bf16; H % 8 == 0; both 16-byte aligned
 * A token without a pair here gets exact zeros; padding rows are not read.
 */
int mxfp8_token_dispatch_grad(const uint16_t* dxs, int64_t rows, int64_t T, int H, int top_k, const int32_t* slot,
                              uint16_t* dx, void* stream);

/*
 * Back to token order with the router's weights:
 *   out[t] = bf16_rne( sum over j with a slot of weights[t][j] * y[slot[t][j]] )   (fp32, ascending j)
 *   y [rows][H] bf16, weights [T][top_k] fp32, out [T][H] bf16; H % 8 == 0; y and out 16-byte aligned
 * Weights of absent pairs and padding rows are not read into the sum, whatever they hold.
 */
int mxfp8_token_combine(const uint16_t* y, int64_t rows, const float* weights, int64_t T, int H, int top_k,
                        const int32_t* slot, uint16_t* out, void* stream);

/*
 * The gradients of mxfp8_token_combine, from dout [T][H] bf16:
 *   dy[r]          = bf16_rne( weights[p] * dout[p / top_k] ), p = src[r]; exact zeros where src[r] = -1
 *   dweights[t][j] = sum over h of dout[t][h] * y[slot[t][j]][h]   (fp32; 0 for absent pairs)
 *   y, dy [rows][H] bf16, weights, dweights [T][top_k] fp32; H % 8 == 0; dout, y and dy 16-byte aligned
 * dy may be y (each row is read before it is written). Bit-reproducible.
 */
int mxfp8_token_combine_grad(const uint16_t* dout, const uint16_t* y, const float* weights, int64_t T, int H, int top_k,
                             const int32_t* slot, const int32_t* src, int64_t rows, uint16_t* dy, float* dweights,
                             void* stream);

/* Largest number of tensors of one mxfp8_grad_norm or mxfp8_clip_grads call. */
#define MXFP8_GRAD_MAX_TENSORS 65536

/*
 * Global 2-norm of many gradients:  *norm = sqrt( sum over all elements of g^2 ).
 *
 *   grads [n]  HOST array of device pointers, aligned to their element size
 *              (views into a flat buffer will do); NULL where the size is 0
 *   sizes [n]  HOST array of element counts, >= 0
 *   types [n]  HOST array of MXFP8_GRAD_BF16 / MXFP8_GRAD_F32
 *   norm       device fp32, 4-byte aligned
 *   0 <= n <= MXFP8_GRAD_MAX_TENSORS; the arrays are not needed after the call
 *
 * Squares are summed in fp32 over at most 64 elements and joined in 64 bits,
 * in a fixed order (bit-reproducible for tensors at the same addresses modulo 16;
 * elsewhere the last bit may differ); elements whose squares leave fp32's
 * range are summed in 64 bits, so that nothing over- or underflows but the
 * result's own rounding. A NaN gives NaN, an infinity without a NaN infinity.
 *
 * Scratch (5 KB for every 1024 tensors, 328 KB at most) as for mxfp8_moe_layer: the per-(device, stream) cache, or
 * the _ws form with a 256-byte aligned workspace of mxfp8_grad_workspace_bytes(n).
 */
int mxfp8_grad_norm(const void* const* grads, const int64_t* sizes, const int32_t* types, int n, float* norm,
                    void* stream);
int mxfp8_grad_norm_ws(const void* const* grads, const int64_t* sizes, const int32_t* types, int n, float* norm,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients scaled so that their global norm is at most max_norm:
 *
 *   c = min(1, max_norm / (norm + eps)),   out_i = round(c * g_i)  (to g_i's type)
 *
 *   norm_in  NULL: norm is that of these gradients (64 bits until c). Otherwise
 *            a device fp32 that holds it (the norm over the ranks of a job, for
 *            instance); norm must then be NULL or norm_in.
 *   norm     device fp32 that receives the norm, or NULL
 *   outs [n] HOST array of device pointers, or NULL for in place. outs[i] may be
 *            grads[i]; otherwise an output overlaps no other output and no gradient
 *            (MXFP8_EINVAL).
 *   max_norm >= 0 and finite, eps >= 0 and finite
 *
 * In place and with c = 1 nothing is written. A norm of infinity gives c = 0
 * (infinite elements become NaN, the others 0), a NaN norm makes every element
 * NaN. Other arguments, limits and scratch as for mxfp8_grad_norm.
 */
int mxfp8_clip_grads(const void* const* grads, const int64_t* sizes, const int32_t* types, int n, float max_norm,
                     float eps, const float* norm_in, float* norm, void* const* outs, void* stream);
int mxfp8_clip_grads_ws(const void* const* grads, const int64_t* sizes, const int32_t* types, int n, float max_norm,
                        float eps, const float* norm_in, float* norm, void* const* outs, void* workspace,
                        size_t workspace_bytes, void* stream);

/* Scratch for n tensors; 0 if n is invalid. Host-only, no CUDA call. */
size_t mxfp8_grad_workspace_bytes(int n);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_STEP_H */
