/*
 * mxfp8_experts.h — C ABI of two operators on the expert weights whose
 * gradient mxfp8_wgrad_grouped computes: the orthogonalised update of a stack
 * of gradients (training) and the whole expert layer for a few tokens
 * (serving). Status codes, mxfp8_last_error(), mxfp8_device_status() and the
 * conventions on pointers, streams and errors are those of mxfp8_wgrad.h.
 */
#ifndef MXFP8_EXPERTS_H
#define MXFP8_EXPERTS_H

#include "mxfp8_wgrad.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest token count, expert count and top-k of one mxfp8_moe_layer call. */
#define MXFP8_MOE_MAX_TOKENS 128
#define MXFP8_MOE_MAX_EXPERTS 1024
#define MXFP8_MOE_MAX_TOPK 16

/* Router scores (mxfp8_moe_layer, `score`). */
#define MXFP8_SCORE_SOFTMAX 0
#define MXFP8_SCORE_SIGMOID 1

/*
 * A whole mixture-of-experts layer for a few tokens: router, choice of
 * experts, the experts' gated MLPs on MXFP8 weights, weighted sum.
 *
 *   logit[t][e] = sum_h x[t][h] router[e][h]                  (e < experts; fp32)
 *   score       = softmax over e, or sigmoid, of the logits
 *   chosen(t)   = the top_k experts by score + bias (by score when bias is
 *                 NULL); equal values go to the lower index, NaN counts as -inf
 *   weight      = scale * score (without the bias) of each chosen expert,
 *                 divided by the sum of the chosen scores when renormalize != 0
 *   h(t,e)      = silu(g) * u,  g = W13[e][0..I) x[t],  u = W13[e][I..2I) x[t]
 *   out[t]      = bf16_rne( sum over the chosen e in [first, first + local) of
 *                 weight(t,e) * W2[e] h(t,e) )
 *
 * Only experts [first, first + local) live here (expert parallelism): a token
 * whose chosen experts all live elsewhere gets exact zeros.
 *
 *   x      [T][H]               bf16, 16-byte aligned, 0 <= T <= MXFP8_MOE_MAX_TOKENS (T == 0: no-op)
 *   router [experts][H]         bf16, 16-byte aligned
 *   bias   [experts]            fp32 or NULL
 *   w13    [local][2 I][H]      E4M3 (gate rows, then up rows), 16-byte aligned
 *   s13    [local][2 I][H/32]   E8M0, 4-byte aligned
 *   w2     [local][H][I]        E4M3, 16-byte aligned;  s2 [local][H][I/32] E8M0, 4-byte aligned
 *   H, I   multiples of 32, at most 32768
 *   experts 1..MXFP8_MOE_MAX_EXPERTS; 0 <= first, 1 <= local, first + local <= experts
 *   top_k  1..min(experts, MXFP8_MOE_MAX_TOPK)
 *   out    [T][H] bf16, 16-byte aligned; every element is written
 *   topk_ids [T][top_k] int32 and topk_weights [T][top_k] fp32 (either may be
 *          NULL): the chosen experts in descending order of score + bias (global
 *          indices) and their weights
 *
 * The activations keep bf16 precision (x) and about nine bits (h); products
 * are accumulated in fp32 and summed in a fixed order: the output is
 * bit-reproducible.
 *
 * Scratch comes from the per-(device, stream) cache of mxfp8_wgrad_grouped
 * (same rule under stream capture) unless the _ws form is used: `workspace`
 * is a device pointer, 256-byte aligned, of at least
 * mxfp8_moe_layer_workspace_bytes() bytes (else MXFP8_ENOWS).
 */
int mxfp8_moe_layer(const uint16_t* x, int T, const uint16_t* router, const float* bias, const uint8_t* w13,
                    const uint8_t* s13, const uint8_t* w2, const uint8_t* s2, int experts, int first, int local, int H,
                    int I, int top_k, int score, int renormalize, float scale, uint16_t* out, int32_t* topk_ids,
                    float* topk_weights, void* stream);

int mxfp8_moe_layer_ws(const uint16_t* x, int T, const uint16_t* router, const float* bias, const uint8_t* w13,
                       const uint8_t* s13, const uint8_t* w2, const uint8_t* s2, int experts, int first, int local,
                       int H, int I, int top_k, int score, int renormalize, float scale, uint16_t* out,
                       int32_t* topk_ids, float* topk_weights, void* workspace, size_t workspace_bytes, void* stream);

/* Scratch for these sizes; 0 if they are invalid. Host-only, no CUDA call. */
size_t mxfp8_moe_layer_workspace_bytes(int T, int experts, int local, int H, int I, int top_k);

/* Types of the gradient (mxfp8_muon_update, `grad_type`). */
#define MXFP8_GRAD_BF16 0
#define MXFP8_GRAD_F32 1

/* Largest number of Newton-Schulz steps of one call. */
#define MXFP8_MUON_MAX_STEPS 16

/*
 * Orthogonalised update of a stack of gradients, with momentum: for every
 * matrix e of the stack
 *
 *   momentum' = mu * momentum + grad                  (fp32, written back)
 *   u  = grad + mu * momentum'  (nesterov != 0), else momentum';  without a
 *        momentum buffer (NULL) u = grad
 *   X0 = u / (||u||_F + eps)
 *   X <- a X + (b A + c A A) X,  A = X X^T            (`steps` times; when N > K
 *        the same iteration on X^T, which gives the same matrix)
 *   out[e] = bf16_rne(X)
 *
 * which drives the singular values of u towards one and keeps its singular
 * vectors. A zero matrix (an expert without tokens) gives exact zeros; a
 * matrix holding a NaN or an infinity, or whose sum of squares overflows
 * fp32, gives NaN and leaves the other matrices alone. Small elements lose
 * nothing: the norm is right down to the smallest subnormals.
 *
 *   grad     [E][N][K] bf16 (the output of mxfp8_wgrad_grouped) or fp32, 16-byte aligned
 *   momentum [E][N][K] fp32, 16-byte aligned, or NULL
 *   out      [E][N][K] bf16, 16-byte aligned; every element is written
 *   E        0 <= E <= MXFP8_MAX_EXPERTS (E == 0: no-op); N, K >= 1, at most 32768, K % 8 == 0
 *   steps    1..MXFP8_MUON_MAX_STEPS;  a, b, c finite, |a|, |b|, |c| <= 16;  eps >= 0
 *
 * Coefficients whose iteration can leave the range of the fp16 operands are
 * refused (MXFP8_EINVAL). With X0's singular values anywhere in [0, 1], no
 * singular value of an X that is multiplied may pass sqrt(14), and no
 * eigenvalue of b A + c A A - beta I may pass 14 in magnitude, where beta is
 * 0.875 (b + c) in the last step, half of that in the one before and zero in the
 * others. Maps that keep [0, 1] near [0, 1.3], the default among them, pass for
 * every step count; a X alone passes for a^(steps - 1) up to 3.7.
 *
 * The products run on fp16 operands with 11 significant bits (scaled by
 * powers of two) and fp32 accumulation; the a X term keeps 22 bits. What becomes
 * of the roundings depends on how far the iteration carries them. With the
 * coefficients above, on matrices of full rank, the 2-norm error before the
 * rounding to bf16, relative to the exact iteration, is (median / 99% of 720
 * matrices with normal, heavy-tailed, decaying and few-strong-directions
 * spectra; rounding model on the host):
 *
 *   steps                    up to 5           8                 12                16
 *   shorter side 96 ..       1.0e-3 / 1.6e-3   2.4e-3 / 3.5e-3   3.9e-3 / 6e-3     4.9e-3 / 1.3e-2
 *   shorter side 8 .. 52     1.5e-3 / 3.1e-3   2.6e-3 / 6e-3     3.7e-3 / 1.5e-2   4.6e-3 / 3.5e-2
 *
 * It is no bound: it is about a thousand times what the same iteration in fp32
 * leaves, and grows with it where the map is steep at some singular values.
 * Directions that have no part in u hold rounding noise that each step
 * multiplies by a: nothing at five steps, most of the result after some twelve
 * (in fp32 too). Where ||u|| is far below eps, elements of the result below
 * 2^-35 are lost on the general path. Other coefficients: a step rounds A, R and
 * the X that R multiplies to 11 bits each, so its error is a few 2^-12 of the
 * largest of its terms. The output is bit-reproducible.
 *
 * Scratch as for mxfp8_moe_layer (cache, or the _ws form). Matrices with a
 * shorter side up to 128 and a longer one up to 2048 stay on chip: nothing is
 * taken from the cache (such a call can be captured on any stream), and the _ws
 * form asks for a nominal 512 bytes that it does not touch.
 */
int mxfp8_muon_update(const void* grad, int grad_type, float* momentum, int E, int N, int K, float mu, int nesterov,
                      int steps, float a, float b, float c, float eps, uint16_t* out, void* stream);

int mxfp8_muon_update_ws(const void* grad, int grad_type, float* momentum, int E, int N, int K, float mu, int nesterov,
                         int steps, float a, float b, float c, float eps, uint16_t* out, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Scratch for these sizes; 0 if they are invalid. Host-only, no CUDA call. */
size_t mxfp8_muon_update_workspace_bytes(int E, int N, int K);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_EXPERTS_H */
