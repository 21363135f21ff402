/*
 * q3_block.h -- C ABI of the operators that stand between two packed products
 * and behind the last one (MI355X, gfx950): the gated feed-forward block and
 * products of many tokens on packed weights with the gradients of their inputs,
 * the residual norms that turn a product's fp32 outputs into the next product's
 * bf16 activations, and the choice of a token from the vocabulary logits.
 *
 * The conventions are q3.h's: device pointers, caller-owned buffers, no
 * allocation, asynchronous on `stream`, arguments validated on the host before
 * any HIP call.  Packed weights are frozen: gradients are those of activations,
 * norm weights and gates.  A workspace's contents are scratch and need not
 * be initialised; calls that overlap in time must not share one (two captured
 * graphs that may run at once need two).  Buffers of one call must not
 * overlap, except where a comment allows it.
 *
 * Types: activations that enter a product are bf16 bit patterns, products and
 * the gradients that products compute are fp32; Q3_BF16 or Q3_F32 says what the
 * residual stream is kept in.  Every result is rounded once, to the type it is
 * written in; sums and statistics are held in 32 bits or more.  Row pitches (ld)
 * are in elements.
 */
#ifndef Q3_BLOCK_H
#define Q3_BLOCK_H

#include "q3.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum q3_dtype { Q3_F32 = 0, Q3_BF16 = 1 } q3_dtype;

/* The gate's activation: silu(z) = z / (1 + e^-z), or the tanh form of GELU,
 * z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))). */
typedef enum q3_act { Q3_ACT_SILU = 0, Q3_ACT_GELU_TANH = 1 } q3_act;

/* ---- Products of any number of tokens ------------------------------------ */

/* y[m][n] = x[m][:] . w[n][:], m >= 1: q3_gemm_small_m for up to 64 tokens, and
 * for more the matrix dequantised exactly to bf16 in the workspace, multiplied
 * on the matrix cores with fp32 accumulation (or, where that is faster, 64 or
 * 128 tokens at a time straight from the packed planes).  x bf16 [m][ldx],
 * ldx % 8 == 0, 16-byte aligned, 256 of its rows below 2 GiB; y fp32 [m][ldy];
 * m < 2^31; n and k up to 2^21 here and in what follows.
 * workspace: 256-byte aligned, at least q3_gemm_workspace_bytes(n, k, m) bytes
 * (Q3_ERR_INVALID_ARG otherwise; it may be NULL where that is 0). */
Q3_API int64_t q3_gemm_workspace_bytes(int64_t n, int64_t k, int64_t m);
Q3_API q3_status q3_gemm(const q3_matrix* w, const uint16_t* x, int64_t m, int64_t ldx, float* y, int64_t ldy,
                         void* workspace, int64_t workspace_bytes, void* stream);

/* The gradient of that product's input: dx[m][k] = sum_n dy[m][n] w[n][k].
 * dy bf16 [m][ld_dy], ld_dy % 8 == 0, 16-byte aligned (what stands between n
 * and ld_dy is not read as values); dx fp32 [m][ld_dx].  n = 0 gives zeros.
 * workspace as above, q3_gemm_backward_workspace_bytes(n, k, m) bytes. */
Q3_API int64_t q3_gemm_backward_workspace_bytes(int64_t n, int64_t k, int64_t m);
Q3_API q3_status q3_gemm_backward(const q3_matrix* w, const uint16_t* dy, int64_t m, int64_t ld_dy, float* dx,
                                  int64_t ld_dx, void* workspace, int64_t workspace_bytes, void* stream);

/* ---- Gated feed-forward block ----------------------------------------------- */

/* h[m][i] = act(g) * u with g = x[m] . w[i], u = x[m] . w[I + i], both products,
 * the activation and the product in one kernel (behind a pass that widens the
 * matrix where the workspace is not 0 bytes): gate_up is a packed matrix of
 * n = 2I rows [gate rows 0..I-1; up rows I..2I-1], I % 32 == 0.
 * x bf16 [m][ldx] as in q3_gemm; h bf16 [m][ldh], ldh >= I, ldh % 8 == 0,
 * 16-byte aligned (so it is the down product's x).
 * pre (may be NULL): fp32 [m][ld_pre], the pre-activations [g; u] for the
 * backward pass, ld_pre >= 2I, ld_pre % 4 == 0, 16-byte aligned.
 * workspace: 256-byte aligned, q3_glu_workspace_bytes(2I, k, m) bytes (0
 * where the packed planes are read directly, as for up to 64 tokens). */
Q3_API int64_t q3_glu_workspace_bytes(int64_t n_gu, int64_t k, int64_t m);
Q3_API q3_status q3_glu(const q3_matrix* gate_up, const uint16_t* x, int64_t m, int64_t ldx, int32_t act,
                        uint16_t* h, int64_t ldh, float* pre, int64_t ld_pre, void* workspace,
                        int64_t workspace_bytes, void* stream);

/* The gradient of the pre-activations: dpre[m][i] = dh u act'(g),
 * dpre[m][I + i] = dh act(g), for pre as q3_glu wrote it and dh fp32 [m][ld_dh]
 * (q3_gemm_backward of the down projection).  dpre bf16 [m][ld_dpre], so that
 * q3_gemm_backward(gate_up, dpre) is the gradient of x.  All rows 16-byte
 * aligned (ld_pre % 4, ld_dh % 4, ld_dpre % 8 == 0), inter % 32 == 0,
 * m * inter <= 2^34 - 1024 (one launch). */
Q3_API q3_status q3_glu_backward(const float* pre, int64_t ld_pre, const float* dh, int64_t ld_dh, int32_t act,
                                 int64_t m, int64_t inter, uint16_t* dpre, int64_t ld_dpre, void* stream);

/* ---- Residual norms --------------------------------------------------------- */

/* The end of one block and the start of the next, one pass over each row:
 *   t  = post_weight ? post_weight * y * rsqrt(mean(y^2) + eps) : y
 *   r' = r + scale * gate * t            (gate: 1 when NULL)
 *   x  = pre_weight * r' * rsqrt(mean(r'^2) + eps)   (pre_weight: 1 when NULL)
 * x is computed from r' before r' is rounded to r_type.
 *   y        fp32 [m][ldy] (a product's output), or NULL: r' = r; then
 *            post_weight and gate must be NULL and r_out may be
 *   gate     fp32 [m][ld_gate], or with ld_gate == 0 one row for all tokens
 *   r, r_out [m][ldr], [m][ldr_out] of r_type; r_out may be r itself (same
 *            pointer and pitch); NULL only when y is
 *   x        bf16 [m][ldx] or NULL (then only r' is computed)
 *   weights  fp32 [n]
 * 1 <= n <= 16384, m >= 1, eps >= 0 (a row of zeros with eps = 0 gives NaN).
 * Elements are naturally aligned; rows whose starts are all aligned to four
 * elements (and n % 4 == 0) move in vectors. */
Q3_API q3_status q3_residual_norm(const float* y, int64_t ldy, const float* post_weight, const float* gate,
                                  int64_t ld_gate, float scale, const void* r, int64_t ldr, void* r_out,
                                  int64_t ldr_out, int32_t r_type, const float* pre_weight, uint16_t* x, int64_t ldx,
                                  float eps, int64_t m, int64_t n, void* stream);

/* Its backward pass, from the kept r' (r_out as it was written) and y:
 *   dx (may be NULL: zero) fp32 [m][ld_dx], the gradient of x; dr_out (may be
 *   NULL: zero) [m][ld_dr_out] of r_type, the gradient of r' from later blocks;
 *   dr [m][ld_dr] of r_type, the whole gradient of r' (which is r's); it may
 *   be dr_out itself
 *   dy bf16 [m][ld_dy] (what q3_gemm_backward takes); NULL when y is
 *   dgate fp32 [m][ld_dgate], or with ld_gate == 0 [n], summed over the
 *   tokens; NULL when gate is, may be NULL otherwise
 *   dpost_weight, dpre_weight fp32 [n], summed over the tokens; may be NULL
 * Sums over tokens are taken in a fixed order: equal calls give equal bits.
 * workspace: 256-byte aligned, q3_residual_norm_backward_workspace_bytes(m, n)
 * bytes. */
typedef struct q3_residual_norm_grads {
  const float* dx;
  int64_t ld_dx;
  const void* dr_out;
  int64_t ld_dr_out;
  void* dr;
  int64_t ld_dr;
  uint16_t* dy;
  int64_t ld_dy;
  float* dgate;
  int64_t ld_dgate;
  float* dpost_weight;
  float* dpre_weight;
} q3_residual_norm_grads;
Q3_API int64_t q3_residual_norm_backward_workspace_bytes(int64_t m, int64_t n);
Q3_API q3_status q3_residual_norm_backward(const float* y, int64_t ldy, const float* post_weight, const float* gate,
                                           int64_t ld_gate, float scale, const void* r_out, int64_t ldr_out,
                                           int32_t r_type, const float* pre_weight, float eps, int64_t m, int64_t n,
                                           const q3_residual_norm_grads* grads, void* workspace,
                                           int64_t workspace_bytes, void* stream);

/* ---- Feed-forward sublayer ----------------------------------------------------- */

/* The operators above as one call, the dense counterpart of q3_moe_mlp:
 *   y  = down . (act(g) * u),  [g; u] = gate_up . norm(r; pre_weight)
 *   r' = r + scale * gate * norm(y; post_weight)    (norm, gate: as in q3_residual_norm)
 *   x_next = norm(r'; next_weight)                  (NULL: not computed)
 * bitwise what q3_residual_norm, q3_glu, q3_gemm and q3_residual_norm give one
 * after the other.  gate_up [2I][k] and down [k][I], I % 32 == 0, k <= 16384;
 * weights, gate, r, r_out and x_next as in q3_residual_norm (n = k; r_out may be
 * r); any of the three weights may be NULL, next_weight must be where x_next is.
 * workspace: 256-byte aligned, q3_ffn_workspace_bytes(2I, k, m) bytes. */
typedef struct q3_ffn_norms {
  const float* pre_weight;
  const float* post_weight;
  const float* next_weight;
  const float* gate;
  int64_t ld_gate;
  float scale;
  float eps;
} q3_ffn_norms;
Q3_API int64_t q3_ffn_workspace_bytes(int64_t n_gu, int64_t k, int64_t m);
Q3_API q3_status q3_ffn(const q3_matrix* gate_up, const q3_matrix* down, int32_t act, const q3_ffn_norms* norms,
                        const void* r, int64_t ldr, void* r_out, int64_t ldr_out, int32_t r_type, uint16_t* x_next,
                        int64_t ldx_next, int64_t m, void* workspace, int64_t workspace_bytes, void* stream);

/* ---- Sampling ----------------------------------------------------------------- */

/* One token per row of logits (the vocabulary product's fp32 outputs), from a
 * given random number per row.  With weights w = exp((l - max l) / temperature)
 * and the row's entries ranked by logit (larger first, equal logits: lower
 * index first), an entry is kept while
 *   top_k:  its rank is below top_k          (off when <= 0)
 *   top_p:  the weights ranked before it sum to less than top_p times the sum
 *           over the top_k entries            (off when >= 1; rank 0 stays)
 *   min_p:  w >= min_p                        (off when <= 0; above 1 as 1)
 * and the token is the first kept entry, in index order, whose running sum of
 * kept weights exceeds u times their whole sum (the last one with weight when
 * none does).  logprobs (may be NULL): ln(w / that sum) of the token.
 *   temperature <= 0 takes the entry of rank 0 (logprob 0); NaN settings are off
 *   (temperature 1).  u: below 0 or NaN as 0.
 *   Logits of -inf and NaN are masked; a row with nothing else gives token -1
 *   and logprob -inf.  If some are +inf, only those count.
 * temperature, top_p, min_p, u: fp32 [m]; top_k: int32 [m]; device memory; each
 * but u may be NULL (off).  tokens int32 [m].
 * Weights are summed exactly, as integers of 2^-44 (entries below 2^-45 of the
 * largest weigh nothing): results do not depend on the order of summation.
 * 1 <= n <= 524288, 1 <= m <= 65535, ld >= n.  workspace: 256-byte aligned,
 * at least q3_sample_workspace_bytes(m, n) bytes. */
Q3_API int64_t q3_sample_workspace_bytes(int64_t m, int64_t n);
Q3_API q3_status q3_sample(const float* logits, int64_t m, int64_t n, int64_t ld, const float* temperature,
                           const int32_t* top_k, const float* top_p, const float* min_p, const float* u,
                           void* workspace, int64_t workspace_bytes, int32_t* tokens, float* logprobs, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* Q3_BLOCK_H */
