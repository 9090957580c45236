/*
 * moe_train.h -- what a training step needs beside the layer (included by
 * moe.h, whose conventions hold here too): the router's losses with their
 * gradient, and the update of the experts' weights by Newton-Schulz products.
 */
#ifndef MOE_TRAIN_H
#define MOE_TRAIN_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------------------------------------------- router losses */

/* The tokens are cut into S = ceil(T / seq_len) sequences of seq_len (the last
 * one may be shorter); seq_len = T takes the batch as one.  mask [T] u8 (or
 * NULL: every token counts) is 0 for padding: such a token adds to nothing,
 * whatever its logits hold.  With p_te = softmax_e(logits[t]), n_s the tokens of
 * sequence s, c_se the picks of expert e among them and P_se the sum of p_te over
 * them,
 *   loss[0] = mean over the sequences with tokens of E / (K n_s^2) sum_e c_se P_se
 *             (1 where picks and probabilities are spread evenly),
 *   loss[1] = mean over all tokens of (log sum_e exp logits[t, e])^2.
 *  logits [T, E] f32, topk_idx [T, K] i32 (as moe_route writes it; ids outside
 *           [0, E) are skipped), mask in
 *  counts [S, E] i32 (c), tokens [S + 2] i32 (n, then their sum, then the number of
 *           sequences with tokens), probs [S, E] f32 (P), loss [2] f32 out
 *  ws: at least moe_balance_workspace_bytes(d, seq_len) bytes, 256-byte aligned,
 *           in any state; calls that overlap in time need separate ones.
 * Without any token both losses are 0.  A logit of -inf takes its expert out of a
 * row.  A row of only -inf, or with +inf or NaN, makes its sequence's probs, and
 * the losses, NaN.  Uses T, E and K of the dims (all are checked); T <= 2^28.
 * Errors: MOE_EINVAL for seq_len outside [1, T], MOE_EWORKSPACE. */
size_t moe_balance_workspace_bytes(const moe_dims* d, int seq_len);
int moe_balance(const moe_dims* d, int seq_len, const float* logits, const int32_t* topk_idx,
                const uint8_t* mask, int32_t* counts, int32_t* tokens, float* probs, float* loss,
                void* ws, size_t ws_bytes, void* stream);

/* Gradient of dloss[0] loss[0] + dloss[1] loss[1] for the logits, with the picks
 * held fixed:
 *   dlogits[t, e] = p_te (q_se - sum_j p_tj q_sj + dloss[1] 2 / N lse_t),
 *   q_se = dloss[0] E / (K n_s^2 S') c_se,  N = tokens[S],  S' = tokens[S + 1],
 * 0 for padding; plus, where dtopk_w, topk_w and topk_idx are given, what
 * moe_route_bwd writes for them (padding included), in the same pass: it takes
 * that call's place in a backward with these losses.
 *  logits, mask, counts, tokens as above (counts and tokens may be sums over the
 *           ranks of a larger batch, where seq_len = T: then tokens[2] stays 1),
 *  dloss [2] f32; dtopk_w, topk_w [T, K] f32 and topk_idx [T, K] i32: all three
 *           or none (NULL) in
 *  dlogits [T, E] f32 out; may be logits itself. */
int moe_balance_bwd(const moe_dims* d, int seq_len, const float* logits, const uint8_t* mask,
                    const int32_t* counts, const int32_t* tokens, const float* dloss,
                    const float* dtopk_w, const float* topk_w, const int32_t* topk_idx,
                    float* dlogits, void* stream);

/* --------------------------------------- update by Newton-Schulz products */

/* The iteration: X <- a X + (b X X^T + c (X X^T)^2) X, `steps` times from
 * X = U / |U|_F (Frobenius norm), with coefficients of its own for every step.
 * Singular values in (0, 1] go towards 1 while the singular vectors stay, so the
 * result is close to the nearest matrix with orthonormal rows (or columns). */
#define MOE_NEWTON_MAX_STEPS 16
typedef struct {
  int32_t steps;                          /* 1 .. MOE_NEWTON_MAX_STEPS                       */
  float coef[MOE_NEWTON_MAX_STEPS][3];    /* a, b, c of each step; magnitudes at most 32     */
} moe_newton;

/* Or'ed to MOE_BF16 in the calls below: results and weights in bf16, products as exact
 * as for MOE_F32 (and at their time, 2.3 to 2.8 times that of MOE_BF16 alone for large matrices). */
#define MOE_EXACT 16

/* Workspace of the two calls below for G matrices [R, C] (0 for sizes that they
 * refuse, dtype as theirs): at most a few copies of a part of the stack, which is worked on part by part,
 * with sides rounded up to 64; for any coefficients.
 * 256-byte aligned, in any state; one for calls that overlap in time each. */
size_t moe_muon_workspace_bytes(int G, int R, int C, int dtype);

/* out[g] = the iteration's result for matrix g of the stack.
 *  g [G, R, C] f32 in (not changed), out [G, R, C] of `dtype` out
 *  n: the iteration (host memory, read during the call), or NULL: 5 steps of
 *           (3.4445, -4.7750, 2.0315)
 * dtype MOE_BF16: products of 11-bit (fp16) factors with f32 sums, X itself in 22
 * bits as long as later steps would enlarge its roundings.  With the default steps the
 * result is off by 1e-3 (full rank) to 4e-3 (rank 1) of its norm, before its rounding to
 * bf16.  With others by what they make of changes of 2^-12: rank 1 loses 6e-3 for
 * (4, -6.8, 2.9), (3.9, -6.3, 2.6), (3.7, -5.6, 2.3), (2.9, -3.1, 1.2), (2.8, -3, 1.2), low
 * ranks 1e-2 to 3e-2 where the first step has a = 8, and steps close to where the
 * iteration no longer settles (which f32 arithmetic shows by an error of 1e-3) lose the
 * result: such ones need the exact form.
 * MOE_F32, MOE_EXACT, and matrices with fewer than 32 rows or columns: factors of 22 bits, about as
 * exact as f32 arithmetic (default steps: 1e-6 for a full rank, 1e-4 for rank 1).  Up to 48 rows or columns (64 if the other side has 2048 or more),
 * where the magnitudes above 1 of the steps' a multiply to at most 4096: 64 bits
 * up to the result.
 * Any G from 1 to 2^30 and R, C from 1 to 2^20 with R*C <= 2^32 and G*R*C <= 2^39.  No step but
 * the last may leave a singular value above 15 (the range of fp16; such a matrix becomes
 * infinite or NaN); the last may leave any.  A matrix of zeros gives zeros; an infinity or NaN makes its own matrix
 * NaN and no other.  The scale of a matrix has no effect, down to subnormal entries.  A
 * matrix's bits depend on its values and on G, R and C, not on the other matrices. */
int moe_orthogonalize(int G, int R, int C, int dtype, const moe_newton* n, const float* g, void* out,
                      void* ws, size_t ws_bytes, void* stream);

/* One step of the Muon optimizer on a stack of weights:
 *   mom <- momentum mom + grad;   U = nesterov ? grad + momentum mom : mom
 *   master <- (1 - lr weight_decay) master - lr scale O,  O = the iteration's result for U
 *   w <- master rounded to bf16 (MOE_BF16 only)
 *  grad [G, R, C] f32 in (as the weight-gradient calls write it), mom and master
 *           [G, R, C] f32 in and out
 *  w [G, R, C] bf16 out; NULL for MOE_F32, where master is the weight itself
 *  lr: device f32[1], or NULL: p->lr (a captured step follows a schedule by it)
 * Precision and sizes as above (O is not rounded to dtype).  MOE_BF16 | MOE_EXACT gives
 * the bits of MOE_F32 in mom and master, and w beside them. */
typedef struct {
  float lr, momentum, weight_decay, scale;
  int32_t nesterov;
} moe_muon_params;
int moe_muon(int G, int R, int C, int dtype, const moe_newton* n, const moe_muon_params* p,
             const float* lr, const float* grad, float* mom, float* master, void* w, void* ws,
             size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TRAIN_H */
