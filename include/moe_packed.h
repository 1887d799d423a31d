/*
 * moe_packed.h - training and serving the layer on packed batches, beside
 * moe.h (whose conventions, limits and status codes hold here): the balance
 * loss per sequence with its gradient, dropout whose mask is never stored, and
 * low-rank adapters of many requests with their gradients.
 *
 * The pages that moe.h cites print none of these ([MLG] is cited where a
 * formula of theirs is extended); the formulas stand beside each call.
 */
#ifndef MOE_B200_PACKED_H
#define MOE_B200_PACKED_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Balance loss and z-loss of packed, padded sequences, with per-expert
 * counts.  [MLG Algorithm 4: aux = E sum_e f_e P_e, here for each sequence]
 * Sequence s holds tokens [seq_offsets[s], seq_offsets[s+1]); its counted
 * tokens are those whose mask byte is not 0, n_s of them.  With k = top_k, N
 * counted tokens in all, S+ sequences with at least one:
 *   counts[s,e] = slots of s's counted tokens on e,  f = counts / (n_s k)
 *   P[s,e]      = mean over s's counted tokens of softmax(logits)[e]
 *   losses[0]   = 1/S+ sum_s E sum_e f[s,e] P[s,e]
 *   losses[1]   = 1/N sum_t (log sum_e exp logits[t,e])^2
 * One sequence that holds the whole batch gives moe_dispatch's aux_loss.
 * A batch split over ranks: each rank takes whole sequences (one that is cut
 * would need its f and P over all its tokens, which no call forms).  With N_r
 * and S+_r a rank's, N and S+ their sums over the ranks, the whole batch's
 * losses are the sums of S+_r / S+ losses_r[0] and N_r / N losses_r[1], and a
 * rank's dlogits are the whole batch's for dlosses (S+_r / S+ dlosses[0],
 * N_r / N dlosses[1]).
 *   n_seqs       sequences, >= 1
 *   seq_offsets  (n_seqs+1) int32, 0 <= non-decreasing <= T, or NULL with
 *                n_seqs = 1: all T tokens.  Tokens before the first or at and
 *                beyond the last offset belong to no sequence.  Other offsets
 *                are recorded on the error word (code 2), results undefined.
 *   token_mask   (T) uint8 or NULL: 0 = not counted (padding).  Logits and
 *                indices of tokens not counted may hold anything.
 *   logits       (T, E) fp32: moe_route's logits_out.  -INFINITY is allowed
 *                (an expert switched off) if the token has a finite logit.
 *   expert_indices (T, top_k); an index outside [0, E) of a counted token is
 *                recorded (code 1) and not counted
 *   counts       (n_seqs, E) int32 out; prob_mean (n_seqs, E) fp32 out (0 for
 *                a sequence without counted tokens)
 *   tokens       (n_seqs+2) int32 out: n_s, then N, then S+
 *   losses       (2) fp32 out (0 where nothing is counted)
 *   ws           moe_balance_workspace_size bytes, its own workspace; first
 *                256 bytes as in moe_workspace_init / moe_device_status
 * A probability whose logit is D below its token's largest is within
 * 2.3 D + 44 units of 2^-24 of exact, relative (2^x of a rounded product; below
 * 2^-126 it is 0).
 * Sums over tokens: fp32 for at most 64 tokens (and 8 such sums in pairs up to
 * T = 303103), fp64 above; fixed orders, no floating-point atomics.  T * top_k
 * and n_seqs at most 2^30. */
size_t moe_balance_workspace_size(const moe_config_t* cfg, int32_t n_seqs);
int moe_balance_loss(const moe_config_t* cfg, int32_t n_seqs, const int32_t* seq_offsets,
                     const uint8_t* token_mask, const float* logits,
                     const int32_t* expert_indices, int32_t* counts, float* prob_mean,
                     int32_t* tokens, float* losses, void* ws, size_t ws_bytes,
                     moe_stream_t stream);

/* Its gradient: with p = softmax(logits[t]), a_e = dlosses[0] E f[s,e] /
 * (S+ n_s) and lse the log-sum-exp,
 *   dlogits[t,e] = p_e (a_e - sum_e' p_e' a_e' + dlosses[1] 2 lse / N)
 * and 0 for tokens not counted, so that all T rows are written.  counts and
 * tokens are moe_balance_loss's outputs for the same arguments; dlosses (2)
 * fp32 device; dlogits (T, E) fp32 out, for moe_route_backward_add. */
int moe_balance_loss_backward(const moe_config_t* cfg, int32_t n_seqs, const int32_t* seq_offsets,
                              const uint8_t* token_mask, const float* logits,
                              const int32_t* counts, const int32_t* tokens, const float* dlosses,
                              float* dlogits, void* ws, size_t ws_bytes, moe_stream_t stream);

/* moe_route_backward with a further gradient of the logits: dL += dlogits_add
 * (T, E) fp32 before dx, dW_router and dbias are formed (one fp32 add; a sum
 * of zeros gives moe_route_backward's results).  dlogits may be dlogits_add. */
int moe_route_backward_add(const moe_config_t* cfg, const void* x, const float* W_router,
                           const float* logits, const int32_t* expert_indices, const float* gates,
                           const float* f, const float* dgates, const float* daux,
                           int32_t T_batch, const float* dlogits_add, float* dx, float* dW_router,
                           float* dbias, float* dlogits, void* ws, size_t ws_bytes,
                           moe_stream_t stream);

/* Dropout whose mask comes from a counter-based generator and is never
 * stored: the same arguments draw the same mask, forward and backward.
 *   p            drop probability, 0 <= p < 1, rounded to a multiple of 2^-16
 *                (one that rounds to 1 is refused); kept elements are
 *                multiplied by 1 / (1 - p) of the rounded p
 *   seed, offset the draws are Philox4x32-10 (Salmon et al., SC 2011) of the
 *                counter (b low, b high, offset low, offset high) under the
 *                key (seed low, seed high), b = (token_base + t) * width / 8
 *                + c / 8 for element c of row t: 8 elements share a call,
 *                element c takes the low (c even) or high (c odd) half of
 *                word (c mod 8) / 2 and is kept where it is >= 65536 p.
 *                Change `offset` (e.g. a step counter) for a fresh mask.
 *   offset_dev   device pointer to a further offset, added to `offset` when
 *                the kernel runs, or NULL: a captured graph draws a fresh
 *                mask at each replay if the word is changed between them
 *   token_base   index of the first row in the whole batch, as in
 *                moe_gate_noise: a sharded batch draws the single batch's mask
 * p = 0 keeps everything.  Dropped elements are selected away, not multiplied
 * by 0: Inf and NaN there have no effect. */
typedef struct {
  double p;
  uint64_t seed;
  uint64_t offset;
  const uint64_t* offset_dev;
  int64_t token_base;
} moe_dropout_t;

/* out[t,c] = add[t,c] + keep(t,c) * x[t,c] / (1 - p) over (cfg->T, width) rows.
 *   width  a multiple of 8 (cfg's d and d_out are not used); dtype MOE_F32 or
 *   MOE_BF16, of x, add and out; add may be NULL (nothing is added); out may
 *   be x or add.  fp32 arithmetic, one rounding.
 * Its gradient is the call itself on dLoss/d out (add: a gradient to add to). */
int moe_dropout(const moe_config_t* cfg, const moe_dropout_t* drop, int32_t width, int32_t dtype,
                const void* x, const void* add, void* out, moe_stream_t stream);

/* The combine with dropout and a residual in one pass:
 *   output[t] = residual[t] + keep[t] / (1 - p) * sum_j gates[t,j] *
 *               y_perm[dest[t,j]]  over the kept slots (moe_combine's sum)
 * residual (T, d_out) act_dtype or NULL (0); output may be residual; the other
 * arguments as moe_combine.  The mask's rows are d_out wide.
 * moe_combine_dropout_backward: moe_combine_backward for this forward, with
 * D = keep * dy / (1 - p) in the place of dy (the residual's gradient is dy).
 * y_perm is not multiplied where the mask dropped. */
int moe_combine_dropout(const moe_config_t* cfg, const moe_dropout_t* drop, const void* y_perm,
                        const int32_t* dest, const float* gates, const void* residual,
                        void* output, moe_stream_t stream);
int moe_combine_dropout_backward(const moe_config_t* cfg, const moe_dropout_t* drop,
                                 const void* dy, const void* y_perm, const int32_t* dest,
                                 const float* gates, float* dy_perm, float* dgates,
                                 moe_stream_t stream);

/* Low-rank adapters of many requests at once, beside a projection that all
 * requests share: the layer itself, from x (T, d) to output (T, d_out).  Token
 * t of a request with adapter a = token_adapter[t] gets
 *   output[t] = base[t] + u[t] B_a,   u[t] = scale_a x[t] A_a
 * and a token with a negative one output[t] = base[t].  bf16 activations;
 * 1 <= n_adapters <= 1024; rank a multiple of 8, at most 128; T <= 2^30.
 *
 * moe_adapter_plan groups the tokens by adapter.  A plan serves every later
 * call on the same T, n_adapters and token_adapter (all layers of a step,
 * forward and backward), which only read it.
 *   token_adapter (T) int32; an index >= n_adapters is recorded (code 1) and
 *                 treated as none
 *   plan          moe_adapter_plan_size bytes, 256-byte aligned.  Its first
 *                 256 bytes hold an error word (moe_workspace_init before the
 *                 first plan, moe_device_status); a call whose T or
 *                 n_adapters are not the plan's, or without a plan, does
 *                 nothing and records code 5.
 * moe_adapter:
 *   x (T, d) bf16; A (n_adapters, d, rank) bf16; B (n_adapters, rank, d_out)
 *   bf16; scale (n_adapters) fp32; base (T, d_out) bf16 or NULL (0);
 *   output (T, d_out) bf16 out, may be base, must not overlap x;
 *   u (T, rank) fp32 out or NULL: kept for the backward (rows of tokens
 *   without an adapter are left untouched); output is the same either way
 * moe_adapter_backward, for dy = dLoss/d output (T, d_out) bf16:
 *   v[t] = scale_a dy[t] B_a^T
 *   dx[t] = dx_add[t] + v[t] A_a^T        (dx_add alone without an adapter)
 *   dA_a = sum_t x[t]^T v[t],  dB_a = sum_t u[t]^T dy[t]
 *   u as moe_adapter wrote it; dx_add (T, d) fp32 or NULL (0); dx (T, d) fp32
 *   out, may be dx_add; dA, dB fp32 out, shaped like A and B, every adapter's
 *   written (0 for one without tokens).  base's gradient is dy.
 *   ws: moe_adapter_workspace_size bytes, 256-byte aligned.
 * Tensor cores with fp32 sums; u and v are fp32 and enter the products as sums
 * of bf16 terms: two (16 bits) for the bf16 output, three (24 bits) for dx, dA
 * and dB.  Where one is infinite, or rounds to bf16's infinity, its row and the
 * gradients of its adapter are NaN.  Fixed orders, no floating-point atomics.
 * Calls on several streams may share a plan; each needs a workspace of its own.
 * n_adapters is the number loaded, and every call's cost follows it: the plan
 * reads token_adapter n_adapters + 1 times from L2 (131072 tokens on 1024
 * adapters 152 us, on 64 36 us), and the row tiles are chosen as if the tokens
 * were spread over all of them.  A batch that uses a few of many adapters is
 * faster on tensors of those alone. */
size_t moe_adapter_plan_size(const moe_config_t* cfg, int32_t n_adapters);
int moe_adapter_plan(const moe_config_t* cfg, int32_t n_adapters, const int32_t* token_adapter,
                     void* plan, size_t plan_bytes, moe_stream_t stream);
int moe_adapter(const moe_config_t* cfg, int32_t n_adapters, int32_t rank, void* plan,
                size_t plan_bytes, const void* x, const void* A, const void* B,
                const float* scale, const void* base, void* output, float* u,
                moe_stream_t stream);
size_t moe_adapter_workspace_size(const moe_config_t* cfg, int32_t n_adapters, int32_t rank);
int moe_adapter_backward(const moe_config_t* cfg, int32_t n_adapters, int32_t rank, void* plan,
                         size_t plan_bytes, const void* x, const float* u, const void* dy,
                         const void* A, const void* B, const float* scale, const float* dx_add,
                         float* dx, float* dA, float* dB, void* ws, size_t ws_bytes,
                         moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_B200_PACKED_H */
