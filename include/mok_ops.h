/*
 * mok_ops.h - operators around the MoE layer of mok.h: routing to experts, its balance loss,
 * low-rank adapters beside a shared projection, counter-based dropout, the norm before a
 * block, and the optimiser step. (No counterpart in the articles that mok.h cites.)
 *
 * Routing feeds the layer: its topk_idx and gates are what mok_plan takes with
 * dims.router = 0, and the dgates that mok_moe_bwd writes are what mok_route_bwd takes.
 * Adapted projections are the layer's dense neighbours: the projections of a shared expert
 * or a router's logits, with one frozen weight matrix and many small adapters. The balance
 * loss takes what mok_route chose, and adds its gradient to mok_route_bwd's. The norm gives
 * the layer's x and takes its dX; the optimiser step takes the layer's weight gradients.
 *
 * Conventions as in mok.h: row-major dense tensors, caller-owned DEVICE pointers, calls
 * that only enqueue work on `stream` and never allocate device memory, argument errors
 * returned before anything is launched, bitwise reproducible results. These entry points
 * take no context; they run on the current CUDA device. Zero rows are a valid call.
 */
#ifndef MOK_OPS_H_
#define MOK_OPS_H_

#include <stddef.h>
#include <stdint.h>

#include "mok.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- routing to experts --------------------------------------------------------- */

/* Scores s of a token's E logits: MOK_SCORE_SOFTMAX over the E logits, or
 * MOK_SCORE_SIGMOID of each. */
typedef enum { MOK_SCORE_SOFTMAX = 0, MOK_SCORE_SIGMOID = 1 } mok_score;
/* Score of an expert group: its largest choice score, or the sum of its two largest. */
typedef enum { MOK_GROUP_MAX = 0, MOK_GROUP_TOP2 = 1 } mok_group_score;

/* Routing rule. Choice scores are c = s + bias, or without a bias the logits, which have the
 * scores' order (MOK_GROUP_TOP2 sums s also then). With groups > 1 the E experts form `groups`
 * groups of E / groups consecutive ids, and only experts of the top_groups best groups can be
 * chosen. The k largest choice scores are chosen; equal scores go to the lower id (group or
 * expert).
 * gates_j = scale * s_j, divided by the sum of the k chosen scores when renormalize != 0
 * (the bias steers the choice only). A logit of -inf or NaN masks its expert: score 0,
 * chosen only when fewer than k unmasked experts are left (lowest id first), then with gate
 * 0; a +inf logit counts as the largest finite value. All arithmetic is fp32.
 * 1 <= E <= 512, 1 <= k <= 32, 1 <= groups <= 32 dividing E, 1 <= top_groups <= groups,
 * k <= top_groups * (E / groups), scale finite. */
typedef struct {
  int E, k;
  int score;       /* mok_score */
  int groups, top_groups;
  int group_score; /* mok_group_score */
  int renormalize;
  float scale;
} mok_routing;

/* topk_idx [T][k] int32 and gates [T][k] fp32 in descending order of choice score, from
 * logits [T][E] (logits_type: MOK_OUT_BF16 or MOK_OUT_F32) and bias [E] fp32 or NULL. */
mok_status mok_route(const mok_routing* rule, int T, const void* logits,
                     mok_out_dtype logits_type, const float* bias, int32_t* topk_idx,
                     float* gates, void* stream);

/* dlogits [T][E] (dlogits_type) from dgates [T][k] fp32, the gradient of the gates, at the
 * choice topk_idx that mok_route made from these logits (the choice has no gradient). Every
 * element is written; experts without a gradient get 0. Ids outside [0, E) are ignored. */
mok_status mok_route_bwd(const mok_routing* rule, int T, const void* logits,
                         mok_out_dtype logits_type, const int32_t* topk_idx,
                         const float* dgates, void* dlogits, mok_out_dtype dlogits_type,
                         void* stream);

/* ---- dropout -------------------------------------------------------------------- */

/* y_i = (add_i or 0) + (keep_i ? x_i * 65536 / (65536 - t) : 0), t = round(65536 p), over n
 * elements of one type (MOK_OUT_BF16 or MOK_OUT_F32). keep_i: the i-th 16-bit word of the
 * Philox4x32-10 stream (J. Salmon et al., "Parallel random numbers: as easy as 1, 2, 3",
 * 2011) of key `seed` is at least t; counter offset + i / 8 gives elements 8 (i / 8) .. + 7,
 * words in order, low half first. The mask is never stored: the backward is the same call
 * on the gradient with the same p, seed and offset. A call uses (n + 7) / 8 counters.
 * 0 <= p and t < 65536. y may be x or add. */
mok_status mok_dropout(const void* x, const void* add, void* y, size_t n, float p,
                       uint64_t seed, uint64_t offset, mok_out_dtype type, void* stream);

/* ---- low-rank adapters beside a shared projection --------------------------------- */

/* T rows, K input and N output features (multiples of 8), n adapters of rank r
 * (1 <= r <= 128; adapters of smaller rank are padded with zeros). T up to 2^24, K, N and n up to
 * 2^20. The backward reads the ids once per adapter: its cost has a part that grows with n T. */
typedef struct {
  int T, K, N, n, r;
} mok_lora_dims;

/* W [K][N] bf16, the shared projection; A [n][r][K] and B [n][r][N] bf16; scale [n] fp32.
 * 16-byte aligned. */
typedef struct {
  const void* W;
  const void* A;
  const void* B;
  const float* scale;
} mok_lora_weights;

typedef struct {
  size_t saved_bytes;     /* written by mok_lora_fwd, read by mok_lora_bwd  */
  size_t workspace_bytes; /* scratch of mok_lora_bwd                        */
} mok_lora_sizes;

mok_status mok_lora_get_sizes(const mok_lora_dims* dims, mok_lora_sizes* out);

/* y [T][N] (out) = x W, plus in each row t with an adapter a = ids[t]
 *   scale[a] (xa A_a^T) B_a,
 * xa = x_ad when given (the adapters' own input, e.g. x after dropout), else x [T][K] bf16.
 * ids [T] int32 on the device; a row whose id lies outside [0, n) has no adapter. Rows may
 * come in any order; an adapter's values reach its own rows only, also when they are not
 * finite. Sums are fp32; the r values xa A_a^T enter the second product as the sum of two
 * bf16 values (16 significant bits). `saved` (mok_lora_sizes.saved_bytes, 256-byte aligned)
 * is scratch of this call and, for training, an input of mok_lora_bwd. `status`, when not
 * NULL, is a device word that the caller zeroed (mok_lora_get_status). */
mok_status mok_lora_fwd(const mok_lora_dims* dims, const mok_lora_weights* w, const void* x,
                        const void* x_ad, const int32_t* ids, void* y, mok_out_dtype out,
                        void* saved, uint32_t* status, void* stream);

/* Gradients for dY [T][N] bf16, W frozen, all in the type `out`:
 *   dX [T][K] = dY W^T + dXa, dXa_t = scale[a] (dY_t B_a^T) A_a (0 without an adapter);
 *   dA [n][r][K], dB [n][r][N], summed over the rows of each adapter in ascending order
 *   (zeros for an adapter without rows).
 * With x_ad, the gradient dXa of the adapters' own input goes to dXa [T][K] and dX holds
 * dY W^T alone; without x_ad, dXa must be NULL. `workspace`: mok_lora_sizes.workspace_bytes,
 * 256-byte aligned. `saved` as mok_lora_fwd left it for the same dims, weights, inputs. */
mok_status mok_lora_bwd(const mok_lora_dims* dims, const mok_lora_weights* w, const void* x,
                        const void* x_ad, const int32_t* ids, const void* saved,
                        const void* dY, void* dX, void* dXa, void* dA, void* dB,
                        mok_out_dtype out, void* workspace, uint32_t* status, void* stream);

/* Synchronise `stream`, read and clear a status word of the calls above: MOK_OK, or
 * MOK_ERR_TIMEOUT when a device wait passed its bound of two seconds. */
mok_status mok_lora_get_status(uint32_t* status, void* stream);

/* ---- norm before a block --------------------------------------------------------- */

typedef enum { MOK_NORM_LAYER = 0, MOK_NORM_RMS = 1 } mok_norm_kind;

/* T rows of H elements, 0 <= T <= 2^31 - 1, 1 <= H <= 32768; eps >= 0, finite. Types
 * (MOK_OUT_BF16 or MOK_OUT_F32) of three groups of tensors: x_type of the stream (x, add, h,
 * dX), y_type of the normalised rows (y, dY), w_type of the parameters (w, b, dW, dB).
 * Addresses need their type's alignment only; tensors at 16-byte aligned addresses are the
 * fast case, rows of whole 16 bytes the fastest. */
typedef struct {
  int T, H;
  int kind; /* mok_norm_kind */
  float eps;
  mok_out_dtype x_type, y_type, w_type;
} mok_norm_dims;

typedef struct {
  size_t stats_bytes;     /* written by mok_norm_fwd, read by mok_norm_bwd */
  size_t workspace_bytes; /* scratch of mok_norm_bwd                       */
} mok_norm_sizes;

mok_status mok_norm_get_sizes(const mok_norm_dims* dims, mok_norm_sizes* out);

/* h = x + add, rounded to x_type (add and h both given), or h = x (both NULL); then per row
 *   MOK_NORM_LAYER  m = mean h, r = 1 / sqrt(mean (h - m)^2 + eps);   MOK_NORM_RMS  m = 0
 *   y = (h - m) r w + b                                               (b [H] may be NULL)
 * in fp32. stats: (m, r) of each row, 8-byte aligned, or NULL when no backward follows.
 * h may be x or add; y, where its type is theirs, may be one of them that h is not. */
mok_status mok_norm_fwd(const mok_norm_dims* dims, const void* x, const void* add, const void* w,
                        const void* b, void* h, void* y, float* stats, void* stream);

/* With xh = (h - m) r and t = dY w:
 *   dX = r (t - [mean t] - xh mean(t xh)) + add      ([..]: MOK_NORM_LAYER only)
 *   dW = sum over rows of dY xh;  dB = sum over rows of dY      (dB may be NULL)
 * add [T][H] (x_type) or NULL: the gradient that reaches h along the residual stream; dX is
 * the gradient of x and of mok_norm_fwd's add alike, and may be add. Row sums are fp32, in an
 * order that depends on the dims and the alignment only; T = 0 writes zeros. `workspace`:
 * mok_norm_sizes.workspace_bytes, 256-byte aligned. */
mok_status mok_norm_bwd(const mok_norm_dims* dims, const void* dY, const void* h, const void* w,
                        const float* stats, const void* add, void* dX, void* dW, void* dB,
                        void* workspace, void* stream);

/* ---- balance loss of a router ---------------------------------------------------- */

/* 1 <= E <= 512, 1 <= k <= 32; coef and z_coef >= 0, finite; score: mok_score. */
typedef struct {
  int E, k;
  int score;
  float coef, z_coef;
} mok_balance;

/* Bytes of `saved` for T rows in S sequences (at least 1): written by mok_balance_fwd, read
 * by mok_balance_bwd. */
mok_status mok_balance_get_sizes(const mok_balance* rule, int T, int S, size_t* saved_bytes);

/* Losses of logits [T][E] (logits_type) whose router chose topk_idx [T][k]. seqs: S + 1
 * ascending row offsets on the device, sequence s holding the rows seqs[s] .. seqs[s + 1] - 1
 * (S <= 2^20), or NULL: one sequence of all rows (S = 1). T_s: a sequence's rows, Tv: the
 * rows of all sequences; rows in none take no part (padding).
 *   p_te = s_te / sum_e s_te: softmax, or sigmoid scores over their sum
 *   c_se = choices of expert e in sequence s (ids outside [0, E) are not counted)
 *   losses[0] = coef   sum_s E / (k T_s Tv) sum_e c_se (sum_{t in s} p_te)
 *   losses[1] = z_coef / Tv  sum_t (log sum_e exp l_te)^2     (0 when z_coef is 0)
 * losses[0] is coef times the mean over rows of E sum_e f_e p_e with f_e the share of their
 * sequence's choices: coef for choices spread evenly. counts [E] int32: choices of all
 * sequences' rows. As in mok_route a logit of -inf or NaN masks its expert (p = 0) and +inf
 * is the largest finite value; a row without an unmasked expert has p = 0 and no part in
 * losses[1]. losses 4-, saved 256-byte aligned. Offsets that do not ascend, or lie outside
 * [0, T], give unspecified results, and no access outside the tensors. */
mok_status mok_balance_fwd(const mok_balance* rule, int T, const void* logits,
                           mok_out_dtype logits_type, const int32_t* topk_idx,
                           const int32_t* seqs, int S, float* losses, int32_t* counts,
                           void* saved, void* stream);

/* dlogits [T][E] (dlogits_type) = (add or 0) + dlosses[0] d losses[0] / d logits
 * + dlosses[1] d losses[1] / d logits; the choices have no gradient. dlosses: 2 fp32 values on
 * the device, or NULL for ones. add: dlogits_type, and dlogits may be add (mok_route_bwd's
 * result). Rows in no sequence get add or 0. logits, seqs, saved as for mok_balance_fwd. */
mok_status mok_balance_bwd(const mok_balance* rule, int T, const void* logits,
                           mok_out_dtype logits_type, const int32_t* seqs, int S,
                           const void* saved, const float* dlosses, const void* add,
                           void* dlogits, mok_out_dtype dlogits_type, void* stream);

/* ---- gradients of many tensors, and the step that applies them -------------------- */

/* A gradient of n elements on the device, in a type; n = 0 or NULL: none. */
typedef struct {
  const void* g;
  size_t n;
  mok_out_dtype type;
} mok_grad;

/* Bytes of mok_grad_norm's workspace for any number of tensors. */
mok_status mok_grad_norm_get_sizes(size_t* workspace_bytes);

/* norm = scale sqrt(sum of all squares), fp32 on the device (sums of squares in fp32 over runs
 * of elements whose squares neither overflow nor vanish, else in fp64; sums of runs in fp64);
 * coef = scale min(1, max_norm / norm), or NaN when norm is not finite: the factor that
 * mok_adamw takes. max_norm > 0, may be infinite; scale > 0 (the inverse of a loss scale, or
 * of the number of summed micro-batches). `grads`: a host array, read during the call.
 * `workspace`: 256-byte aligned. */
mok_status mok_grad_norm(int count, const mok_grad* grads, float max_norm, float scale,
                         float* norm, float* coef, void* workspace, void* stream);

/* One parameter tensor: n elements p of p_type with gradient g of g_type (NULL: the tensor
 * stays as it is in this step), decay: its weight decay. A bf16 p has its fp32 value in
 * mok_adamw_state.master. */
typedef struct {
  void* p;
  const void* g;
  size_t n;
  double decay;
  mok_out_dtype p_type, g_type;
} mok_adamw_tensor;

/* 0 <= beta < 1, eps > 0 (as fp32 a normal number), bits: 32 or 8, of the moments. */
typedef struct {
  double beta1, beta2, eps;
  int bits;
} mok_adamw_rule;

/* The state of all tensors, in one piece per kind: tensor i's elements begin at the sum of
 * the sizes before it, each rounded up to whole blocks of 256 elements. All 16-byte aligned;
 * a new state is all zeros, but for master, a copy of p.
 *   master  fp32, needed when a p is bf16 (else NULL); the places of fp32 tensors stay unused
 *   m, v    fp32 (bits = 32), or one byte an element (bits = 8) with
 *   scales  two bytes (a, b) per block, the exponent fields of the block's largest |m| and v:
 *           a code of m is an E4M3 value times 2^(a - 134); a code c > 0 of v stands for
 *           2^(c / 8 - 30) (1 + (c % 8) / 8) 2^(b - 127), 0 for 0. */
typedef struct {
  float* master;
  void* m;
  void* v;
  uint8_t* scales;
} mok_adamw_state;

/* elements: of the state, i.e. of n[0 .. count - 1] rounded up to whole blocks. */
mok_status mok_adamw_get_sizes(int count, const size_t* n, size_t* elements);

/* One step of AdamW over all tensors, in fp32:
 *   g' = coef g;  m = beta1 m + (1 - beta1) g';  v = beta2 v + (1 - beta2) g'^2
 *   p = p - lr decay p - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * with the step number t >= 1 and lr from host values, or from the device where t_dev (int32)
 * or lr_dev is given, so that a captured graph can advance them. coef: a device value, or
 * NULL for 1; a coef that is not finite skips the step, nothing is written. A bf16 p is the
 * rounded master. Moments in 8 bits are rounded after p has been computed. v goes up or down at
 * random so that its mean is kept (a nearest rounding would never move it), but never from above
 * 0 to 0, by 16-bit words of Philox4x32-7 keyed by `seed`: counter words (position / 8 in the
 * state, 64 bits; t; 0) give elements 8 (position / 8) .. + 7, words in order, low half first. m
 * goes to nearest (ties to even) where beta1 <= 0.9 and |m| >= 2^(a - 140), i.e. where a step's
 * decay is more than half a code, so that m follows a gradient that fades; a gradient that stays
 * leaves m at a code within 1 / 16 / (1 - beta1) of it, relative to m. Elsewhere m goes up or down
 * at random too, with the same words' bits in reverse order, the highest inverted. An m or v that
 * is not finite becomes an m of NaN and counts for no block's scale. `tensors`: a host array,
 * read during the call; p's may not overlap one another, gradients or the state. */
mok_status mok_adamw(const mok_adamw_rule* rule, int count, const mok_adamw_tensor* tensors,
                     const mok_adamw_state* state, double lr, const float* lr_dev, int t,
                     const int32_t* t_dev, const float* coef, uint64_t seed, void* stream);

/* The values of 8-bit moments of `elements` state elements (a multiple of 256) in bf16: exact, but
 * for an m in a block with a < 10 (none above 2^-117), which is rounded to bf16's last step 2^-133. */
mok_status mok_adamw_moments(size_t elements, const mok_adamw_state* state, void* m, void* v,
                             void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOK_OPS_H_ */
