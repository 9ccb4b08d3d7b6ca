/*
 * mok_ops.h - operators around the MoE layer of mok.h: routing to experts, low-rank
 * adapters beside a shared projection, and counter-based dropout. (No counterpart in the
 * articles that mok.h cites.)
 *
 * Routing feeds the layer: its topk_idx and gates are what mok_plan takes with
 * dims.router = 0, and the dgates that mok_moe_bwd writes are what mok_route_bwd takes.
 * Adapted projections are the layer's dense neighbours: the projections of a shared expert
 * or a router's logits, with one frozen weight matrix and many small adapters.
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

#ifdef __cplusplus
}
#endif
#endif /* MOK_OPS_H_ */
