/*
 * mm_ops.h -- C ABI of the operators beside the fused MoE-FFN layer (mm.h), in the same library:
 *
 *   mm_residual_norm_*   the step between two blocks: the norm after a block, its gate, the scaled
 *                        residual sum and the norm before the next block, forward and backward;
 *   mm_router_*          top-k selection over expert logits, the routing weights and the loss
 *                        statistics, forward and backward: what mm_forward takes as topk_ids and
 *                        topk_weights;
 *   mm_decode            the whole MoE layer for a few tokens (inference): router product,
 *                        selection, experts and weighted sum in two or three launches, with bf16
 *                        expert weights or e4m3 ones that carry a scale per 128 x 128 block;
 *   mm_quantize_blocks   bf16 weights to e4m3 and the scales of their blocks.
 *
 * The rules of mm.h hold here too: row-major contiguous device memory, every buffer (workspaces
 * included) belongs to the caller, nothing is allocated, all work is enqueued on `stream` and
 * nothing synchronises with the host. Host-side checks return an error before anything is
 * enqueued; mm_last_error_detail and mm_status_string describe it. Host threads may call
 * concurrently on different workspaces. Pointers are aligned to their element; 16-byte alignment
 * where a function says so. Sums, statistics and products are held in 32 bits; every output is
 * rounded once to its type. Results depend on the inputs and the device's SM count only.
 */
#ifndef MM_OPS_H_
#define MM_OPS_H_

#include "mm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mm_dtype { MM_BF16 = 0, MM_FP32 = 1, MM_E4M3 = 2 } mm_dtype;

/* Version of this header's functions and structs (mm_abi_version is mm.h's). */
int mm_ops_version(void);

/* ---- residual_norm ------------------------------------------------------------------------
 *
 *   p[t]  = f[t] * rsqrt(mean(f[t]^2) + eps) * post_weight       (p = f without a post weight)
 *   r'[t] = residual_scale * r[t] + gate[t / (T / groups)] * p[t]         (gate = 1 without one)
 *   n[t]  = r'[t] * rsqrt(mean(r'[t]^2) + eps) * pre_weight
 *
 * r (residual) and r' (residual_out) have the stream type, f (branch) and n (normed) the block
 * type, the two weights and the gate the parameter type; a gradient has the type of what it is
 * the gradient of. Type triples: stream bf16 or fp32, block no wider than the stream, parameters
 * bf16 or fp32. A gate has `groups` rows of H, each for T / groups consecutive tokens (1: one
 * gate per channel; T: one per token; 0: no gate).
 * Sizes: T >= 0 (T = 0 does nothing forward and writes zero parameter gradients backward),
 * 1 <= H <= 16384, T a multiple of groups. Fastest are H a multiple of 8 and 16-byte aligned
 * tensors; aligned tensors of other widths up to 3840 come next.
 * Device waits are bounded. One that runs out (a failing device) leaves NaN in the rows of its block
 * that were still to come, and in the parameter gradients. */
typedef struct mm_norm_desc {
  int64_t T, H, groups;
  int32_t stream_type, block_type, param_type; /* mm_dtype */
  float residual_scale, eps;
} mm_norm_desc;

/* branch may be NULL (a norm before the first block: r' = residual_scale * r; no post weight or
 * gate then). pre_weight and normed are both given or both NULL (after the last block: no norm
 * before). residual_out may be NULL (r' not wanted) and may be `residual` itself. */
mm_status mm_residual_norm_forward(const mm_norm_desc* d, const void* residual, const void* branch,
                                   const void* post_weight, const void* pre_weight,
                                   const void* gate, void* residual_out, void* normed,
                                   void* stream);

/* Bytes of workspace the backward needs (0: unsupported sizes). Needs no initialisation. */
size_t mm_residual_norm_workspace_size(const mm_norm_desc* d);

/* Gradients at the forward's residual_out (r', as stored) and branch, for the gradients of r' and
 * n. Both norms' statistics are computed from these inputs. d_residual_out may be NULL (zero);
 * d_normed is given exactly if pre_weight is. d_branch, d_post_weight, d_pre_weight and d_gate are
 * given exactly if branch, post_weight, pre_weight and gate are. d_residual may be d_residual_out
 * itself. The parameter gradients are sums over tokens in a fixed order. Workspace: 256-byte
 * aligned. */
mm_status mm_residual_norm_backward(const mm_norm_desc* d, const void* residual_out,
                                    const void* branch, const void* post_weight,
                                    const void* pre_weight, const void* gate,
                                    const void* d_residual_out, const void* d_normed,
                                    void* d_residual, void* d_branch, void* d_post_weight,
                                    void* d_pre_weight, void* d_gate, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* Test hook: while on, residual_norm calls of this host thread let the loads of one block stop after
 * its first row (in the kernels that load rows ahead) and limit device waits to 50 ms. */
void mm_residual_norm_test_stall(int on);

/* ---- router -------------------------------------------------------------------------------
 *
 * Over logits z [T, E] (bf16 or fp32), per token:
 *   key_e = z_e + bias_e (MM_SCORE_SOFTMAX), sigmoid(z_e) + bias_e (MM_SCORE_SIGMOID with a bias),
 *           z_e (no bias); the K largest keys are selected, largest first, equal ones from the
 *           lowest expert up. -0 equals 0; NaN ranks below -inf.
 *   a_e   = exp(z_e - max z) or sigmoid(z_e);  A = sum_e a_e
 *   weight of a selected expert j, without the bias:
 *     normalize:   scale * a_j / sum of the selected a   (all 0 where that sum is 0: a token whose
 *                  selected logits are all -inf)
 *     otherwise:   scale * a_j / A (softmax; 0 where every logit is -inf) or scale * a_j (sigmoid)
 *   prob_sum_e = sum_t a_te / A_t     (a row whose A is 0 adds nothing)
 *   lse_t = log sum_e exp(z_te)       (-inf for a row of -inf)
 * prob_sum and lse are the statistics of load-balancing and z losses; each may be NULL.
 * topk_ids are distinct and in [0, E) for any input, so they are valid for mm_forward.
 * Sizes: T >= 0, 1 <= E <= 1024, 1 <= K <= 16, K <= E. */
#define MM_SCORE_SOFTMAX 0
#define MM_SCORE_SIGMOID 1
typedef struct mm_router_desc {
  int64_t T;
  int32_t E, K;
  int32_t logits_type; /* MM_BF16 or MM_FP32 */
  int32_t score;       /* MM_SCORE_* */
  int32_t normalize;
  float scale;
} mm_router_desc;

/* Bytes of workspace for a forward that writes prob_sum (0: unsupported sizes). */
size_t mm_router_workspace_size(const mm_router_desc* d);

/* bias fp32 [E] or NULL; topk_ids int32 [T, K], topk_weights fp32 [T, K]; prob_sum fp32 [E] or
 * NULL (the workspace, 256-byte aligned, is needed only with it), lse fp32 [T] or NULL. */
mm_status mm_router_forward(const mm_router_desc* d, const void* logits, const float* bias,
                            int32_t* topk_ids, float* topk_weights, float* prob_sum, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream);

/* d_logits (the logits' type) from the gradients of topk_weights (fp32 [T, K]), prob_sum (fp32
 * [E] or NULL) and lse (fp32 [T] or NULL). topk_ids are the forward's; an id outside [0, E)
 * contributes nothing. The selection itself has no gradient. Masked (-inf) logits get a gradient
 * of 0. */
mm_status mm_router_backward(const mm_router_desc* d, const void* logits, const int32_t* topk_ids,
                             const float* d_topk_weights, const float* d_prob_sum,
                             const float* d_lse, void* d_logits, void* stream);

/* ---- decode -------------------------------------------------------------------------------
 *
 * The whole MoE layer for T <= 64 tokens with T * K <= 1024, inference only, in two launches (three
 * with a router from 13 tokens on):
 *   logits = x router^T (fp32), selection and weights as the router above (or the caller's ids
 *   and weights), y_t = sum_k w_tk o_tk + o_shared_t with o = (silu(x Wg) * (x Wu)) Wd. Products
 *   and sums are in 32 bits, y is rounded once. Between the two products, w * h is kept as the sum
 *   of two bf16 numbers (16 significant bits). With e4m3 weights x is the sum of two e4m3 numbers
 *   and w * h of three, times a power of two (of a row of x; of a row and 128 columns of h): 8 (12)
 *   significant bits of every value down to 2^-13 of the row's (its 128 columns') largest, in steps
 *   of at most 2^-20 (2^-24) of the largest below that.
 * Every selected expert's weights are read once per 32 (e4m3: 16) of its tokens.
 *
 * weight_type MM_BF16: up bf16 [E, H, 2I], down bf16 [E, I, H] as in mm.h; H, I, shared_I multiples
 * of 8. MM_E4M3: the same shapes in e4m3 with fp32 scales of their 128 x 128 blocks,
 * up_scale [E, ceil(H/128), ceil(2I/128)], down_scale [E, ceil(I/128), ceil(H/128)] (rows and
 * columns counted over the whole matrix, so a block may hold the last gate and the first up
 * columns); a weight's value is its e4m3 number times its block's scale. H and both I multiples
 * of 16. The shared expert's matrices have the experts' type, E = 1.
 * Sizes: H, I, shared_I <= 65536, E <= 1024, K <= 16. */
typedef struct mm_decode_desc {
  mm_dims dims;
  int64_t shared_I; /* 0: no shared expert */
  int32_t weight_type;
  int32_t router_type; /* MM_BF16 or MM_FP32: the router weight's type */
  int32_t score, normalize;
  float scale;
} mm_decode_desc;

typedef struct mm_decode_weights {
  const void *up, *down;                     /* 16-byte aligned */
  const float *up_scale, *down_scale;        /* MM_E4M3 only */
  const void *shared_up, *shared_down;       /* with shared_I > 0 */
  const float *shared_up_scale, *shared_down_scale;
  const void* router;                        /* [E, H], 16-byte aligned; NULL: the caller routes */
  const float* router_bias;                  /* fp32 [E] or NULL */
} mm_decode_weights;

/* Bytes of workspace (0: unsupported). Needs no initialisation; one call at a time may use it. */
size_t mm_decode_workspace_size(const mm_decode_desc* d);

/* x, y bf16 [T, H], 16-byte aligned. With a router, topk_ids and topk_weights are outputs (either
 * may be NULL: not wanted); without one they are inputs, int32 and fp32 [T, K]; an id outside
 * [0, E) records MM_ERR_BAD_EXPERT_ID in the workspace's status word (mm_get_status) and y is NaN.
 * Device waits are bounded; one that runs out records MM_ERR_TIMEOUT the same way, and what of y was
 * not computed is NaN. */
mm_status mm_decode(const mm_decode_desc* d, const mm_decode_weights* w, const void* x,
                    int32_t* topk_ids, float* topk_weights, void* y, void* workspace,
                    size_t workspace_bytes, void* stream);

/* bf16 matrices w [n, R, C] to e4m3 q [n, R, C] and the scales [n, ceil(R/128), ceil(C/128)] of
 * their 128 x 128 blocks: scale = max |w| / 448 (1 for a block of zeros), q = w / scale rounded to
 * nearest even and saturated; a block with an infinity or a NaN gets a NaN scale. C a multiple of
 * 8, w 16-byte and q 8-byte aligned. */
mm_status mm_quantize_blocks(int64_t n, int64_t R, int64_t C, const void* w, void* q, float* scale,
                             void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MM_OPS_H_ */
